// zn_kv.hip -- the key-value cache's bookkeeping (pages of a step's new tokens,
// their slots, pages that come back) and its rows (written and read by slots).
#include "zn_kv.h"

namespace zn {
namespace {

// ------------------------------------------------------------------ tables --
constexpr int kStepThreads = 256;
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t at_least_0(int32_t v) { return v < 0 ? 0u : uint32_t(v); }
__device__ __forceinline__ uint32_t clip(uint64_t v) { return v > kMost ? kMost : uint32_t(v); }

// The sum of v over the workgroup's threads before this one, and over all.
__device__ __forceinline__ uint64_t before(uint64_t v, uint64_t &sum) {
  __shared__ uint64_t part[kStepThreads / 64];
  const uint32_t wave = threadIdx.x >> 6;
  const uint64_t x = scan(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) part[wave] = x;
  __syncthreads();
  uint64_t at = x - v;
  sum = 0;
#pragma unroll
  for (uint32_t w = 0; w < kStepThreads / 64; w++) {
    if (w < wave) at += part[w];
    sum += part[w];
  }
  return at;
}

// The last i in [0, n) whose first[i] (without its top bit) is at most v; first
// rises, and first[0] <= v.
__device__ __forceinline__ uint32_t owner(const uint32_t *first, uint32_t n, uint32_t v) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if ((first[mid] & kMost) <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Bookkeeping is bound by latency (64 requests' step moves 4 KB): one launch, in
// which every workgroup makes the sums over the requests for itself (a load and
// a scan) and then does its share of pages and tokens by a search in the sums.
// A thread takes `per` requests in a row.  64 requests with a token each: 4.0 us to
// extend, 2.6 to release, most of it the launch and four loads that wait for each
// other; 512 requests with 123,000 tokens 8.8 (1.1 MB) and 4.8.
//
// LDS, a word each for every request: len; first, the pages before its own, with the
// top bit set if it is served; and begin, the tokens before its own, one more.
template <bool EXTEND>
__global__ __launch_bounds__(kStepThreads) void k_kv_step(KvStepArgs a) {
  extern __shared__ uint32_t lds[];
  uint32_t *len = lds, *first = lds + a.batch, *begin = lds + 2 * a.batch;
  __shared__ uint32_t most;
  const uint32_t per = (a.batch + kStepThreads - 1) / kStepThreads;
  const uint32_t b0 = min(threadIdx.x * per, a.batch), b1 = min(b0 + per, a.batch);
  const uint32_t round = (1u << a.shift) - 1;
  const uint32_t n_free = min(at_least_0(*a.n_free), a.free_cap);
  auto pages_of = [&](uint64_t tokens) { return (tokens + round) >> a.shift; };
  if (threadIdx.x == 0) most = 0;

  // tokens, then pages, of this thread's requests and of all before them
  uint64_t tokens = 0, all_tokens = 0;
  for (uint32_t b = b0; b < b1; b++) {
    len[b] = at_least_0(a.lens[b]);
    if constexpr (EXTEND) tokens += begin[b] = at_least_0(a.add[b]);   // for now
  }
  if constexpr (EXTEND) tokens = before(tokens, all_tokens);
  uint64_t pages = 0, all_pages, at_token = tokens;
  // what request b asks for
  auto wants = [&](uint32_t b, bool &fits) -> uint64_t {
    if constexpr (EXTEND) {
      const uint64_t want = pages_of(uint64_t(len[b]) + begin[b]);
      at_token += begin[b];
      fits = want <= a.width && at_token <= a.tokens;
      return fits ? want - pages_of(len[b]) : 0;
    } else {
      fits = a.done[b] != 0;
      return fits ? min(pages_of(len[b]), uint64_t(a.width)) : 0;
    }
  };
  bool fits;
  for (uint32_t b = b0; b < b1; b++) pages += wants(b, fits);
  uint64_t at_page = before(pages, all_pages);
  at_token = tokens;
  uint32_t taken = 0;
  for (uint32_t b = b0; b < b1; b++) {
    const uint64_t need = wants(b, fits);
    if constexpr (EXTEND) {
      const bool served = fits && (need == 0 || at_page + need <= n_free);
      const uint32_t more = begin[b];
      begin[b] = clip(at_token - more);
      first[b] = clip(at_page) | (served ? 0x80000000u : 0u);
      if (served && need) taken = uint32_t(at_page + need);
      if (blockIdx.x == 0) {
        a.new_lens[b] = int32_t(served ? len[b] + more : len[b]);
        a.starts[b] = int32_t(begin[b]);
      }
    } else {
      first[b] = clip(at_page);
      if (blockIdx.x == 0) a.new_lens[b] = fits ? 0 : int32_t(len[b]);
    }
    at_page += need;
  }
  if (EXTEND && threadIdx.x == 0) begin[a.batch] = clip(all_tokens);
  if (EXTEND && taken) atomicMax(&most, taken);
  __syncthreads();
  const uint32_t id = blockIdx.x * kStepThreads + threadIdx.x, step = gridDim.x * kStepThreads;
  if constexpr (EXTEND) {
    taken = most;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.starts[a.batch] = int32_t(clip(all_tokens));
      *a.n_left = int32_t(n_free - taken);
    }
    // tokens, four in a row a thread; a page that this step enters is looked up on the stack
    const uint32_t end = begin[a.batch];
    for (uint64_t t0 = 4ull * id; t0 < a.tokens; t0 += 4ull * step) {
      uint32_t b = t0 < end ? owner(begin, a.batch, uint32_t(t0)) : 0;
      int32_t page[4], place[4];
      bool live[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; i++) {
        const uint64_t t = t0 + i;
        live[i] = t < end && t < a.tokens;
        page[i] = -1;
        place[i] = 0;
        if (!live[i]) continue;
        while (t >= begin[b + 1]) b++;
        live[i] = first[b] >> 31;
        if (!live[i]) continue;
        const uint32_t p = len[b] + uint32_t(t) - begin[b], at = p >> a.shift, have = uint32_t(pages_of(len[b]));
        place[i] = int32_t(p);
        page[i] = at < have ? a.table[b * a.table_stride + at] : a.free[n_free - 1 - ((first[b] & kMost) + at - have)];
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; i++) {
        if (t0 + i >= a.tokens) break;
        const bool good = page[i] >= 0 && uint32_t(page[i]) < a.n_pages;
        a.slots[t0 + i] = good ? int32_t((uint32_t(page[i]) << a.shift) | (uint32_t(place[i]) & round)) : -1;
        a.positions[t0 + i] = place[i];
      }
    }
    // pages: the i-th one taken is the i-th from the stack's end
    for (uint32_t i = id; i < taken; i += step) {
      const uint32_t b = owner(first, a.batch, i);
      a.table[b * a.table_stride + pages_of(len[b]) + i - (first[b] & kMost)] = a.free[n_free - 1 - i];
    }
  } else {
    const uint32_t room = a.free_cap - n_free;
    const uint32_t back = all_pages < room ? uint32_t(all_pages) : room;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_left = int32_t(n_free + back);
    for (uint32_t i = id; i < back; i += step) {
      const uint32_t b = owner(first, a.batch, i);
      a.free[n_free + i] = a.table[b * a.table_stride + i - first[b]];
    }
  }
}

template <bool EXTEND>
hipError_t step(const KvStepArgs &a, uint64_t work, hipStream_t s) {
  // four tokens a thread; more workgroups only repeat the sums
  const uint64_t grid = (work + 4 * kStepThreads - 1) / (4 * kStepThreads);
  const uint32_t lds = (3 * a.batch + 1) * sizeof(uint32_t);
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&k_kv_step<EXTEND>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e != hipSuccess) return e;
  }
  k_kv_step<EXTEND><<<uint32_t(grid < 1 ? 1 : grid > 256 ? 256 : grid), kStepThreads, lds, s>>>(a);
  return hipGetLastError();
}

// -------------------------------------------------------------------- rows --
// Eight consecutive elements of a dense row, at their own alignment.
template <int DT>
__device__ __forceinline__ void take8(const uint8_t *p, float (&v)[8]) {
  if constexpr (DT == BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const f32x4 x = *reinterpret_cast<const f32x4_any *>(p), y = *reinterpret_cast<const f32x4_any *>(p + 16);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = x[i];
      v[4 + i] = y[i];
    }
  }
}

// Group g of 8 values -> token, head and place within the row; the blocks of one
// row lie on neighbouring lanes, a block on one quad.
struct RowMap {
  FastDiv per_row, heads;  // groups of a row; heads
  __device__ __forceinline__ void at(uint32_t g, uint32_t &t, uint32_t &h, uint32_t &in_row) const {
    const uint32_t row = per_row.div(g);
    in_row = g - row * per_row.d;
    t = heads.div(row);
    h = row - t * heads.d;
  }
};

__device__ __forceinline__ bool slot_at(const KvCache &c, int32_t slot, uint32_t h, uint64_t &block) {
  if (slot < 0 || (uint32_t(slot) >> c.shift) >= c.n_pages) return false;
  const uint32_t page = uint32_t(slot) >> c.shift, place = uint32_t(slot) & ((1u << c.shift) - 1);
  block = page * c.page_stride + h * c.head_stride + place * c.place_stride;
  return true;
}

// Quantises as k_mx_quantize does: a lane takes 8 values, a quad shares out a
// block's maximum.  Keys and values are the grid's y = 0 and 1.  Bound by memory: 32768
// tokens of 8 heads of 128 values (BF16, 170 MB) 43 us, 3.9 TB/s; 64 tokens 3.2 us,
// the launch.  Two groups a lane; one or
// four made no difference, nor did 4, 16 or 64 tokens of a head beside each other.
template <int DT, int U>
__global__ __launch_bounds__(256) void k_kv_write(KvRowsArgs a, RowMap m, uint32_t groups) {
  const bool keys = blockIdx.y == 0;
  const uint8_t *x = keys ? a.k : a.v;
  uint8_t *codes = keys ? a.c.k : a.c.v, *scales = keys ? a.c.ks : a.c.vs;
  const uint64_t ts = keys ? a.k_token : a.v_token, hs = keys ? a.k_head : a.v_head;
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  float v[U][8];
  uint64_t block[U];
  uint32_t r[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    uint32_t t, h;
    m.at(g < groups ? g : 0, t, h, r[u]);
    live[u] = g < groups && slot_at(a.c, a.slots[t], h, block[u]);
    take8<DT>(x + (t * ts + h * hs + r[u] * 8) * esize(DT), v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t b = __float_as_uint(v[u][i]) & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
    const uint32_t s = mx_scale_byte<FP4X2>(quad_max(top));
    const u32x2 c = s == 255u ? u32x2{0, 0} : mx_codes8<FP4X2>(v[u], mx_inverse(s));
    if (!live[u]) continue;
    const uint64_t b = block[u] + (r[u] >> 2);
    *reinterpret_cast<uint32_t *>(codes + b * 16 + (r[u] & 3) * 4) = c[0];
    if ((r[u] & 3) == 0) scales[b] = uint8_t(s);
  }
}

// The way back: the same 170 MB in 36 us, 4.8 TB/s.
template <int DT, int U>
__global__ __launch_bounds__(256) void k_kv_read(KvRowsArgs a, RowMap m, uint32_t groups) {
  const bool keys = blockIdx.y == 0;
  const uint8_t *codes = keys ? a.c.k : a.c.v, *scales = keys ? a.c.ks : a.c.vs;
  uint8_t *out = keys ? a.k_out : a.v_out;
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  uint32_t w[U], s[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    uint32_t t, h, r;
    uint64_t block;
    m.at(g < groups ? g : 0, t, h, r);
    w[u] = s[u] = 0;
    if (g < groups && slot_at(a.c, a.slots[t], h, block)) {
      w[u] = *reinterpret_cast<const uint32_t *>(codes + (block + (r >> 2)) * 16 + (r & 3) * 4);
      s[u] = scales[block + (r >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t g = first + 256u * u;
    if (g >= groups) continue;
    const float f = mx_scale_value(s[u]);
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3);
    const f32x4 lo = {p0[0] * f, p0[1] * f, p1[0] * f, p1[1] * f}, hi = {p2[0] * f, p2[1] * f, p3[0] * f, p3[1] * f};
    if constexpr (DT == BF16) {
      const u32x4 o = {f32_bf16x2(lo[0], lo[1]), f32_bf16x2(lo[2], lo[3]), f32_bf16x2(hi[0], hi[1]), f32_bf16x2(hi[2], hi[3])};
      *reinterpret_cast<u32x4_any *>(out + uint64_t(g) * 16) = o;
    } else {
      *reinterpret_cast<f32x4_any *>(out + uint64_t(g) * 32) = lo;
      *reinterpret_cast<f32x4_any *>(out + uint64_t(g) * 32 + 16) = hi;
    }
  }
}

// Calls f(first token, tokens) for pieces whose groups of 8 stay below 2^31.
template <class F>
hipError_t by_tokens(const KvRowsArgs &a, F f) {
  const uint64_t most = 0x7FFF0000u / (uint64_t(a.c.heads) * a.c.blocks * 4);
  for (uint64_t t = 0; t < a.tokens; t += most) {
    const hipError_t e = f(t, a.tokens - t < most ? a.tokens - t : most);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t write_rows(const KvRowsArgs &a, hipStream_t s) {
  constexpr int U = 2;
  const uint32_t per_row = a.c.blocks * 4;
  return by_tokens(a, [&](uint64_t t0, uint64_t tokens) {
    KvRowsArgs p = a;
    p.k += t0 * a.k_token * esize(DT);
    p.v += t0 * a.v_token * esize(DT);
    p.slots += t0;
    const uint32_t groups = uint32_t(tokens * a.c.heads * per_row);
    k_kv_write<DT, U><<<dim3((groups + 256 * U - 1) / (256 * U), 2), 256, 0, s>>>(
        p, RowMap{FastDiv(per_row), FastDiv(a.c.heads)}, groups);
    return hipGetLastError();
  });
}

template <int DT>
hipError_t read_rows(const KvRowsArgs &a, hipStream_t s) {
  constexpr int U = 2;
  const uint32_t per_row = a.c.blocks * 4;
  return by_tokens(a, [&](uint64_t t0, uint64_t tokens) {
    KvRowsArgs p = a;
    const uint64_t skip = t0 * a.c.heads * per_row * 8 * esize(DT);
    p.k_out += skip;
    p.v_out += skip;
    p.slots += t0;
    const uint32_t groups = uint32_t(tokens * a.c.heads * per_row);
    k_kv_read<DT, U><<<dim3((groups + 256 * U - 1) / (256 * U), 2), 256, 0, s>>>(
        p, RowMap{FastDiv(per_row), FastDiv(a.c.heads)}, groups);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_kv_extend(const KvStepArgs &a, hipStream_t s) { return step<true>(a, a.tokens, s); }
hipError_t launch_kv_release(const KvStepArgs &a, hipStream_t s) {
  return step<false>(a, uint64_t(a.batch) * a.width / 8, s);
}
hipError_t launch_kv_write(int dtype, const KvRowsArgs &a, hipStream_t s) {
  return dtype == BF16 ? write_rows<BF16>(a, s) : write_rows<FP32>(a, s);
}
hipError_t launch_kv_read(int dtype, const KvRowsArgs &a, hipStream_t s) {
  return dtype == BF16 ? read_rows<BF16>(a, s) : read_rows<FP32>(a, s);
}

}  // namespace zn
