// zn_attn.hip -- attention over the key-value cache in 4 bits.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q.k_j - m),  c = scale log2(e),
//
// in one pass over the keys: m is a running bound of the exponents.  When one
// passes it, it rises to 8 above that one and the sums so far are multiplied by
// 2^(old - new); with the 8 this is seldom, and weights stay under 1.
//
// Rows and tiles.  All queries of a request that read one key head share its
// keys: row r of such a group is query r / group, query head r % group.  A wave
// takes 16 rows and 64 keys at a time with v_mfma_f32_16x16x32_bf16, keys as the
// first operand: the scores come out with a lane holding row l % 16 and keys 4 j
// + i of each 16 (j = l / 16).  That is already the layout of the second operand
// of the product with the values, whose 8 keys a lane may be any as long as the
// values agree; no score moves between lanes.
//   Keys: the first operand wants 8 values of one key a lane and step; which 8
// is free too, so a lane reads its quarter of a row, consecutive (NB dwords, for
// 128 values one block with its scale), straight from memory.
//   Values: the first operand wants 8 keys of one value, across rows.  A lane
// converts whole blocks (one scale each) to BF16, writes them to LDS as they
// lie, and reads them back through ds_read_b64_tr_b16, 4 keys of 16 values at a
// time.  Rows are 32 bytes apart modulo 64, so eight of them fill the banks.
// Codes become BF16 exactly: 2 significant bits and BF16's range.
#include "zn_kv.h"

namespace zn {
namespace {

constexpr int kTile = 64;       // keys a wave takes at a time
constexpr int kWaves = 4;       // of a workgroup, which share out its keys
constexpr float kRise = 8.0f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The largest of the four lanes l % 16 + 16 j (NaNs lose), by exchanges of 16 and
// 32 lanes: two registers that hold the same come out with both halves in each.
__device__ __forceinline__ float max_j(float x) {
  const uint32_t w = __float_as_uint(x);
  const auto p = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t y = __float_as_uint(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
  const auto q = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_j(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// A wave's own LDS operations run in order; the compiler keeps it.
__device__ __forceinline__ void lds_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Eight codes under a scale (a float's exponent field: 0 is 2^-127, 255 a NaN).
__device__ __forceinline__ bf16x8 values8(uint32_t w, float s) {
  union {
    bf16x2 p[4];
    bf16x8 all;
  } o;
  o.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  o.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  o.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  o.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return o.all;
}
// Bytes over 252 would leave BF16's range: NaNs, like 255.
__device__ __forceinline__ float scale_of(uint32_t s) {
  return __uint_as_float(s > 252u ? 0x7FC00000u : s << 23);
}

// Eight FP32 values as N BF16 pieces whose sum they are (up to 2^-(8 N) of them).
template <int N>
__device__ __forceinline__ void pieces(const float (&x)[8], bf16x8 (&out)[N]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; i++) rest[i] = x[i];
#pragma unroll
  for (int n = 0; n < N; n++) {
    union {
      uint32_t w[4];
      bf16x8 all;
    } o;
#pragma unroll
    for (int i = 0; i < 4; i++) o.w[i] = f32_bf16x2(rest[2 * i], rest[2 * i + 1]);
    out[n] = o.all;
    if (n + 1 < N) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        rest[2 * i] -= bf16_lo(o.w[i]);
        rest[2 * i + 1] -= bf16_hi(o.w[i]);
      }
    }
  }
}

// Eight keys of one value from LDS: 4 rows from `p`, 4 from `p + next`, where this
// lane's address is its part of a row (4 values of a row a lane, 4 lanes a row).
union Turned {
  s16x4 half[2];
  bf16x8 all;
  uint16_t bits[8];
};
__device__ __forceinline__ Turned turned(const uint8_t *p, int next) {
  typedef __attribute__((address_space(3))) s16x4 lds16;
  Turned t;
  t.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds16 *)(p));
  t.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds16 *)(p + next));
  return t;
}

// A request of the call: its queries and the keys that any of them sees.
struct Request {
  uint32_t start, n, len;    // first query, queries, keys in the cache
  uint32_t lo, tiles;        // tiles of keys from lo (a multiple of kTile) to len
  bool bad;                  // longer than its table
};
__device__ __forceinline__ Request request(const AttnArgs &a, uint32_t b) {
  Request r;
  if (a.starts) {
    const int32_t s = a.starts[b], e = a.starts[b + 1];
    const uint32_t from = s < 0 ? 0 : min(uint32_t(s), a.tokens), to = e < 0 ? 0 : min(uint32_t(e), a.tokens);
    r.start = from;
    r.n = to > from ? to - from : 0;
  } else {
    r.start = b;
    r.n = 1;
  }
  const int32_t len = a.lens[b];
  r.len = len < 0 ? 0 : uint32_t(len);
  r.bad = r.len > (uint64_t(a.width) << a.c.shift);
  if (r.bad) r.len = 0;
  const uint32_t back = r.n + a.window - 1;   // keys before the end that the first query's window reaches
  r.lo = a.window && r.len > back ? (r.len - back) / kTile * kTile : 0;
  r.tiles = r.n ? (r.len - r.lo + kTile - 1) / kTile : 0;
  return r;
}

// How the work is shared out.  Rows go in groups of ROWS (a power of two), the
// keys of a group in pieces of `piece` tiles, so that a head's items, (request,
// rows, piece), come to about `items`: with tiles t_b and row groups g_b,
//   sum g_b ceil(t_b / piece) <= sum g_b t_b / piece + sum g_b <= items + sum g_b.
// Every workgroup finds its own item from the lengths (two sums over the
// requests); the host knows the bound alone.
struct Plan {
  uint32_t items;      // wanted of a head
  uint32_t least;      // tiles of a piece at least
};
struct Item {
  uint32_t b, group, piece, pieces, first;   // first: item number of the request's first
  uint32_t from, to;                         // tiles of keys
};

template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t &sum) {
  __shared__ uint32_t part[THREADS / 64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t p = __shfl_up(x, d);
    if (lane >= uint32_t(d)) x += p;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  uint32_t before = 0;
  sum = 0;
#pragma unroll
  for (uint32_t w = 0; w < THREADS / 64; w++) {
    if (w < wave) before += part[w];
    sum += part[w];
  }
  return x - v + before;
}

// Row groups and items are counted in 32 bits: the host keeps tokens * group +
// batch below 2^30, and starts in order then keep every count there.  Starts out
// of order may wrap the counts: an item found is one of its request all the same.
template <int THREADS>
__device__ __forceinline__ bool find_item(const AttnArgs &a, const Plan &plan, uint32_t rows, uint32_t want, Item &it,
                                          uint2 *meta) {
  __shared__ unsigned long long total;
  __shared__ Item found;
  if (threadIdx.x == 0) {
    total = 0;
    found.pieces = 0;
  }
  __syncthreads();
  uint64_t mine = 0;
  for (uint32_t b = threadIdx.x; b < a.batch; b += THREADS) {
    const Request r = request(a, b);
    mine += uint64_t((r.n * a.group + rows - 1) / rows) * r.tiles;
  }
  if (mine) atomicAdd(&total, (unsigned long long)mine);
  __syncthreads();
  const uint64_t each = (total + plan.items - 1) / plan.items;
  const uint32_t piece = each < plan.least ? plan.least : uint32_t(each);
  uint32_t done = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += THREADS) {
    const uint32_t b = b0 + threadIdx.x;
    Request r = {};
    uint32_t groups = 0, pieces = 0;
    if (b < a.batch) {
      r = request(a, b);
      groups = (r.n * a.group + rows - 1) / rows;
      pieces = (r.tiles + piece - 1) / piece;
      pieces = pieces ? pieces : 1;
    }
    uint32_t sum;
    const uint32_t first = done + block_scan<THREADS>(groups * pieces, sum);
    if (meta && b < a.batch) meta[b] = make_uint2(first, pieces);
    if (want >= first && want - first < groups * pieces) {
      const uint32_t i = want - first;
      found.b = b;
      found.group = i / pieces;
      found.piece = i - found.group * pieces;
      found.pieces = pieces;
      found.first = first;
      found.from = found.piece * piece;
      found.to = min(r.tiles, found.from + piece);
    }
    done += sum;
    if (done > want && !meta) break;
  }
  __syncthreads();
  it = found;
  return it.pieces != 0;
}

// ---------------------------------------------------------------- few rows --
// Scratch: where each request's items begin and how many pieces it has; then
// per item and key head 16 rows of sums, and their (m, l).
struct Parts {
  uint2 *meta;
  float2 *ml;
  float *sums;
  uint32_t items;   // of a key head
};
__host__ __device__ __forceinline__ Parts parts(uint8_t *scratch, uint32_t batch, uint32_t kv_heads, uint32_t items) {
  Parts p;
  p.meta = reinterpret_cast<uint2 *>(scratch);
  const uint64_t head = (uint64_t(batch) * 8 + 255) / 256 * 256;
  p.ml = reinterpret_cast<float2 *>(scratch + head);
  p.sums = reinterpret_cast<float *>(scratch + head + uint64_t(kv_heads) * items * 16 * 8);
  p.items = items;
  return p;
}

template <int DT>
__device__ __forceinline__ void store4(uint8_t *p, f32x4 v) {
  if constexpr (DT == BF16) {
    *reinterpret_cast<u32x2_any *>(p) = u32x2{f32_bf16x2(v[0], v[1]), f32_bf16x2(v[2], v[3])};
  } else {
    *reinterpret_cast<f32x4_any *>(p) = v;
  }
}

// Result of a row from its sums, weight and bound.
__device__ __forceinline__ float over(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.6931471805599453f;
}

// One wave's tiles: sums o (values 16 d + 4 j + i of row l % 16), bound m and this
// lane's share of the weights l.
template <int DT, int NB>
struct Rows16 {
  static constexpr int QP = DT == BF16 ? 1 : 3;   // pieces of a query
  static constexpr int WP = DT == BF16 ? 2 : 3;   // pieces of a weight
  static constexpr int kPitch = 64 * NB + 32;     // bytes of a row of values in LDS
  static constexpr int kLds = 32 * kPitch;        // of a wave
  bf16x8 q[NB][QP];
  f32x4 o[2 * NB];
  float m, l;
};

template <int DT, int NB>
__global__ __launch_bounds__(64 * kWaves, DT == BF16 && NB <= 4 ? 2 : 1) void k_attend(AttnArgs a, Plan plan, Parts out, FastDiv per_group, float c) {
  using R = Rows16<DT, NB>;
  constexpr int D = 32 * NB;
  constexpr int kPad = D + 4;   // floats of a row where the waves join
  constexpr int kShared = kWaves * (R::kLds > 64 * kPad ? R::kLds : 64 * kPad);
  __shared__ __attribute__((aligned(16))) uint8_t lds[kShared];
  __shared__ float2 ml_of[kWaves][16];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t n = lane & 15, j = lane >> 4;
  const uint32_t head = blockIdx.y;

  Item it;
  if (!find_item<64 * kWaves>(a, plan, 16, blockIdx.x, it, blockIdx.x + blockIdx.y == 0 ? out.meta : nullptr)) return;
  it.b = __builtin_amdgcn_readfirstlane(it.b);
  it.from = __builtin_amdgcn_readfirstlane(it.from);
  it.to = __builtin_amdgcn_readfirstlane(it.to);
  const Request rq = request(a, it.b);
  // this lane's row
  const uint32_t row = it.group * 16 + n;
  const bool live = row < rq.n * a.group;
  const uint32_t token = live ? per_group.div(row) : 0;
  const uint32_t qh = head * a.group + (live ? row - token * a.group : 0);
  // keys that it sees: first + 0 .. count - 1
  uint32_t first = 0, count = 0;
  if (live) {
    const int64_t at = int64_t(rq.len) - rq.n + token;   // its position
    const int64_t end = a.causal ? at + 1 : int64_t(rq.len);
    const int64_t begin = a.window && end > a.window ? end - a.window : 0;
    if (end > begin) {
      first = uint32_t(begin);
      count = uint32_t(end - begin);
    }
  }
  // tiles that some row of the wave sees, and those that all see whole
  uint32_t low = count ? first : ~0u, high = count ? first + count : 0;
  uint32_t low_all = live ? first : 0, high_all = live ? first + count : ~0u;
#pragma unroll
  for (int d = 1; d < 16; d *= 2) {
    low = min(low, uint32_t(__shfl_xor(int(low), d)));
    high = max(high, uint32_t(__shfl_xor(int(high), d)));
    low_all = max(low_all, uint32_t(__shfl_xor(int(low_all), d)));
    high_all = min(high_all, uint32_t(__shfl_xor(int(high_all), d)));
  }
  low = __builtin_amdgcn_readfirstlane(low);
  high = __builtin_amdgcn_readfirstlane(high);
  low_all = __builtin_amdgcn_readfirstlane(low_all);
  high_all = __builtin_amdgcn_readfirstlane(high_all);

  R r;
#pragma unroll
  for (int s = 0; s < NB; s++) {
    float x[8] = {};
    if (live) {
      const uint8_t *p = a.q + ((rq.start + token) * a.q_token + qh * a.q_head + 8 * (NB * j + s)) * esize(DT);
      if constexpr (DT == BF16) {
        const u32x4 w = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          x[2 * i] = bf16_lo(w[i]);
          x[2 * i + 1] = bf16_hi(w[i]);
        }
      } else {
        const f32x4 y = *reinterpret_cast<const f32x4_any *>(p), z = *reinterpret_cast<const f32x4_any *>(p + 16);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          x[i] = y[i];
          x[4 + i] = z[i];
        }
      }
    }
    pieces<R::QP>(x, r.q[s]);
  }
#pragma unroll
  for (int d = 0; d < 2 * NB; d++) r.o[d] = f32x4{0, 0, 0, 0};
  r.m = -__builtin_inff();
  r.l = 0.0f;

  uint8_t *mine = lds + wave * R::kLds;
  const uint8_t *kc = a.c.k + head * a.c.head_stride * 16, *vc = a.c.v + head * a.c.head_stride * 16;
  const uint8_t *ksc = a.c.ks + head * a.c.head_stride, *vsc = a.c.vs + head * a.c.head_stride;
  const int32_t *pages = a.table + it.b * a.table_stride;
  const uint32_t mask = (1u << a.c.shift) - 1;
  const uint32_t place = uint32_t(a.c.place_stride);
  const uint32_t last = a.c.n_pages;

  // Codes and scale bytes of a tile on their way.  Both are asked for as soon as
  // the registers of the tile before are free: a tile's keys before the values of
  // the one before are used, its values before its scores are computed.
  constexpr int kBytes = (NB % 4 == 0 ? NB / 4 : NB < 3 ? 1 : NB == 7 ? 3 : 2);   // blocks that a lane's quarter touches
  constexpr int kUnits = (NB + 1) / 2;                                            // blocks of 32 keys' values a lane
  uint32_t kw[4][NB], kb[4][kBytes];
  u32x4 vw[2][kUnits];
  uint32_t vb[2][kUnits];
  // The page of each 16 keys; a place outside any page is taken from page 0 and
  // counts as a NaN.
  struct Where {
    uint64_t base[4];
    uint32_t gone;
  };
  auto where = [&](uint32_t key0) {
    Where w;
    w.gone = 0;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const uint32_t key = key0 + 16 * g;
      uint32_t page = key < rq.len ? uint32_t(pages[key >> a.c.shift]) : 0;
      if (page >= last) {
        page = 0;
        w.gone |= 1u << g;
      }
      w.base[g] = page * a.c.page_stride + (key & mask) * uint64_t(place);
    }
    return w;
  };
  auto ask_keys = [&](const Where &w) {
#pragma unroll
    for (int g = 0; g < 4; g++) {
      const u32_any *p = reinterpret_cast<const u32_any *>(kc + w.base[g] * 16 + (n * place * 16 + 4 * NB * j));
#pragma unroll
      for (int st = 0; st < NB; st++) kw[g][st] = p[st];
      const uint8_t *q = ksc + w.base[g];
#pragma unroll
      for (int i = 0; i < kBytes; i++) kb[g][i] = q[n * place + min(NB * j / 4 + i, uint32_t(NB - 1))];
    }
  };
  auto ask_values = [&](const Where &w) {
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int u = 0; u < kUnits; u++) {
        const uint32_t unit = min(lane + 64 * u, uint32_t(32 * NB - 1));
        const uint32_t key = unit / NB, off = (key & 15) * place + unit % NB;
        const uint64_t base = key < 16 ? w.base[2 * h] : w.base[2 * h + 1];
        vw[h][u] = *reinterpret_cast<const u32x4 *>(vc + base * 16 + off * 16);
        vb[h][u] = *(vsc + base + off);
      }
  };

  // this wave's tiles that some row sees
  uint32_t t = it.from + wave, end = it.to;
  if (high > rq.lo) end = min(end, (high - rq.lo + kTile - 1) / kTile);
  else end = 0;
  if (low > rq.lo + t * kTile) {
    const uint32_t skip = ((low - rq.lo) / kTile - t + kWaves - 1) / kWaves;   // low >= rq.lo + t * kTile
    t += skip * kWaves;
  }
  Where w = {};
  if (t < end) {
    w = where(rq.lo + t * kTile);
    ask_keys(w);
    ask_values(w);
  }
  for (; t < end; t += kWaves) {
    const uint32_t key0 = rq.lo + t * kTile;
    // scores
    f32x4 s[4];
#pragma unroll
    for (int g = 0; g < 4; g++) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < NB; st++) {
        uint32_t byte = kb[g][0];
#pragma unroll
        for (int i = 1; i < kBytes; i++)
          if ((NB * j + st) / 4 - NB * j / 4 == i) byte = kb[g][i];
        const bf16x8 k = values8(kw[g][st], scale_of(w.gone >> g & 1 ? 255u : byte));
#pragma unroll
        for (int p = R::QP - 1; p >= 0; p--) acc = mfma(k, r.q[st][p], acc);
      }
      s[g] = acc;
    }
    const bool more = t + kWaves < end;
    if (more) {
      w = where(key0 + kWaves * kTile);
      ask_keys(w);
    }
    // keys that the row does not see
    if (key0 < low_all || key0 + kTile > high_all) {
#pragma unroll
      for (int g = 0; g < 4; g++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (key0 + 16 * g + 4 * j + i - first >= count) s[g][i] = -__builtin_inff();
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < 4; g++)
#pragma unroll
      for (int i = 0; i < 4; i++) top = fmaxf(top, s[g][i]);
    top = max_j(top) * c;
    if (__any(top > r.m)) {
      const float m = top > r.m ? top + kRise : r.m;
      const float f = m > r.m ? __builtin_amdgcn_exp2f(r.m - m) : 1.0f;
      r.l *= f;
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) r.o[d] *= f;
      r.m = m;
    }
    const float m = r.m == -__builtin_inff() ? 0.0f : r.m;
    // values of 32 keys to LDS
    const bool cut = key0 < low || key0 + kTile > high;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      bool nan = false;
#pragma unroll
      for (int u = 0; u < kUnits; u++) {
        const uint32_t unit = lane + 64 * u;
        if (NB % 2 == 0 || unit < 32 * NB) {
          const uint32_t key = unit / NB, blk = unit % NB;
          // no row sees a key outside [low, high)
          if (cut && key0 + 32 * h + key - low >= high - low) {
            vw[h][u] = u32x4{0, 0, 0, 0};
            vb[h][u] = 127;
          }
          nan |= vb[h][u] > 252;
          const float f = scale_of(vb[h][u]);
          uint8_t *p = mine + key * R::kPitch + blk * 64;
#pragma unroll
          for (int i = 0; i < 4; i++) *reinterpret_cast<bf16x8 *>(p + 16 * i) = values8(vw[h][u][i], f);
        }
      }
      const bool any_nan = __any(nan);
      lds_in_order();
      if (h == 1 && more) ask_values(w);
      bf16x8 wp[R::WP];
      {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * h + i / 4][i & 3], c, -m));
          r.l += x[i];
        }
        pieces<R::WP>(x, wp);
      }
      // and back, 4 keys of one value at a time
      const uint8_t *from = mine + (4 * j + n / 4) * R::kPitch + (n & 3) * 8;
      if (__builtin_expect(any_nan, 0)) {
        // A NaN would meet the weight 0 of rows that do not see its key.  It is left
        // out here, and rows that see one are found by a product of their own.
        union {
          uint16_t bits[8];
          bf16x8 all;
        } seen;
#pragma unroll
        for (int i = 0; i < 8; i++)
          seen.bits[i] = key0 + 32 * h + 16 * (i / 4) + 4 * j + (i & 3) - first < count ? 0x3F80 : 0;
#pragma unroll
        for (int d = 0; d < 2 * NB; d++) {
          Turned v = turned(from + 32 * d, 16 * R::kPitch), bad;
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const bool is = (v.bits[i] & 0x7FFF) > 0x7F80;
            bad.bits[i] = is ? 0x3F80 : 0;
            v.bits[i] = is ? 0 : v.bits[i];
          }
          const f32x4 hit = mfma(bad.all, seen.all, f32x4{0, 0, 0, 0});
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (hit[i] > 0.0f) r.o[d][i] = __builtin_nanf("");
#pragma unroll
          for (int p = R::WP - 1; p >= 0; p--) r.o[d] = mfma(v.all, wp[p], r.o[d]);
        }
      } else {
#pragma unroll
        for (int d = 0; d < 2 * NB; d++) {
          const Turned v = turned(from + 32 * d, 16 * R::kPitch);
#pragma unroll
          for (int p = R::WP - 1; p >= 0; p--) r.o[d] = mfma(v.all, wp[p], r.o[d]);
        }
      }
      lds_in_order();
    }
  }

  // the waves' sums join
  r.l = sum_j(r.l);
  if (rq.bad) r.l = __builtin_nanf("");
  if (j == 0) ml_of[wave][n] = make_float2(r.m, r.l);
  __syncthreads();
  float *joined = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int d = 0; d < 2 * NB; d++)
    *reinterpret_cast<f32x4 *>(joined + (wave * 16 + n) * kPad + 16 * d + 4 * j) = r.o[d];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 16 * D / 4; i += 64 * kWaves) {
    const uint32_t rr = i / (D / 4), col = (i % (D / 4)) * 4;
    const uint32_t rw = it.group * 16 + rr;
    if (rw >= rq.n * a.group) continue;
    float top = ml_of[0][rr].x;
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = fmaxf(top, ml_of[w][rr].x);
    float l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const float2 ml = ml_of[w][rr];
      const float f = ml.x == -__builtin_inff() && top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
      l += ml.y * f;
      o += *reinterpret_cast<const f32x4 *>(joined + (w * 16 + rr) * kPad + col) * f;
    }
    if (it.pieces == 1) {
      const uint32_t tk = per_group.div(rw), h = head * a.group + rw - tk * a.group;
      const uint64_t y = rq.start + tk;
      const float f = over(l);
      store4<DT>(a.out + (y * a.out_token + h * a.out_head + col) * esize(DT), o * f);
      if (a.lse && col == 0) a.lse[y * a.heads + h] = log_sum(top, l);
    } else {
      const uint64_t p = (uint64_t(head) * out.items + blockIdx.x) * 16 + rr;
      *reinterpret_cast<f32x4 *>(out.sums + p * D + col) = o;
      if (col == 0) out.ml[p] = make_float2(top, l);
    }
  }
}

// Joins the pieces of a row, in their order: a wave a row, four values a lane.
template <int DT, int NB>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, Parts in, FastDiv per_group) {
  constexpr int D = 32 * NB;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t head = blockIdx.y;
  // the rows' groups of 16, numbered with gaps: request b's from starts[b] group / 16 + b
  const uint32_t slot = blockIdx.x;
  uint32_t b;
  if (a.starts) {
    uint32_t lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1;
      const int32_t s = a.starts[mid];
      const uint32_t from = s < 0 ? 0 : min(uint32_t(s), a.tokens);
      if (from * a.group / 16 + mid <= slot)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
  } else {
    b = slot / ((a.group + 15) / 16);
  }
  const Request rq = request(a, b);
  const uint32_t group = a.starts ? slot - (rq.start * a.group / 16 + b) : slot % ((a.group + 15) / 16);
  const uint2 meta = in.meta[b];
  if (meta.y <= 1 || group >= (rq.n * a.group + 15) / 16) return;
  // starts out of order: items past the grid were not made
  if (meta.x >= in.items || uint64_t(group + 1) * meta.y > in.items - meta.x) return;
  for (uint32_t rr = threadIdx.x >> 6; rr < 16; rr += 4) {
    const uint32_t row = group * 16 + rr;
    if (row >= rq.n * a.group) return;
    const uint64_t p0 = uint64_t(head) * in.items + meta.x + group * meta.y;
    float top = -__builtin_inff();
    for (uint32_t i = lane; i < meta.y; i += 64) top = fmaxf(top, in.ml[(p0 + i) * 16 + rr].x);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    float l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (uint32_t i = 0; i < meta.y; i++) {
      const uint64_t p = (p0 + i) * 16 + rr;
      const float2 ml = in.ml[p];
      const float f = ml.x == -__builtin_inff() && top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
      l += ml.y * f;
      if (lane < D / 4) o += *reinterpret_cast<const f32x4 *>(in.sums + p * D + 4 * lane) * f;
    }
    const uint32_t tk = per_group.div(row), h = head * a.group + row - tk * a.group;
    const uint64_t y = rq.start + tk;
    if (lane < D / 4) store4<DT>(a.out + (y * a.out_token + h * a.out_head + 4 * lane) * esize(DT), o * over(l));
    if (a.lse && lane == 0) a.lse[y * a.heads + h] = log_sum(top, l);
  }
}

// ------------------------------------------------------------------ launch --
struct Sizes {
  Plan plan;
  uint32_t groups, items;  // row groups of 16 and items of a key head, at most
  bool split;              // some request may be cut into pieces
};
Sizes sizes(const AttnArgs &a) {
  Sizes s;
  s.groups = a.starts ? uint32_t(uint64_t(a.tokens) * a.group / 16 + a.batch) : a.batch * ((a.group + 15) / 16);
  const uint32_t want = 1024 / a.c.heads;
  s.plan.items = want ? want : 1;
  s.plan.least = 4;
  const uint64_t longest = (uint64_t(a.width) << a.c.shift) / kTile + 1;
  s.split = longest > s.plan.least;
  s.items = s.groups + (s.split ? s.plan.items : 0);
  return s;
}

template <int DT, int NB>
hipError_t attend(const AttnArgs &a, hipStream_t s) {
  const Sizes z = sizes(a);
  const Parts p = parts(a.scratch, a.batch, a.c.heads, z.items);
  const float c = float(double(a.scale) * 1.4426950408889634);
  const FastDiv per_group(a.group);
  Parts q = p;
  if (!z.split) q.meta = nullptr;
  k_attend<DT, NB><<<dim3(z.items, a.c.heads), 64 * kWaves, 0, s>>>(a, z.plan, q, per_group, c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !z.split) return e;
  k_join<DT, NB><<<dim3(z.groups, a.c.heads), 256, 0, s>>>(a, p, per_group);
  return hipGetLastError();
}

template <int DT>
hipError_t by_blocks(const AttnArgs &a, hipStream_t s) {
  switch (a.c.blocks) {
    case 1: return attend<DT, 1>(a, s);
    case 2: return attend<DT, 2>(a, s);
    case 3: return attend<DT, 3>(a, s);
    case 4: return attend<DT, 4>(a, s);
    case 5: return attend<DT, 5>(a, s);
    case 6: return attend<DT, 6>(a, s);
    case 7: return attend<DT, 7>(a, s);
    default: return attend<DT, 8>(a, s);
  }
}

}  // namespace

uint64_t attention_scratch(int dtype, const AttnArgs &a) {
  const Sizes z = sizes(a);
  if (!z.split) return 0;
  const Parts p = parts(nullptr, a.batch, a.c.heads, z.items);
  return reinterpret_cast<uint64_t>(p.sums) + uint64_t(a.c.heads) * z.items * 16 * a.c.blocks * 32 * 4;
}

hipError_t launch_attention(int dtype, const AttnArgs &a, hipStream_t s) {
  return dtype == BF16 ? by_blocks<BF16>(a, s) : by_blocks<FP32>(a, s);
}

}  // namespace zn
