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
#include <algorithm>

#include "zn_kv.h"

namespace zn {
namespace {

constexpr int kTile = 64;       // keys a wave takes at a time
constexpr int kWaves = 4;       // of a workgroup
constexpr uint32_t kLeast = 2;  // tiles that a wave takes at least
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

// Values that are the same in all lanes, known to be so.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return uint64_t(uniform(uint32_t(v >> 32))) << 32 | uniform(uint32_t(v));
}
__device__ __forceinline__ Request uniform(const Request &r) {
  return Request{uniform(r.start), uniform(r.n), uniform(r.len), uniform(r.lo), uniform(r.tiles), uniform(uint32_t(r.bad)) != 0};
}

// How the work is shared out.  Rows of a request go in groups of `rows`, and the
// tiles of all groups of all requests, one after the other (a group without any
// counts as one), are cut into equal shares, one for each of a head's `takers`,
// whatever the requests' lengths are.  A group that lies in several shares is left
// in pieces and joined by a second launch: its first piece in slot 2 f + 1 of its
// first taker f, the others in slots 2 i, so that no taker has two of a kind.
// Every taker finds its place by itself, with a sum over the requests.
// Groups are counted in 32 bits: the host keeps tokens * group + batch below 2^30.
struct Plan {
  uint32_t takers;     // of a head
  uint32_t least;      // tiles of a share at least
};
struct Shares {
  uint64_t total, each;
};
__device__ __forceinline__ uint32_t groups_of(const AttnArgs &a, const Request &r, uint32_t rows) {
  return (r.n * a.group + rows - 1) / rows;
}
__device__ __forceinline__ uint64_t tiles_of(const AttnArgs &a, const Request &r, uint32_t rows) {
  return uint64_t(groups_of(a, r, rows)) * max(r.tiles, 1u);
}

// The request of tile `taker * each` and the tiles before it, by one wave: a lane
// sums batch / 64 requests in a row.
__device__ __forceinline__ bool find_start(const AttnArgs &a, const Plan &plan, uint32_t rows, uint32_t taker,
                                           Shares &sh, uint32_t &b, uint64_t &before) {
  const uint32_t lane = threadIdx.x & 63, per = (a.batch + 63) / 64;
  uint64_t mine = 0;
  for (uint32_t i = 0; i < per; i++)
    if (lane * per + i < a.batch) mine += tiles_of(a, request(a, lane * per + i), rows);
  uint64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t p = __shfl_up(upto, d);
    if (lane >= uint32_t(d)) upto += p;
  }
  sh.total = __shfl(upto, 63);
  sh.each = (sh.total + plan.takers - 1) / plan.takers;
  if (sh.each < plan.least) sh.each = plan.least;
  const uint64_t want = taker * sh.each;
  if (want >= sh.total) return false;
  const uint32_t owner = __popcll(__ballot(upto <= want));
  before = __shfl(upto - mine, int(owner));
  b = owner * per;
  for (;; b++) {
    const uint64_t t = tiles_of(a, request(a, b), rows);
    if (want < before + t) return true;
    before += t;
  }
}

// Scratch: the shares' size; the tiles before each request's; then per head and
// slot `rows` rows of sums, and their (m, l).
struct Parts {
  uint64_t *each, *before;
  float2 *ml;
  float *sums;
  uint32_t slots;   // of a key head
};
__host__ __device__ __forceinline__ Parts parts(uint8_t *scratch, uint32_t batch, uint32_t kv_heads, uint32_t slots,
                                                uint32_t rows) {
  Parts p;
  p.each = reinterpret_cast<uint64_t *>(scratch);
  p.before = p.each + 1;
  const uint64_t head = (uint64_t(batch) * 8 + 8 + 255) / 256 * 256;
  p.ml = reinterpret_cast<float2 *>(scratch + head);
  p.sums = reinterpret_cast<float *>(scratch + head + uint64_t(kv_heads) * slots * rows * 8);
  p.slots = slots;
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
constexpr int kResident = DT == BF16 && NB <= 2 ? 3 : DT == BF16 && NB <= 4 ? 2 : 1;   // waves a SIMD

template <int DT, int NB>
__global__ __launch_bounds__(64 * kWaves, (kResident<DT, NB>)) void k_attend(AttnArgs a, Plan plan, Parts out,
                                                                        FastDiv per_group, float c) {
  using R = Rows16<DT, NB>;
  constexpr int D = 32 * NB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * R::kLds];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t n = lane & 15, j = lane >> 4;
  const uint32_t head = blockIdx.y, taker = blockIdx.x * kWaves + wave;

  Shares share;
  uint32_t b;
  uint64_t before;
  if (taker >= plan.takers || !find_start(a, plan, 16, taker, share, b, before)) return;
  share.each = uniform(share.each);
  b = uniform(b);
  before = uniform(before);
  uint64_t at_tile = taker * share.each;
  const uint64_t end_tile = min(at_tile + share.each, uniform(share.total));
  if (taker == 0 && head == 0 && out.each && lane == 0) *out.each = share.each;
  // group after group, request after request
  while (at_tile < end_tile) {
  const Request rq = uniform(request(a, b));
  const uint32_t whole = max(rq.tiles, 1u);
  const uint32_t groups = groups_of(a, rq, 16);
  const uint32_t grp = groups > 1 ? uint32_t((at_tile - before) / whole) : 0;
  const uint32_t from = uint32_t(at_tile - before - uint64_t(grp) * whole);
  const uint32_t to = uint32_t(min(uint64_t(whole), from + (end_tile - at_tile)));
  if (out.before && at_tile == before && head == 0 && lane == 0) out.before[b] = before;
  // this lane's row
  const uint32_t row = grp * 16 + n;
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
  low = uniform(low);
  high = uniform(high);
  low_all = uniform(low_all);
  high_all = uniform(high_all);

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
  const int32_t *pages = a.table + b * a.table_stride;
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
  // The page of each 16 keys of a tile, lane g % 4 that of 16 g; asked for a tile
  // ahead of the codes.  Behind the last key it is the last one's.
  auto ask_pages = [&](uint32_t key0) {
    return uint32_t(pages[min(key0 + 16 * (lane & 3), rq.len - 1) >> a.c.shift]);
  };
  // A place outside any page is taken from page 0 and counts as a NaN.
  struct Where {
    uint64_t base[4];
    uint32_t gone;
  };
  auto where = [&](uint32_t key0, uint32_t asked) {
    Where w;
    w.gone = 0;
#pragma unroll
    for (int g = 0; g < 4; g++) {
      uint32_t page = __builtin_amdgcn_readlane(asked, g);
      if (page >= last) {
        page = 0;
        w.gone |= 1u << g;
      }
      w.base[g] = page * a.c.page_stride + ((key0 + 16 * g) & mask) * uint64_t(place);
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

  // the tiles that some row sees
  uint32_t t = from, end = min(to, rq.tiles);
  end = high > rq.lo ? min(end, (high - rq.lo + kTile - 1) / kTile) : 0;
  if (low > rq.lo) t = max(t, (low - rq.lo) / kTile);
  Where w = {};
  uint32_t asked = 0;
  if (t < end) {
    asked = ask_pages(rq.lo + t * kTile);
    w = where(rq.lo + t * kTile, asked);
    asked = ask_pages(rq.lo + (t + 1) * kTile);
    ask_keys(w);
    ask_values(w);
  }
  for (; t < end; t++) {
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
    const bool more = t + 1 < end;
    if (more) {
      w = where(key0 + kTile, asked);
      asked = ask_pages(key0 + 2 * kTile);
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

  r.l = sum_j(r.l);
  if (rq.bad) r.l = __builtin_nanf("");
  if (live) {
    if (to - from == whole) {
      const uint64_t y = rq.start + token;
      const float f = over(r.l);
      uint8_t *p = a.out + (y * a.out_token + qh * a.out_head + 4 * j) * esize(DT);
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) store4<DT>(p + 16 * d * esize(DT), r.o[d] * f);
      if (a.lse && j == 0) a.lse[y * a.heads + qh] = log_sum(r.m, r.l);
    } else {
      const uint64_t p = (uint64_t(head) * out.slots + 2 * taker + (from == 0)) * 16 + n;
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) *reinterpret_cast<f32x4 *>(out.sums + p * D + 16 * d + 4 * j) = r.o[d];
      if (j == 0) out.ml[p] = make_float2(r.m, r.l);
    }
  }
  at_tile += to - from;
  if (at_tile == before + uint64_t(groups) * whole) {
    before = at_tile;
    do b++;
    while (at_tile < end_tile && uniform(request(a, b)).n == 0);
  }
  }
}

// Joins the pieces of a row: a workgroup a row, four values a lane; its lanes make
// 256 / (D / 4) teams that take every so manieth piece in order, and their sums are
// added in order.
template <int DT, int NB>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, Parts in, FastDiv per_group) {
  constexpr int D = 32 * NB, kLanes = D / 4, kTeams = 256 / kLanes;
  __shared__ float tops[4];
  __shared__ __attribute__((aligned(16))) float sums[kTeams][D + 4];
  __shared__ float weights[kTeams];
  const uint32_t head = blockIdx.y;
  // the rows' groups of 16, numbered with gaps: request b's from starts[b] group / 16 + b
  const uint32_t rows = a.starts ? 16 : min(16u, a.group);   // of a group, at most
  const uint32_t slot = blockIdx.x / rows, rr = blockIdx.x - slot * rows;
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
  const uint32_t row = group * 16 + rr;
  if (group >= groups_of(a, rq, 16) || row >= rq.n * a.group) return;
  const uint64_t whole = max(rq.tiles, 1u), at = in.before[b] + group * whole, each = *in.each;
  const uint64_t f = at / each, pieces = (at + whole - 1) / each - f + 1;
  if (pieces <= 1) return;
  if (pieces > in.slots || 2 * f > in.slots - pieces) return;   // starts out of order: not all tiles had a taker
  const uint32_t count = uint32_t(pieces);
  const uint64_t p0 = uint64_t(head) * in.slots + 2 * f;
  // a row's piece i
  auto piece = [&](uint32_t i) { return (p0 + (i ? 2 * i : 1)) * 16 + rr; };

  float top = -__builtin_inff();
  for (uint32_t i = threadIdx.x; i < count; i += 256) top = fmaxf(top, in.ml[piece(i)].x);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));

  const uint32_t team = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 4;
  if (team < kTeams) {
    float l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t i = team; i < count; i += kTeams) {
      const uint64_t p = piece(i);
      const float2 ml = in.ml[p];
      const float f = ml.x == -__builtin_inff() && top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
      l += ml.y * f;
      o += *reinterpret_cast<const f32x4 *>(in.sums + p * D + col) * f;
    }
    *reinterpret_cast<f32x4 *>(&sums[team][col]) = o;
    if (col == 0) weights[team] = l;
  }
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  float l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kTeams; i++) {
    l += weights[i];
    o += *reinterpret_cast<const f32x4 *>(&sums[i][col]);
  }
  const uint32_t tk = per_group.div(row), h = head * a.group + row - tk * a.group;
  const uint64_t y = rq.start + tk;
  store4<DT>(a.out + (y * a.out_token + h * a.out_head + col) * esize(DT), o * over(l));
  if (a.lse && col == 0) a.lse[y * a.heads + h] = log_sum(top, l);
}

// ------------------------------------------------------------------ launch --
// The takers fill the chip once, so that they all run at the same time.
template <int DT, int NB>
Plan few_plan(const AttnArgs &a) {
  constexpr uint32_t kSimds = 1024;
  const uint32_t n = kSimds * kResident<DT, NB> / a.c.heads;
  return Plan{n ? n : 1, kLeast};
}
struct Sizes {
  uint32_t groups;         // row groups of a key head, at most
  bool split;              // some request may be cut into pieces
};
Sizes sizes(const AttnArgs &a, uint32_t rows, uint32_t least) {
  Sizes s;
  s.groups = a.starts ? uint32_t(uint64_t(a.tokens) * a.group / rows + a.batch) : a.batch * ((a.group + rows - 1) / rows);
  // a share never ends inside a request that is all there is
  s.split = (uint64_t(a.width) << a.c.shift) > uint64_t(least) * kTile || s.groups > 1;
  return s;
}

template <int DT, int NB>
struct Few {
  static uint64_t scratch(const AttnArgs &a) {
    const Plan plan = few_plan<DT, NB>(a);
    if (!sizes(a, 16, plan.least).split) return 0;
    const Parts p = parts(nullptr, a.batch, a.c.heads, 2 * plan.takers, 16);
    return reinterpret_cast<uint64_t>(p.sums) + uint64_t(a.c.heads) * 2 * plan.takers * 16 * NB * 32 * 4;
  }
  static hipError_t run(const AttnArgs &a, hipStream_t s) {
    const Plan plan = few_plan<DT, NB>(a);
    const Sizes z = sizes(a, 16, plan.least);
    Parts p = {};
    if (z.split) p = parts(a.scratch, a.batch, a.c.heads, 2 * plan.takers, 16);
    const FastDiv per_group(a.group);
    // no more takers than the table's width gives tiles to
    const uint64_t tiles = uint64_t(z.groups) * (((uint64_t(a.width) << a.c.shift) + kTile - 1) / kTile + 1);
    const uint64_t busy = std::min<uint64_t>(plan.takers, (tiles + plan.least - 1) / plan.least);
    k_attend<DT, NB><<<dim3(uint32_t((busy + kWaves - 1) / kWaves), a.c.heads), 64 * kWaves, 0, s>>>(
        a, plan, p, per_group, float(double(a.scale) * 1.4426950408889634));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !z.split) return e;
    const uint32_t rows = a.starts || a.group > 16 ? 16 : a.group;
    k_join<DT, NB><<<dim3(z.groups * rows, a.c.heads), 256, 0, s>>>(a, p, per_group);
    return hipGetLastError();
  }
};

// f of the kernels for the call's type and head size.
template <int DT, class F>
auto by_blocks(uint32_t blocks, F f) {
  switch (blocks) {
    case 1: return f(Few<DT, 1>());
    case 2: return f(Few<DT, 2>());
    case 3: return f(Few<DT, 3>());
    case 4: return f(Few<DT, 4>());
    case 5: return f(Few<DT, 5>());
    case 6: return f(Few<DT, 6>());
    case 7: return f(Few<DT, 7>());
    default: return f(Few<DT, 8>());
  }
}

}  // namespace

uint64_t attention_scratch(int dtype, const AttnArgs &a) {
  auto f = [&](auto k) { return k.scratch(a); };
  return dtype == BF16 ? by_blocks<BF16>(a.c.blocks, f) : by_blocks<FP32>(a.c.blocks, f);
}

hipError_t launch_attention(int dtype, const AttnArgs &a, hipStream_t s) {
  auto f = [&](auto k) { return k.run(a, s); };
  return dtype == BF16 ? by_blocks<BF16>(a.c.blocks, f) : by_blocks<FP32>(a.c.blocks, f);
}

}  // namespace zn
