// zn_attn.hip -- attention over the key-value cache in 4 bits.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c (q.k_j - m) - 8),  c = scale log2(e),
//
// in one pass over the keys: m is one of the scores so far.  When one passes it by
// more than 2^8 in weight, m becomes that one and the sums so far are multiplied by
// 2^(c (old - new)); with the 8 this is seldom, and weights stay under 1.  Scores
// are subtracted before they are scaled: the largest weights are exact however
// large the scores.
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
//   Queries and weights have more bits: queries in FP32 go as three BF16 pieces,
// weights as two beside BF16 queries (16 bits; one would leave 8) and three beside
// FP32.
//
// What bounds it is memory: 64 requests of up to 8192 keys (8 key heads of 128, 325
// MB of codes and scales) 69 us and 6 for the join, 4.7 TB/s where a large copy has
// 5.2; two of 32768 keys 20 + 6 us.  Below that it is the chain of dependent loads
// (lengths, pages, codes) and of launches: one request of 1000 keys 10 us.
#include <algorithm>

#include "zn_attn.h"

namespace zn {
namespace {

constexpr int kWaves = 4;       // of a workgroup

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

// How the work is shared out.  Rows of a request go in groups of `rows`, and the
// tiles of all groups of all requests, one after the other (a group without any
// counts as one), are cut into equal shares, one for each of a head's `takers`,
// whatever the requests' lengths are.  A group that lies in several shares is left
// in pieces and joined by a second launch: its first piece in slot 2 f + 1 of its
// first taker f, the others in slots 2 i, so that no taker has two of a kind.
// Every taker finds its place by itself, with a sum over the requests.  With a fixed
// number of pieces a request the batch of 64 took 102 to 115 us, whatever the number.
// Groups are counted in 32 bits: the host keeps tokens * group + batch below 2^30.
struct Plan {
  uint32_t takers;     // of a head
};
struct Shares {
  uint64_t total, each;
};
__device__ __forceinline__ uint64_t tiles_of(const AttnArgs &a, const Request &r, uint32_t rows) {
  return uint64_t(groups_of(a, r, rows)) * max(r.tiles, 1u);
}

// The request of tile `taker * each` and the tiles before it, by one wave: a lane
// sums batch / 64 requests in a row.
__device__ __forceinline__ bool find_start(const AttnArgs &a, const Plan &plan, uint32_t rows, uint32_t taker,
                                           Shares &sh, uint32_t &b, uint64_t &before, uint64_t *tell_each, uint64_t *tell_before) {
  const uint32_t lane = threadIdx.x & 63, per = (a.batch + 63) / 64;
  uint64_t mine = 0;
  for (uint32_t i = 0; i < per; i++)
    if (lane * per + i < a.batch) mine += tiles_of(a, request(a, lane * per + i), rows);
  const uint64_t upto = scan(mine);
  sh.total = of_lane(upto, 63);
  sh.each = (sh.total + plan.takers - 1) / plan.takers;
  if (tell_each) {
    uint64_t at = upto - mine;
    for (uint32_t i = 0; i < per; i++)
      if (lane * per + i < a.batch) {
        tell_before[lane * per + i] = at;
        at += tiles_of(a, request(a, lane * per + i), rows);
      }
    if (lane == 0) *tell_each = sh.each;
  }
  const uint64_t want = taker * sh.each;
  if (want >= sh.total) return false;
  const uint32_t owner = uniform(uint32_t(__popcll(__ballot(upto <= want))));
  before = of_lane(upto - mine, owner);
  b = owner * per;
  for (;; b++) {
    const uint64_t t = tiles_of(a, request(a, b), rows);
    if (want < before + t) return true;
    before += t;
  }
}

// What a wave has of a group of rows: sums o (values 16 d + 4 j + i of row l % 16),
// bound m and this lane's share of the weights l.
template <int DT, int NB>
struct Rows16 {
  static constexpr int QP = DT == BF16 ? 1 : 3;   // pieces of a query
  static constexpr int WP = DT == BF16 ? 2 : 3;   // pieces of a weight
  static constexpr int kPitch = 64 * NB + 32;     // bytes of a row of values in LDS
  static constexpr int kLds = 32 * kPitch;        // of a wave
  bf16x8 q[NB][QP];
  f32x4 o[2 * NB];
  float m, l;
  uint32_t marks;                                 // blocks of values that have a NaN for this row
  bool live;
  uint32_t token, qh;
  Span sees;
  uint32_t low, high, low_all, high_all;          // keys that some row sees, and that all see
};

template <int DT, int NB>
__device__ __forceinline__ void set_rows(const AttnArgs &a, const Request &rq, uint32_t group, uint32_t head,
                                         const FastDiv &per_group, Rows16<DT, NB> &r) {
  const uint32_t row = group * 16 + (threadIdx.x & 15);
  r.live = row < rq.n * a.group;
  r.token = r.live ? per_group.div(row) : 0;
  r.qh = head * a.group + (r.live ? row - r.token * a.group : 0);
  r.sees = span(a, rq, r.token, r.live);
  const uint32_t first = r.sees.first, count = r.sees.count;
  uint32_t low = count ? first : ~0u, high = count ? first + count : 0;
  uint32_t low_all = r.live ? first : 0, high_all = r.live ? first + count : ~0u;
#pragma unroll
  for (int d = 1; d < 16; d *= 2) {
    low = min(low, uint32_t(__shfl_xor(int(low), d)));
    high = max(high, uint32_t(__shfl_xor(int(high), d)));
    low_all = max(low_all, uint32_t(__shfl_xor(int(low_all), d)));
    high_all = min(high_all, uint32_t(__shfl_xor(int(high_all), d)));
  }
  r.low = uniform(low);
  r.high = uniform(high);
  r.low_all = uniform(low_all);
  r.high_all = uniform(high_all);
#pragma unroll
  for (int d = 0; d < 2 * NB; d++) r.o[d] = f32x4{0, 0, 0, 0};
  r.m = -__builtin_inff();
  r.l = 0.0f;
  r.marks = 0;
}

// One wave's tiles: t, t + STEP .. of those from `from` to `to` that some row sees.
template <int DT, int NB, int STEP>
__device__ __forceinline__ void take_tiles(const AttnArgs &a, const Request &rq, const int32_t *pages, uint32_t head,
                                           uint32_t from, uint32_t to, uint32_t offset, float c, uint8_t *mine,
                                           Rows16<DT, NB> &r) {
  using R = Rows16<DT, NB>;
  const uint32_t lane = threadIdx.x & 63, n = lane & 15, j = lane >> 4;
  const uint32_t first = r.sees.first, count = r.sees.count;
  const uint8_t *kc = a.c.k + head * a.c.head_stride * 16, *vc = a.c.v + head * a.c.head_stride * 16;
  const uint8_t *ksc = a.c.ks + head * a.c.head_stride, *vsc = a.c.vs + head * a.c.head_stride;
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

  uint32_t t = from, end = min(to, rq.tiles);
  end = r.high > rq.lo ? min(end, (r.high - rq.lo + kTile - 1) / kTile) : 0;
  if (r.low > rq.lo) t = max(t, (r.low - rq.lo) / kTile);
  t += offset;
  Where w = {};
  uint32_t asked = 0;
  if (t < end) asked = ask_pages(rq.lo + t * kTile);
#pragma unroll
  for (int s = 0; s < NB; s++)
    take_query8<DT>(a.q + ((rq.start + r.token) * a.q_token + r.qh * a.q_head + 8 * (NB * j + s)) * esize(DT), r.live, r.q[s]);
  if (t < end) {
    w = where(rq.lo + t * kTile, asked);
    asked = ask_pages(rq.lo + (t + STEP) * kTile);
    ask_keys(w);
    ask_values(w);
  }
  for (; t < end; t += STEP) {
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
    const bool more = t + STEP < end;
    const uint64_t here[4] = {w.base[0], w.base[1], w.base[2], w.base[3]};
    if (more) {
      w = where(key0 + STEP * kTile, asked);
      asked = ask_pages(key0 + 2 * STEP * kTile);
      ask_keys(w);
    }
    // keys that the row does not see
    if (key0 < r.low_all || key0 + kTile > r.high_all) {
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
    top = max_j(top);
    if (__any((top - r.m) * c > kRise)) {
      const float m = fmaxf(top, r.m);
      const float f = m > r.m ? __builtin_amdgcn_exp2f((r.m - m) * c) : 1.0f;
      r.l *= f;
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) r.o[d] *= f;
      r.m = m;
    }
    const float m = r.m == -__builtin_inff() ? 0.0f : r.m;
    // values of 32 keys to LDS
    const bool cut = key0 < r.low || key0 + kTile > r.high;
    bool nan = false;
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int u = 0; u < kUnits; u++) {
        const uint32_t unit = lane + 64 * u;
        if (NB % 2 == 0 || unit < 32 * NB) {
          const uint32_t key = unit / NB, blk = unit % NB;
          // no row sees a key outside [low, high)
          if (cut && key0 + 32 * h + key - r.low >= r.high - r.low) {
            vw[h][u] = u32x4{0, 0, 0, 0};
            vb[h][u] = 127;
          }
          if (vb[h][u] > 252) {
            nan = true;
            vw[h][u] = u32x4{0, 0, 0, 0};
            vb[h][u] = 127;
          }
          const float f = __uint_as_float(vb[h][u] << 23);
          uint8_t *p = mine + key * R::kPitch + blk * 64;
#pragma unroll
          for (int i = 0; i < 4; i++) *reinterpret_cast<bf16x8 *>(p + 16 * i) = values8(vw[h][u][i], f);
        }
      }
      lds_in_order();
      if (h == 1 && more) ask_values(w);
      bf16x8 wp[R::WP];
      {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * h + i / 4][i & 3] - m, c, -kRise));
          r.l += x[i];
        }
        pieces<R::WP>(x, wp);
      }
      // and back, 4 keys of one value at a time
      const uint8_t *parts = mine + (4 * j + n / 4) * R::kPitch + (n & 3) * 8;
#pragma unroll
      for (int d = 0; d < 2 * NB; d++) {
        const bf16x8 v = turned(parts + 32 * d, 16 * R::kPitch);
#pragma unroll
        for (int p = R::WP - 1; p >= 0; p--) r.o[d] = mfma(v, wp[p], r.o[d]);
      }
      lds_in_order();
    }
    if (__builtin_expect(__any(nan), 0)) {
      const uint64_t at = (lane < 32 ? lane < 16 ? here[0] : here[1] : lane < 48 ? here[2] : here[3]) + (lane & 15) * place;
      r.marks |= marked<NB>(vsc + at, key0, first, count);
    }
  }
  r.l = sum_j(r.l);
  if (rq.bad) r.l = __builtin_nanf("");
#pragma unroll
  for (int d = 0; d < 2 * NB; d++)
    if (r.marks >> d / 2 & 1) r.o[d] = f32x4{} + __builtin_nanf("");
}

template <int DT, int NB>
constexpr int kResident = DT == BF16 && NB <= 2 ? 3 : DT == BF16 && NB <= 4 ? 2 : 1;   // waves a SIMD

template <int DT, int NB>
__global__ __launch_bounds__(64 * kWaves, (kResident<DT, NB>)) void k_attend(AttnArgs a, Plan plan, Parts out,
                                                                        FastDiv per_group, float c) {
  using R = Rows16<DT, NB>;
  constexpr int D = 32 * NB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * R::kLds];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t n = lane & 15, j = lane >> 4;
  const uint32_t head = blockIdx.y, taker = blockIdx.x * kWaves + wave;

  Shares sh;
  uint32_t b;
  uint64_t before;
  if (taker >= plan.takers || !find_start(a, plan, 16, taker, sh, b, before,
                                            taker + head ? nullptr : out.each, out.before))
    return;
  sh.each = uniform(sh.each);
  b = uniform(b);
  before = uniform(before);
  uint64_t at_tile = taker * sh.each;
  const uint64_t end_tile = min(at_tile + sh.each, uniform(sh.total));
  // group after group, request after request
  while (at_tile < end_tile) {
    const Request rq = uniform(request(a, b));
    const uint32_t whole = max(rq.tiles, 1u);
    const uint32_t groups = groups_of(a, rq, 16);
    const uint32_t group = groups > 1 ? uint32_t((at_tile - before) / whole) : 0;
    const uint32_t from = uint32_t(at_tile - before - uint64_t(group) * whole);
    const uint32_t to = uint32_t(min(uint64_t(whole), from + (end_tile - at_tile)));
    R r;
    set_rows(a, rq, group, head, per_group, r);
    take_tiles<DT, NB, 1>(a, rq, a.table + b * a.table_stride, head, from, to, 0, c, lds + wave * R::kLds, r);
    if (r.live) {
      if (to - from == whole) {
#pragma unroll
        for (int d = 0; d < 2 * NB; d++) put_row<DT>(a, rq, r.token, r.qh, 16 * d + 4 * j, r.o[d], r.m, r.l);
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

// Group x of all requests' groups of 16 rows, numbered with gaps where requests have
// starts: request b's from starts[b] group / 16 + b on.  By one wave, 64 places a step.
__device__ __forceinline__ void group_at(const AttnArgs &a, uint32_t x, uint32_t &b, uint32_t &group) {
  if (!a.starts) {
    const uint32_t groups = (a.group + 15) / 16;
    b = x / groups;
    group = x - b * groups;
    return;
  }
  auto from = [&](uint32_t i) {
    const int32_t s = a.starts[i];
    return (s < 0 ? 0 : min(uint32_t(s), a.tokens)) * a.group / 16 + i;
  };
  const uint32_t lane = threadIdx.x & 63;
  b = 0;
  for (uint32_t n = a.batch; n > 1;) {
    const uint32_t step = (n + 63) / 64, i = lane * step;
    const bool upto = from(b + min(i, n - 1)) <= x;
    const uint32_t last = max(__popcll(__ballot(i < n && upto)), 1) - 1;
    b += last * step;
    n = min(step, n - last * step);
  }
  b = uniform(b);
  group = uniform(x - from(b));   // past the last one's where x is before all
}

// Short caches: a workgroup for each group of rows, whose waves take turns at its
// tiles and join their sums in LDS; no second launch.
template <int DT, int NB>
constexpr int kShortWaves = kResident<DT, NB> >= 2 ? 8 : 4;

template <int DT, int NB, int W>
__global__ __launch_bounds__(64 * W, (W == 2 ? kResident<DT, NB> : 1)) void k_attend_short(AttnArgs a, FastDiv per_group, float c) {
  using R = Rows16<DT, NB>;
  constexpr int D = 32 * NB, kPad = D + 4;
  constexpr int kShared = R::kLds > 16 * kPad * 4 ? R::kLds : 16 * kPad * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[W * kShared];
  __shared__ float2 ml_of[W][16];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t n = lane & 15, j = lane >> 4;
  const uint32_t head = blockIdx.y;
  uint32_t b, group;
  group_at(a, blockIdx.x, b, group);
  const Request rq = uniform(request(a, b));
  if (group >= groups_of(a, rq, 16)) return;
  R r;
  set_rows(a, rq, group, head, per_group, r);
  take_tiles<DT, NB, W>(a, rq, a.table + b * a.table_stride, head, 0, rq.tiles, wave, c, lds + wave * R::kLds, r);
  if (j == 0) ml_of[wave][n] = make_float2(r.m, r.l);
  __syncthreads();   // the sums lie where the values did
  float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int d = 0; d < 2 * NB; d++)
    *reinterpret_cast<f32x4 *>(sums + (wave * 16 + n) * kPad + 16 * d + 4 * j) = r.o[d];
  __syncthreads();
  const uint32_t rows = min(16u, rq.n * a.group - group * 16);
  for (uint32_t i = threadIdx.x; i < rows * (D / 4); i += 64 * W) {
    const uint32_t rr = i / (D / 4), col = i % (D / 4) * 4;
    float top = ml_of[0][rr].x;
#pragma unroll
    for (int w = 1; w < W; w++) top = fmaxf(top, ml_of[w][rr].x);
    float l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; w++) {
      const float2 ml = ml_of[w][rr];
      const float f = share(ml.x, top, c);
      l += ml.y * f;
      o += *reinterpret_cast<const f32x4 *>(sums + (w * 16 + rr) * kPad + col) * f;
    }
    const uint32_t row = group * 16 + rr, token = per_group.div(row);
    put_row<DT>(a, rq, token, head * a.group + row - token * a.group, col, o, top, l);
  }
}

// Joins the pieces of a group's rows, `most` rows a workgroup: with few pieces a row
// for each team (64 requests of 512 keys, 24 rows each, the attention with it: 63 us
// by a workgroup a row, so 30).
template <int DT, int NB>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, Parts in, FastDiv per_group, float c, bool by_edges, uint32_t most,
                                              uint32_t shares) {
  using J = Join<NB>;
  __shared__ typename J::Lds lds;
  const uint32_t head = blockIdx.y, x = blockIdx.x / shares, first = (blockIdx.x - x * shares) * most;
  const uint64_t each = *in.each;
  uint32_t b, group;
  uint64_t at;     // the group's first tile
  if (by_edges) {
    // the group that edge x + 1 lies in, if that is its first one
    const uint64_t edge = (x + 1) * each;
    b = uniform(holder(in.before, a.batch, edge));
    const Request r = uniform(request(a, b));
    const uint32_t whole = max(r.tiles, 1u);
    const uint64_t g = (edge - in.before[b]) / whole;
    if (g >= groups_of(a, r, 16)) return;
    group = uint32_t(g);
    at = in.before[b] + g * whole;
    if (at == edge || at / each != x) return;
  } else {
    group_at(a, x, b, group);
    const Request r = uniform(request(a, b));
    if (group >= groups_of(a, r, 16)) return;
    at = in.before[b] + uint64_t(group) * max(r.tiles, 1u);
  }
  const Request rq = uniform(request(a, b));
  const uint32_t rows = min(16u, rq.n * a.group - group * 16), end = min(first + most, rows);
  const uint64_t f = at / each, pieces = (at + max(rq.tiles, 1u) - 1) / each - f + 1;
  if (pieces <= 1) return;
  // the last piece is taker f + pieces - 1's; `each` being all tiles over the takers, rounded
  // up, that is one of them as long as the arrays hold what the first launch saw
  if (f + pieces > in.slots / 2) return;
  const uint32_t count = uint32_t(pieces);
  const uint64_t p0 = uint64_t(head) * in.slots + 2 * f;
  uint32_t least = 1;
  while (2 * least * most <= J::kTeams) least *= 2;
  const uint32_t teams = J::teams(least, count), at_once = J::kTeams / teams;
  J j;
  for (uint32_t r0 = first; r0 < end; r0 += at_once) {
    const uint32_t rr = r0 + j.team / teams;
    const bool live = j.team / teams < at_once && rr < end;
    j.row(in, [&](uint32_t i) { return (p0 + (i ? 2 * i : 1)) * 16 + rr; }, count, teams, live, c, lds);
    if (!live || (j.team & (teams - 1))) continue;
    const uint32_t row = group * 16 + rr, token = per_group.div(row);
    put_row<DT>(a, rq, token, head * a.group + row - token * a.group, j.col, j.o, j.top, j.l);
  }
}

// ------------------------------------------------------------------ launch --
template <int DT, int NB>
struct Few {
  struct Sizes {
    Plan plan;
    uint32_t groups;       // row groups of a key head, at most
    bool brief, pairs;     // taken by k_attend_short; with two waves a workgroup
    bool split;            // some group may be cut into pieces
    bool few;              // not by workgroups for 128 rows
  };
  // Times below: 8 key heads of 128 values, 4 query heads each, us.
  static Sizes sizes(const AttnArgs &a) {
    Sizes z;
    z.groups = a.starts ? uint32_t(uint64_t(a.tokens) * a.group / 16 + a.batch) : a.batch * ((a.group + 15) / 16);
    // a request's queries, and the tiles that a group of them sees, as far as the sizes tell
    const uint64_t queries = !a.starts ? 1 : a.max_new ? a.max_new : (uint64_t(a.tokens) + a.batch - 1) / a.batch;
    uint64_t tiles = ((uint64_t(a.width) << a.c.shift) + kTile - 1) / kTile;
    if (a.window) tiles = std::min<uint64_t>(tiles, (a.window + queries) / kTile + 2);
    const uint64_t all = uint64_t(z.groups) * a.c.heads;
    // One launch for two where a wave has four tiles at most (8 requests of 500 or 1000
    // keys 7.5 and 10.1 for 11.4 and 13.2, 32 of 2000 18.4 for 24.0) and workgroups do not
    // wait for each other: 64 of 1000 23.4 for 24.2, 128 of 300 26.2 for 21.8; 1000
    // workgroups of FP32 queries 25.8 for 29.5.  Smaller heads have more of them at a time:
    // with 64 values 1008 workgroups 14.5 for 26.6, 2048 of 2 tiles 17.9 for 13.3, of 16
    // 37.1 for 41.7.
    z.brief = tiles <= 4 * kShortWaves<DT, NB> && all <= (DT != BF16 ? 1024 : NB > 2 ? 640 : tiles > 8 ? 2048 : 1024);
    // With two waves a workgroup more of them run at a time.  They win with two tiles a
    // cache as soon as larger ones would wait (33 requests of 100 keys 6.8 for 10.8, 128
    // 7.7 for 14.7), with eight where those would wait twice (64 of 500 keys 14.8 for 14.6,
    // 128 18.3 for 23.9), up to one and a half rounds of them (256 of 300 keys 29.4 for
    // 26.5 by shares), and beyond where heads are small (64 values, 256 of 300 14.3 for
    // 24.5, 1024 43 for 62; rows of several groups go better by 128 then).
    const uint64_t at_once = NB <= 2 || (DT != BF16 && NB <= 4) ? 512 : 256, two = (tiles + 1) / 2;
    const uint64_t most = NB > (DT == BF16 ? 2 : 4) ? 1536 : queries * a.group <= 16 ? 1u << 30 : 2560;
    // (queries is what the caller says: the grid's 2^32 threads hold whatever it is)
    z.pairs = tiles <= 8 && all * 7 > at_once * (5 + 2 * two) && all <= most && z.groups <= 1u << 24;
    z.brief = z.brief || z.pairs;
    // Waves of 16 rows take tiles that hold more rows again and again, but there are more
    // of them.  They win with up to four groups a request (64 x 2048 keys, 32 rows 59 for
    // 77, 64 rows 93 for 96, 96 rows 140 for 100; 256 x 1024 keys, 48 rows 166 for 219, 64
    // rows 220 for 223; FP32 64 x 2048 keys, 64 rows 155 for 211, 128 rows 294 for 227), or
    // where there is little to do: 8 x 2048 keys of 128 rows 40 for 50, of 256 59 for 58.
    // (With fast weights the others win from 48 rows on, 80 for 86; the rule is one, so that
    // the scratch is.)  With few tiles workgroups of 128 rows need no
    // pieces and win (16 x 200 keys of 256 rows 17 for 23).
    z.few = z.brief || queries * a.group <= 64 || (tiles > 8 && all * tiles <= 20480);
    // the takers fill the chip once, so that they all run at the same time; no more
    // of them than tiles (one more a group where a window begins inside one)
    const uint64_t n = std::min<uint64_t>(1024 * kResident<DT, NB> / a.c.heads, z.groups * (tiles + 1));
    z.plan.takers = n ? uint32_t(n) : 1;
    z.split = !z.brief && z.plan.takers > 1;
    return z;
  }
  static uint64_t scratch(const AttnArgs &a) {
    const Sizes z = sizes(a);
    if (!z.split) return 0;
    const Parts p = parts(nullptr, a.batch, a.c.heads, 2 * z.plan.takers, 16);
    return reinterpret_cast<uint64_t>(p.sums) + uint64_t(a.c.heads) * 2 * z.plan.takers * 16 * NB * 32 * 4;
  }
  static hipError_t run(const AttnArgs &a, hipStream_t s) {
    const Sizes z = sizes(a);
    const FastDiv per_group(a.group);
    const float c = float(double(a.scale) * 1.4426950408889634);
    if (z.brief) {
      const dim3 grid(z.groups, a.c.heads);
      if (z.pairs)
        k_attend_short<DT, NB, 2><<<grid, 128, 0, s>>>(a, per_group, c);
      else
        k_attend_short<DT, NB, kShortWaves<DT, NB>><<<grid, 64 * kShortWaves<DT, NB>, 0, s>>>(a, per_group, c);
      return hipGetLastError();
    }
    Parts p = {};
    if (z.split) p = parts(a.scratch, a.batch, a.c.heads, 2 * z.plan.takers, 16);
    k_attend<DT, NB><<<dim3((z.plan.takers + kWaves - 1) / kWaves, a.c.heads), 64 * kWaves, 0, s>>>(a, z.plan, p, per_group, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !z.split) return e;
    // for the rows of every group, or of every group that an edge between two shares can
    // lie in: as many rows a workgroup as it has teams for the pieces that are to be
    // expected
    const uint32_t rows = a.starts || a.group > 16 ? 16 : a.group;
    const bool by_edges = z.plan.takers - 1 < z.groups;
    const uint32_t most = std::max(1u, Join<NB>::kTeams / Join<NB>::teams(1, z.plan.takers / z.groups + 1));
    const uint32_t shares = (rows + most - 1) / most;
    k_join<DT, NB><<<dim3((by_edges ? z.plan.takers - 1 : z.groups) * shares, a.c.heads), 256, 0, s>>>(
        a, p, per_group, c, by_edges, most, shares);
    return hipGetLastError();
  }
};

}  // namespace

uint64_t attention_scratch(int dtype, const AttnArgs &a) {
  return by_kind<Few>(dtype, a.c.blocks, [&](auto k) { return k.sizes(a).few ? k.scratch(a) : attention_tall_scratch(dtype, a); });
}

int attention_kernel(int dtype, const AttnArgs &a) {
  return by_kind<Few>(dtype, a.c.blocks, [&](auto k) {
    const auto z = k.sizes(a);
    return z.pairs ? 1 : z.brief ? 0 : z.few ? 2 : 3;
  });
}

hipError_t launch_attention(int dtype, const AttnArgs &a, hipStream_t s) {
  return by_kind<Few>(dtype, a.c.blocks, [&](auto k) { return k.sizes(a).few ? k.run(a, s) : launch_attention_tall(dtype, a, s); });
}

}  // namespace zn
