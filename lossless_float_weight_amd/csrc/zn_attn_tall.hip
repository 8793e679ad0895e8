// zn_attn_tall.hip -- attention over the key-value cache in 4 bits for requests
// with many rows (a request's queries times the query heads of a key head): the
// method of zn_attn.hip with a workgroup of four waves for 128 rows.
//
// A wave takes 32 rows and 64 keys at a time with v_mfma_f32_32x32x16_bf16, keys
// and values as the first operand: scores come out with a lane holding row l % 32
// and keys 8 b + 4 h + i of each 32 (h = l / 32, b, i = 0 .. 3), which is the
// second operand's layout for the product with the values; a row's maximum is one
// exchange away.  A conversion of two codes takes as long as an exponential (8
// cycles of a SIMD, where other instructions take 2), so a tile is converted once,
// by all four waves, into one of two places in LDS while the other is used: one
// barrier a tile.
//
// A prompt of 8192 queries, 32 heads, takes 741 to 776 us, 0.72 PFLOP/s, or 1.09 with the
// second product that weights of 16 bits take: the matrix units are busy 49% of the
// cycles and the vector units 57% (exponentials, conversions, the split of the weights),
// and the two run beside each other little: two waves, one of each kind, take 0.83 of the
// sum of their times.
#include <algorithm>

#include "zn_attn.h"

namespace zn {
namespace {

constexpr uint32_t kRows = 128;     // of a workgroup
constexpr uint32_t kThreads = 256;
// Tiles of a piece at least.  A piece of 128 rows is 67 KB that the join reads back: 16
// requests of 1000 keys, 64 queries each, 60 us with pieces of 8 tiles, 44 with 16; a
// group by itself loses (one request of 1000 keys, 64 queries: 24 us with 4, 37 with
// 16), but so little work is not taken here.
constexpr uint32_t kLeast = 16;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma_half(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// Eight values, or eight codes under a scale, in FP16.
__device__ __forceinline__ u32x4 half8(const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; i++)
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * i], x[2 * i + 1]}, f16x2));
  return w;
}
__device__ __forceinline__ u32x4 halves8(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3))};
}

// The larger of lanes l and l + 32 (NaNs lose).
__device__ __forceinline__ float max_h(float x) {
  const uint32_t w = __float_as_uint(x);
  const auto p = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// How the work is shared out.  Rows of a request go in groups of 128, and the keys
// of a group in pieces of `piece` tiles, so many that a head's items, (request,
// rows, piece), come to about `items` where the rows alone give fewer: with tiles
// t_b and groups g_b, sum g_b ceil(t_b / piece) <= items + sum g_b.  Requests of
// several pieces have t_b > piece, so at most 2 `items` items are pieces to be
// joined; they are numbered apart.  Items go from the last to the first, all heads'
// of one number together: the last rows of a prompt see the most keys, and long
// items at the end would leave the others waiting (head after head, 8192 rows of 8
// heads took 950 us for 730).  Neighbouring workgroups run on different dies, so
// eight heads keep to one die's cache each.  Every wave finds its item by itself,
// with two sums over the requests; the host knows the bounds alone.
struct Plan {
  uint32_t items;
};
struct Item {
  uint32_t b, group, piece, pieces;
  uint64_t slot;      // where a piece goes
  uint64_t tiles;     // of a piece
};

__device__ __forceinline__ bool find_item(const AttnArgs &a, const Plan &plan, uint32_t number, bool tell, uint64_t *each,
                                          uint64_t *whole, uint64_t *before, Item &it) {
  const uint32_t lane = threadIdx.x & 63, per = (a.batch + 63) / 64;
  uint64_t mine = 0;
  for (uint32_t i = 0; i < per; i++)
    if (lane * per + i < a.batch) {
      const Request r = request(a, lane * per + i);
      mine += uint64_t(groups_of(a, r, kRows)) * max(r.tiles, 1u);
    }
  const uint64_t total = of_lane(scan(mine), 63);
  uint64_t piece = (total + plan.items - 1) / plan.items;
  piece = piece < kLeast ? kLeast : piece;
  uint64_t items = 0, parts = 0;
  for (uint32_t i = 0; i < per; i++)
    if (lane * per + i < a.batch) {
      const Request r = request(a, lane * per + i);
      const uint64_t g = groups_of(a, r, kRows), p = (max(r.tiles, 1u) + piece - 1) / piece;
      items += g * p;
      if (p > 1) parts += g * p;
    }
  const uint64_t upto = scan(items), parts_upto = scan(parts), all = of_lane(upto, 63);
  // the requests' numbers of pieces for the join
  if (tell && threadIdx.x < 64) {
    uint64_t at = parts_upto - parts;
    for (uint32_t i = 0; i < per; i++)
      if (lane * per + i < a.batch) {
        before[lane * per + i] = at;
        const Request r = request(a, lane * per + i);
        const uint64_t g = groups_of(a, r, kRows), p = (max(r.tiles, 1u) + piece - 1) / piece;
        if (p > 1) at += g * p;
      }
    // starts out of order can make more items than there are workgroups: pieces are
    // missing then, and none are joined
    if (lane == 63) {
      *each = piece;
      *whole = all > gridDim.x / a.c.heads ? 0 : parts_upto;
    }
  }
  if (number >= all) return false;
  const uint64_t want = all - 1 - number;
  const uint32_t owner = uniform(uint32_t(__popcll(__ballot(upto <= want))));
  uint64_t first = of_lane(upto - items, owner), slot = of_lane(parts_upto - parts, owner);
  for (uint32_t b = owner * per;; b++) {
    const Request r = request(a, b);
    const uint64_t g = groups_of(a, r, kRows), p = (max(r.tiles, 1u) + piece - 1) / piece;
    if (want < first + g * p) {
      const uint32_t i = uint32_t(want - first);
      it.b = uniform(b);
      it.pieces = uniform(uint32_t(p));
      it.group = uniform(i / it.pieces);
      it.piece = uniform(i - it.group * it.pieces);
      it.slot = uniform(slot + i);
      it.tiles = uniform((r.tiles + p - 1) / p);   // pieces of a request are alike
      return true;
    }
    first += g * p;
    if (p > 1) slot += g * p;
  }
}

template <int DT, int NB>
constexpr int kResident = DT == BF16 ? NB == 1 ? 4 : NB == 2 ? 3 : NB <= 4 ? 2 : 1 : NB <= 2 ? 2 : 1;   // waves a SIMD

template <int DT, int NB>
struct Shape {
  static constexpr int QP = DT == BF16 ? 1 : 3;                  // pieces of a query
  static constexpr int kSteps = 2 * NB;                          // of 16 values of a key
  // bytes of a key's values in LDS: 64 modulo 128, so that four keys' parts fill the
  // banks; and of its keys, 16 modulo 32, for rows of 16 bytes a lane
  static constexpr int kPitch = 64 * NB + (NB % 2 ? 0 : 64), kKeyPitch = 64 * NB + 16;
  // blocks of a tile that a thread converts, of 64 NB of keys and then as many of values
  static constexpr uint32_t kBlocks = kTile * NB;
  static constexpr int kUnits = int((2 * kBlocks + kThreads - 1) / kThreads);
  struct Lds {
    __attribute__((aligned(16))) uint8_t v[2][kTile * kPitch], k[2][kTile * kKeyPitch];
    uint32_t odd[3];     // a tile has a NaN (1), scales out of reach (2): this one, the next, the one after
    uint32_t top;        // the largest scale byte of the first tile
  };
};

// What a wave has of its rows.
template <int DT, int NB>
struct Rows32 {
  bf16x8 q[2 * NB][DT == BF16 ? 1 : 3];
  Span sees;                                   // this lane's row
  uint32_t low, high, low_all, high_all;       // keys that some row of the wave sees, and that all see
  uint32_t wg_low, wg_high;                    // that some row of the workgroup sees
  f32x16 o[NB];                                // sums, times 2^(127 - unit)
  float m, l;
  uint32_t marks;                              // blocks of values that have a NaN for this row
  uint32_t unit;
};

// The product with the values is one of two.
//   HALF, beside BF16 queries where the caller asks for fast weights: weights and values in FP16, one product.  Weights go up
// to 2^15 and keep 11 bits down to 2^-14 (beside a largest one of 2^7 or more), the
// values are held relative to the largest scale of the first tile and are exact normal
// numbers while the tiles' scales lie within 2^-13 and 2^12 of it.  (Subnormal ones are
// exact too, but the instruction adds them with fewer bits: at 2^-23 sums were off by
// 2^-13.)  A tile with others ends it, false is returned, and the rows are taken again
// the other way.
//   Otherwise weights in BF16 pieces (two beside BF16 queries, three beside FP32),
// a product each, and values in BF16, exact whatever their scales.
// The first takes two thirds of the matrix instructions and three quarters of the
// others: 8192 queries of 32 heads 609 us for 769, 64 x 4096 keys of 128 rows 179 for
// 220 (one card).
template <int DT, int NB, bool HALF>
__device__ __forceinline__ bool take_tiles(const AttnArgs &a, const Request &rq, const int32_t *pages, uint32_t head,
                                           uint32_t t, uint32_t end, float c, typename Shape<DT, NB>::Lds &lds,
                                           Rows32<DT, NB> &r) {
  using S = Shape<DT, NB>;
  constexpr int WP = HALF ? 1 : DT == BF16 ? 2 : 3;      // pieces of a weight
  constexpr float kTop = HALF ? 15.0f : 0.0f;            // weights stay under 2^kTop
  constexpr int kBelow = 13, kAbove = 12;                // scales that HALF takes
  const uint32_t lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
  const uint8_t *kc = a.c.k + head * a.c.head_stride * 16, *vc = a.c.v + head * a.c.head_stride * 16;
  const uint8_t *ksc = a.c.ks + head * a.c.head_stride, *vsc = a.c.vs + head * a.c.head_stride;
  const uint32_t mask = (1u << a.c.shift) - 1, place = uint32_t(a.c.place_stride), page_stride = uint32_t(a.c.page_stride);
  const uint32_t wg_low = r.wg_low, wg_high = r.wg_high;
#pragma unroll
  for (int d = 0; d < NB; d++) r.o[d] = f32x16{};
  r.m = -__builtin_inff();
  r.l = 0.0f;
  r.marks = 0;
  r.unit = 127;

  // A thread's unit u is block `number % NB` of key number / NB of a tile, of its keys
  // or of its values, the same for a whole wave.  Pages are asked for a tile ahead of
  // the codes (behind the last key, the last one's).  A place outside any page is
  // taken from page 0 and counts as a NaN.
  const uint32_t wave = uniform(threadIdx.x >> 6);
  auto is_key = [&](int u) {
    return kThreads * (u + 1) <= S::kBlocks || (kThreads * u < S::kBlocks && kThreads * u + 64 * wave < S::kBlocks);
  };
  auto number = [&](int u) {
    const uint32_t x = min(threadIdx.x + kThreads * u, 2 * S::kBlocks - 1);
    return x < S::kBlocks ? x : x - S::kBlocks;
  };
  auto is_unit = [&](int u) { return kThreads * (u + 1) <= 2 * S::kBlocks || kThreads * u + 64 * wave < 2 * S::kBlocks; };
  uint32_t page[S::kUnits];
  auto ask_pages = [&](uint32_t key0) {
#pragma unroll
    for (int u = 0; u < S::kUnits; u++) page[u] = uint32_t(pages[min(key0 + number(u) / NB, rq.len - 1) >> a.c.shift]);
  };
  auto block_of = [&](uint32_t page, uint32_t key) {
    return uint64_t(page < a.c.n_pages ? page : 0) * page_stride + uint64_t(key & mask) * place;
  };
  u32x4 code[S::kUnits];
  uint32_t byte[S::kUnits];
  bool gone[S::kUnits];
  auto ask = [&](uint32_t key0) {
#pragma unroll
    for (int u = 0; u < S::kUnits; u++) {
      const uint64_t block = block_of(page[u], key0 + number(u) / NB) + number(u) % NB;
      gone[u] = page[u] >= a.c.n_pages;
      code[u] = *reinterpret_cast<const u32x4 *>((is_key(u) ? kc : vc) + block * 16);
      byte[u] = (is_key(u) ? ksc : vsc)[block];
    }
  };
  // Whether a thread's block of values counts for scales: no row sees a key outside
  // [wg_low, wg_high), NaNs are marked, and zeros have any scale.
  auto counts = [&](uint32_t key0, int u) {
    return is_unit(u) && !is_key(u) && key0 + number(u) / NB - wg_low < wg_high - wg_low && byte[u] <= 252 &&
           ((code[u][0] | code[u][1] | code[u][2] | code[u][3]) & 0x77777777u) != 0;
  };
  // A thread's blocks to LDS.  Those of values go 16 bytes at a time in an order of
  // the lane's own, so that neighbouring lanes, 64 bytes apart, meet different banks.
  auto put = [&](uint32_t key0, uint32_t buf, uint32_t flag) {
    const bool cut = key0 < wg_low || key0 + kTile > wg_high;
#pragma unroll
    for (int u = 0; u < S::kUnits; u++) {
      if (!is_unit(u)) continue;
      const uint32_t key = number(u) / NB, blk = number(u) % NB;
      if (is_key(u)) {
        const float f = scale_of(gone[u] ? 255u : byte[u]);
        uint8_t *p = lds.k[buf] + key * S::kKeyPitch + blk * 64;
#pragma unroll
        for (int i = 0; i < 4; i++) *reinterpret_cast<bf16x8 *>(p + 16 * i) = values8(code[u][i], f);
        continue;
      }
      if (cut && key0 + key - wg_low >= wg_high - wg_low) {
        code[u] = u32x4{0, 0, 0, 0};
        byte[u] = r.unit;
      }
      // seldom: a NaN, or a scale out of reach
      const bool bad = byte[u] > 252 || (HALF && byte[u] + kBelow - r.unit > kBelow + kAbove);
      if (__builtin_expect(__any(bad), 0)) {
        if (byte[u] > 252) {
          atomicOr(&lds.odd[flag], 1u);
          code[u] = u32x4{0, 0, 0, 0};
        }
        if (HALF && bad && counts(key0, u)) atomicOr(&lds.odd[flag], 2u);
        if (bad) byte[u] = r.unit;
      }
      const float f = __uint_as_float((HALF ? byte[u] + 127 - r.unit : byte[u]) << 23);
      uint8_t *p = lds.v[buf] + key * S::kPitch + blk * 64;
      const bool one = threadIdx.x & 1, two = threadIdx.x & 2;
      const u32x4 x = {one ? code[u][1] : code[u][0], one ? code[u][0] : code[u][1], one ? code[u][3] : code[u][2],
                       one ? code[u][2] : code[u][3]};
      const u32x4 y = {two ? x[2] : x[0], two ? x[3] : x[1], two ? x[0] : x[2], two ? x[1] : x[3]};
      const uint32_t turn = (threadIdx.x & 3) * 16;
#pragma unroll
      for (uint32_t i = 0; i < 4; i++)
        *reinterpret_cast<u32x4 *>(p + (16 * i ^ turn)) =
            HALF ? halves8(y[i], f) : __builtin_bit_cast(u32x4, values8(y[i], f));
    }
  };

  if (threadIdx.x < 3) lds.odd[threadIdx.x] = 0;
  if (HALF && threadIdx.x == 3) lds.top = 0;
  __syncthreads();
  if (t < end) {
    const uint32_t key0 = rq.lo + t * kTile;
    ask_pages(key0);
    ask(key0);
    ask_pages(key0 + kTile);
    if constexpr (HALF) {
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < S::kUnits; u++)
        if (counts(key0, u)) top = max(top, byte[u] + 1);
#pragma unroll
      for (int d = 1; d < 64; d *= 2) top = max(top, uint32_t(__shfl_xor(int(top), d)));
      if (lane == 0) atomicMax(&lds.top, top);
      __syncthreads();
      top = uniform(lds.top);
      r.unit = top ? top - 1 : 127;
    }
    put(key0, t & 1, 0);
  }
  __syncthreads();
  for (uint32_t flag = 0; t < end; t++) {
    const uint32_t next = flag == 2 ? 0 : flag + 1;
    if (threadIdx.x == 0) lds.odd[next == 2 ? 0 : next + 1] = 0;   // read a tile ago, written in the next one
    const uint32_t key0 = rq.lo + t * kTile, buf = t & 1;
    const uint32_t odd = uniform(lds.odd[flag]);
    if (HALF && __builtin_expect(odd & 2, 0)) return false;
    const bool more = t + 1 < end;
    if (more) {
      ask(key0 + kTile);
      ask_pages(key0 + 2 * kTile);
    }
    if (key0 < r.high && key0 + kTile > r.low) {   // some row of this wave sees the tile
      // Scores by themselves: sums that begin with -m would save the subtraction below (no
      // time that could be measured; 2% with fast weights), but round where an old m is
      // large: a score of 0 after a first tile of scores around -768 was off by 2^-15.
      f32x16 s[2] = {};
      const uint8_t *keys = lds.k[buf] + n * S::kKeyPitch + 16 * h;
#pragma unroll
      for (int st = 0; st < S::kSteps; st++)
#pragma unroll
        for (int g = 0; g < 2; g++) {
          const bf16x8 k = *reinterpret_cast<const bf16x8 *>(keys + 32 * g * S::kKeyPitch + 32 * st);
#pragma unroll
          for (int p = S::QP - 1; p >= 0; p--) s[g] = mfma(k, r.q[st][p], s[g]);
        }
      // keys that the row does not see
      if (key0 < r.low_all || key0 + kTile > r.high_all) {
#pragma unroll
        for (int g = 0; g < 2; g++)
#pragma unroll
          for (int i = 0; i < 16; i++)
            if (key0 + 32 * g + 8 * (i / 4) + 4 * h + i % 4 - r.sees.first >= r.sees.count) s[g][i] = -__builtin_inff();
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int g = 0; g < 2; g++)
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, s[g][i]);
      top = max_h(top);
      if (__any((top - r.m) * c > kRise)) {
        const float up = fmaxf(top, r.m);
        const float f = up > r.m ? __builtin_amdgcn_exp2f((r.m - up) * c) : 1.0f;
        r.l *= f;
#pragma unroll
        for (int d = 0; d < NB; d++) r.o[d] *= f;
        r.m = up;
      }
      const float m = r.m == -__builtin_inff() ? 0.0f : r.m;
      // 16 keys of 32 values at a time; the weights of the next 16 keys are made while
      // the matrix unit takes these
      const uint8_t *from = lds.v[buf] + (4 * h + (lane & 15) / 4) * S::kPitch + (lane >> 4 & 1) * 32 + (lane & 3) * 8;
      if (__builtin_expect(odd & 1, 0)) {
        const uint32_t key = min(key0 + lane, rq.len - 1);
        r.marks |= marked<NB>(vsc + block_of(pages[key >> a.c.shift], key), key0, r.sees.first, r.sees.count);
      }
      bf16x8 wp[2][WP], v[NB];
      auto weigh = [&](int g) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
          x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][8 * (g & 1) + i] - m, c, kTop - kRise));
          r.l += x[i];
        }
        if constexpr (HALF)
          wp[g & 1][0] = __builtin_bit_cast(bf16x8, half8(x));
        else
          pieces<WP>(x, wp[g & 1]);
      };
      weigh(0);
#pragma unroll
      for (int g = 0; g < 4; g++) {
#pragma unroll
        for (int d = 0; d < NB; d++) v[d] = turned(from + 16 * g * S::kPitch + 64 * d, 8 * S::kPitch);
        if (g < 3) weigh(g + 1);
#pragma unroll
        for (int p = WP - 1; p >= 0; p--)
#pragma unroll
          for (int d = 0; d < NB; d++) r.o[d] = HALF ? mfma_half(v[d], wp[g & 1][p], r.o[d]) : mfma(v[d], wp[g & 1][p], r.o[d]);
      }
    }
    if (more) put(key0 + kTile, buf ^ 1, next);
    flag = next;
    __syncthreads();
  }
  if constexpr (HALF) {   // weights under 1 again, as the other way leaves them
    constexpr float kDown = 0x1p-15f;
    r.l *= kDown;
#pragma unroll
    for (int d = 0; d < NB; d++) r.o[d] *= kDown;
  }
  return true;
}

template <int DT, int NB, bool FAST>
__global__ __launch_bounds__(kThreads, (kResident<DT, NB>)) void k_attend_tall(AttnArgs a, Plan plan, Parts out,
                                                                          FastDiv per_group, float c) {
  constexpr int D = 32 * NB;
  __shared__ typename Shape<DT, NB>::Lds lds;
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t n = lane & 31, h = lane >> 5;
  const uint32_t number = blockIdx.x / a.c.heads, head = blockIdx.x - number * a.c.heads;

  Item it;
  if (!find_item(a, plan, number, blockIdx.x == 0 && out.each, out.each, out.all, out.before, it)) return;
  const Request rq = uniform(request(a, it.b));
  // this lane's row
  const uint32_t row = it.group * kRows + wave * 32 + n;
  const bool live = row < rq.n * a.group;
  const uint32_t token = live ? per_group.div(row) : 0;
  const uint32_t qh = head * a.group + (live ? row - token * a.group : 0);
  Rows32<DT, NB> r;
  const Span sees = r.sees = span(a, rq, token, live);
  r.low = sees.count ? sees.first : ~0u;
  r.high = sees.count ? sees.first + sees.count : 0;
  r.low_all = live ? sees.first : 0;
  r.high_all = live ? sees.first + sees.count : ~0u;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    r.low = min(r.low, uint32_t(__shfl_xor(int(r.low), d)));
    r.high = max(r.high, uint32_t(__shfl_xor(int(r.high), d)));
    r.low_all = max(r.low_all, uint32_t(__shfl_xor(int(r.low_all), d)));
    r.high_all = min(r.high_all, uint32_t(__shfl_xor(int(r.high_all), d)));
  }
  r.low = uniform(r.low);
  r.high = uniform(r.high);
  r.low_all = uniform(r.low_all);
  r.high_all = uniform(r.high_all);
  // the workgroup's first and last row have the first and the last key
  const uint32_t last_row = min(it.group * kRows + kRows, rq.n * a.group) - 1;
  const Span s0 = span(a, rq, uniform(per_group.div(it.group * kRows)), true);
  const Span s1 = span(a, rq, uniform(per_group.div(last_row)), true);
  r.wg_high = s1.first + s1.count;
  r.wg_low = s0.count ? s0.first : 0;
#pragma unroll
  for (int s = 0; s < 2 * NB; s++) {
    take_query8<DT>(a.q + ((rq.start + token) * a.q_token + qh * a.q_head + 16 * s + 8 * h) * esize(DT), live, r.q[s]);
  }

  const int32_t *pages = a.table + it.b * a.table_stride;
  uint32_t t = uint32_t(min(it.piece * it.tiles, uint64_t(rq.tiles)));
  uint32_t end = uint32_t(min((it.piece + 1) * it.tiles, uint64_t(rq.tiles)));
  end = r.wg_high > rq.lo ? min(end, (r.wg_high - rq.lo + kTile - 1) / kTile) : 0;
  if (r.wg_low > rq.lo) t = max(t, (r.wg_low - rq.lo) / kTile);
  if (!FAST || !take_tiles<DT, NB, FAST>(a, rq, pages, head, t, end, c, lds, r)) {
    __syncthreads();
    take_tiles<DT, NB, false>(a, rq, pages, head, t, end, c, lds, r);
  }

  float l = r.l;
  l += __shfl_xor(l, 32);
  if (rq.bad) l = __builtin_nanf("");
  if (!live) return;
#pragma unroll
  for (int d = 0; d < NB; d++)
    if (r.marks >> d & 1) r.o[d] = f32x16{} + __builtin_nanf("");
  const int unit = int(r.unit) - 127;
  if (it.pieces == 1) {
    const uint64_t y = rq.start + token;
    if (l == 0.0f && sees.count) l = __builtin_nanf("");   // as in put_row
    const float f = over(l);
    uint8_t *p = a.out + (y * a.out_token + qh * a.out_head + 4 * h) * esize(DT);
#pragma unroll
    for (int d = 0; d < NB; d++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = __builtin_ldexpf(r.o[d][4 * i + e] * f, unit);
        store4<DT>(p + (32 * d + 8 * i) * esize(DT), v);
      }
    if (a.lse && h == 0) a.lse[y * a.heads + qh] = log_sum(r.m, l, a.scale);
  } else if (it.slot < out.slots) {   // starts out of order can make more pieces than there is room for
    const uint64_t p = (uint64_t(head) * out.slots + it.slot) * kRows + wave * 32 + n;
#pragma unroll
    for (int d = 0; d < NB; d++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = __builtin_ldexpf(r.o[d][4 * i + e], unit);
        *reinterpret_cast<f32x4 *>(out.sums + p * D + 32 * d + 8 * i + 4 * h) = v;
      }
    if (h == 0) out.ml[p] = make_float2(r.m, l);
  }
}

// Joins the pieces of a group.  Its rows are shared out over the workgroups of all
// its slots, with few pieces a team a row, with many up to a workgroup's teams (one
// request of 32768 keys, 32 rows, the attention with it: 70 us by a team a row, so 38);
// the workgroups go through the slots that there are.
template <int DT, int NB>
__global__ __launch_bounds__(256) void k_join_tall(AttnArgs a, Parts in, FastDiv per_group, float c) {
  using J = Join<NB>;
  constexpr uint32_t kShares = (kRows + J::kTeams - 1) / J::kTeams;
  __shared__ typename J::Lds lds;
  const uint32_t head = blockIdx.y;
  const uint64_t all = min(*in.all, uint64_t(in.slots)) * kShares, piece = *in.each;
  J j;
  for (uint64_t x = blockIdx.x; x < all; x += gridDim.x) {
    const uint32_t slot = uint32_t(x / kShares);
    const uint32_t b = uniform(holder(in.before, a.batch, slot));
    const Request rq = uniform(request(a, b));
    const uint64_t pieces = (max(rq.tiles, 1u) + piece - 1) / piece, rel = slot - in.before[b], group = rel / pieces;
    const uint32_t count = uint32_t(pieces), nth = uint32_t(rel - group * pieces);
    // (the last: starts out of order can make more pieces than there is room for)
    if (count <= 1 || group * kRows >= uint64_t(rq.n) * a.group || slot - nth + pieces > in.slots) continue;
    // no more teams a row than half the pieces: `count * kShares` workgroups have all rows
    const uint32_t teams = J::teams(1, count), rows = J::kTeams / teams;
    const uint32_t first = (nth * kShares + uint32_t(x - uint64_t(slot) * kShares)) * rows;
    if (first >= kRows) continue;
    const uint32_t r = first + j.team / teams, row = uint32_t(group) * kRows + r;
    const bool live = j.team / teams < rows && r < kRows && row < rq.n * a.group;
    const uint64_t p0 = (uint64_t(head) * in.slots + (slot - nth)) * kRows + r;
    j.row(in, [&](uint32_t i) { return p0 + i * uint64_t(kRows); }, count, teams, live, c, lds);
    if (!live || (j.team & (teams - 1))) continue;
    const uint32_t token = per_group.div(row);
    put_row<DT>(a, rq, token, head * a.group + row - token * a.group, j.col, j.o, j.top, j.l);
  }
}

// ------------------------------------------------------------------ launch --
template <int DT, int NB>
struct Tall {
  struct Sizes {
    Plan plan;
    uint32_t groups;   // row groups of a key head, at most
    uint32_t items;    // and their pieces
    uint32_t slots;    // for pieces to be joined; 0: none
  };
  static Sizes sizes(const AttnArgs &a) {
    Sizes z;
    z.groups = a.starts ? uint32_t(uint64_t(a.tokens) * a.group / kRows + a.batch) : a.batch * ((a.group + kRows - 1) / kRows);
    // as many as run at the same time
    const uint32_t want = 256 * kResident<DT, NB> / a.c.heads;
    z.plan.items = want ? want : 1;
    const uint64_t longest = ((uint64_t(a.width) << a.c.shift) + kTile - 1) / kTile + 1;
    const uint64_t most = uint64_t(z.groups) * ((longest + kLeast - 1) / kLeast);
    z.items = uint32_t(std::min<uint64_t>(most, uint64_t(z.groups) + z.plan.items));
    z.slots = longest <= kLeast ? 0 : uint32_t(std::min<uint64_t>(most, 2 * uint64_t(z.plan.items)));
    return z;
  }
  static uint64_t scratch(const AttnArgs &a) {
    const Sizes z = sizes(a);
    if (!z.slots) return 0;
    const Parts p = parts(nullptr, a.batch, a.c.heads, z.slots, kRows);
    return reinterpret_cast<uint64_t>(p.sums) + uint64_t(a.c.heads) * z.slots * kRows * NB * 32 * 4;
  }
  static hipError_t run(const AttnArgs &a, hipStream_t s) {
    const Sizes z = sizes(a);
    Parts p = {};
    if (z.slots) p = parts(a.scratch, a.batch, a.c.heads, z.slots, kRows);
    const FastDiv per_group(a.group);
    const float c = float(double(a.scale) * 1.4426950408889634);
    const dim3 grid(z.items * a.c.heads);
    if (DT == BF16 && a.fast_weights)
      k_attend_tall<DT, NB, DT == BF16><<<grid, kThreads, 0, s>>>(a, z.plan, p, per_group, c);
    else
      k_attend_tall<DT, NB, false><<<grid, kThreads, 0, s>>>(a, z.plan, p, per_group, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !z.slots) return e;
    const uint32_t shares = (kRows * NB * 8 + 255) / 256 + 1, most = 4096 / a.c.heads + 1;
    k_join_tall<DT, NB><<<dim3(std::min(z.slots * shares, most), a.c.heads), 256, 0, s>>>(a, p, per_group, c);
    return hipGetLastError();
  }
};

}  // namespace

uint64_t attention_tall_scratch(int dtype, const AttnArgs &a) {
  return by_kind<Tall>(dtype, a.c.blocks, [&](auto k) { return k.scratch(a); });
}
hipError_t launch_attention_tall(int dtype, const AttnArgs &a, hipStream_t s) {
  return by_kind<Tall>(dtype, a.c.blocks, [&](auto k) { return k.run(a, s); });
}

}  // namespace zn
