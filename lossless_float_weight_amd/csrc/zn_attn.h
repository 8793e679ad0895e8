// zn_attn.h -- attention over the key-value cache in 4 bits: what its kernels
// share.  Codes become BF16 exactly (2 significant bits and BF16's range) and are
// multiplied by the BF16 matrix instructions, which add in FP32.
#pragma once
#include "zn_kv.h"

namespace zn {

constexpr uint32_t kTile = 64;  // keys that a wave takes at a time
// A weight is 2^(c (score - m) - kRise): m is a score, the largest of those so far or
// one that none passes by more than 2^kRise.
constexpr float kRise = 8.0f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

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

// x held to BF16's finite values.  (What an infinity or a NaN loses here lies in its
// rest, which stays infinite or NaN.)
__device__ __forceinline__ float bf16_range(float x) {
  constexpr float kMost = 0x1.fep127f;
  return fminf(fmaxf(x, -kMost), kMost);
}

// Eight FP32 values as N BF16 pieces whose sum they are (up to 2^-(8 N) of them).
// WIDE: values up to FP32's largest, whose first piece would round to infinity.
template <int N, bool WIDE = false>
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
    for (int i = 0; i < 4; i++) o.w[i] = WIDE && n == 0 ? f32_bf16x2(bf16_range(rest[2 * i]), bf16_range(rest[2 * i + 1]))
                                                        : f32_bf16x2(rest[2 * i], rest[2 * i + 1]);
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
__device__ __forceinline__ bf16x8 turned(const uint8_t *p, int next) {
  typedef __attribute__((address_space(3))) s16x4 lds16;
  union {
    s16x4 half[2];
    bf16x8 all;
  } t;
  t.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds16 *)(p));
  t.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds16 *)(p + next));
  return t.all;
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

// Keys that query `token` of a request sees: first + 0 .. count - 1.
struct Span {
  uint32_t first, count;
};
__device__ __forceinline__ Span span(const AttnArgs &a, const Request &r, uint32_t token, bool live) {
  const int64_t at = int64_t(r.len) - r.n + token;   // its position
  const int64_t end = a.causal ? at + 1 : int64_t(r.len);
  const int64_t begin = a.window && end > a.window ? end - a.window : 0;
  return live && end > begin ? Span{uint32_t(begin), uint32_t(end - begin)} : Span{0, 0};
}

// Eight consecutive values of a row of q.
template <int DT>
__device__ __forceinline__ void take_row8(const uint8_t *p, float (&x)[8]) {
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

// The same as the matrix instruction's pieces.
template <int DT, int N>
__device__ __forceinline__ void take_query8(const uint8_t *p, bool live, bf16x8 (&out)[N]) {
  if constexpr (DT == BF16) {
    out[0] = __builtin_bit_cast(bf16x8, live ? u32x4(*reinterpret_cast<const u32x4_any *>(p)) : u32x4{0, 0, 0, 0});
  } else {
    float x[8] = {};
    if (live) take_row8<DT>(p, x);
    pieces<N, true>(x, out);
  }
}

// Values that are the same in all lanes, known to be so.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return uint64_t(uniform(uint32_t(v >> 32))) << 32 | uniform(uint32_t(v));
}
__device__ __forceinline__ Request uniform(const Request &r) {
  return Request{uniform(r.start), uniform(r.n), uniform(r.len), uniform(r.lo), uniform(r.tiles), uniform(uint32_t(r.bad)) != 0};
}

__device__ __forceinline__ uint32_t groups_of(const AttnArgs &a, const Request &r, uint32_t rows) {
  return (r.n * a.group + rows - 1) / rows;
}

// Scratch: how the work was shared out (`each`, `all`, and `before` of every request);
// then per head and slot `rows` rows of (m, l), and of sums.
struct Parts {
  uint64_t *each, *all, *before;
  float2 *ml;
  float *sums;
  uint32_t slots;   // of a key head
};
__host__ __device__ __forceinline__ Parts parts(uint8_t *scratch, uint32_t batch, uint32_t kv_heads, uint32_t slots,
                                                uint32_t rows) {
  Parts p;
  p.each = reinterpret_cast<uint64_t *>(scratch);
  p.all = p.each + 1;
  p.before = p.each + 2;
  const uint64_t head = (uint64_t(batch) * 8 + 16 + 255) / 256 * 256;
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
__device__ __forceinline__ float log_sum(float m, float l, float scale) {
  return l == 0.0f ? -__builtin_inff() : __builtin_fmaf(m, scale, (kRise + __builtin_log2f(l)) * 0.6931471805599453f);
}

// A row's result from its sums over all keys.  A weight of the largest score is at least
// 2^-8, so a row without weights that sees keys has scores of -infinity alone: a NaN, as
// infinities less each other are.
template <int DT>
__device__ __forceinline__ void put_row(const AttnArgs &a, const Request &rq, uint32_t token, uint32_t qh, uint32_t col,
                                        f32x4 o, float m, float l) {
  const uint64_t y = rq.start + token;
  if (l == 0.0f && span(a, rq, token, true).count) l = __builtin_nanf("");
  store4<DT>(a.out + (y * a.out_token + qh * a.out_head + col) * esize(DT), o * over(l));
  if (a.lse && col == 0) a.lse[y * a.heads + qh] = log_sum(m, l, a.scale);
}

// NaNs among a tile's values would meet the weight 0 of rows that do not see their
// key, so such a block goes in as zeros, and the rows that see it are marked: bit i
// for block i of the values.  For the seldom tile that has some; a lane reads the
// scale bytes of one key, at `scales`.
template <int NB>
__device__ __attribute__((noinline)) uint32_t marked(const uint8_t *scales, uint32_t key0, uint32_t first, uint32_t count) {
  uint32_t mine = 0, bad = 0;
  for (int i = 0; i < NB; i++) mine |= uint32_t(scales[i] > 252) << i;
  for (uint64_t left = __ballot(mine != 0); left; left &= left - 1) {
    const int k = __builtin_ctzll(left);
    if (key0 + k - first < count) bad |= __builtin_amdgcn_readlane(mine, k);
  }
  return bad;
}

// A piece's share of a row, whose largest m is `top`.
__device__ __forceinline__ float share(float m, float top, float c) {
  return m == -__builtin_inff() && top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m - top) * c);
}

// Joins `count` pieces of a row, by a workgroup of 256: teams of D / 4 lanes, four
// values each; `each` neighbouring teams (a power of two) have a row, take every so
// manieth piece in order and are joined in order.  The row's sums are its first
// team's.  All threads of a workgroup call it, with the same count and each.
template <int NB>
struct Join {
  static constexpr uint32_t D = 32 * NB, kLanes = D / 4, kTeams = 256 / kLanes;
  struct Lds {
    __attribute__((aligned(16))) float sums[kTeams][D + 4];
    float2 ml[kTeams];
  };
  uint32_t team = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 4;
  float top, l;
  f32x4 o;
  // at least `least` teams a row, four pieces or more for each of further ones
  static __host__ __device__ __forceinline__ uint32_t teams(uint32_t least, uint32_t count) {
    while (4 * least <= count && 2 * least <= kTeams) least *= 2;
    return least;
  }
  template <class P>
  __device__ __forceinline__ void row(const Parts &in, P piece, uint32_t count, uint32_t each, bool live, float c, Lds &lds) {
    const uint32_t mine = team & (each - 1);
    top = -__builtin_inff();
    l = 0.0f;
    o = f32x4{0, 0, 0, 0};
    if (live) {
      constexpr uint32_t U = 8;   // asked for together
      for (uint32_t i0 = mine; i0 < count; i0 += U * each) {
        float2 ml[U];
        f32x4 v[U];
        float up = top;
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
          const uint32_t i = i0 + u * each;
          ml[u] = make_float2(-__builtin_inff(), 0.0f);
          v[u] = f32x4{0, 0, 0, 0};
          if (i < count) {
            const uint64_t p = piece(i);
            ml[u] = in.ml[p];
            v[u] = *reinterpret_cast<const f32x4 *>(in.sums + p * D + col);
          }
        }
#pragma unroll
        for (uint32_t u = 0; u < U; u++) up = fmaxf(up, ml[u].x);
        const float f = share(top, up, c);
        l *= f;
        o *= f;
        top = up;
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
          const float g = share(ml[u].x, top, c);
          l += ml[u].y * g;
          o += v[u] * g;
        }
      }
    }
    if (each == 1) return;
    if (live) {
      *reinterpret_cast<f32x4 *>(&lds.sums[team][col]) = o;
      if (col == 0) lds.ml[team] = make_float2(top, l);
    }
    __syncthreads();
    if (live && mine == 0) {
      for (uint32_t i = 1; i < each; i++) top = fmaxf(top, lds.ml[team + i].x);
      l = 0.0f;
      o = f32x4{0, 0, 0, 0};
      for (uint32_t i = 0; i < each; i++) {
        const float f = share(lds.ml[team + i].x, top, c);
        l += lds.ml[team + i].y * f;
        o += *reinterpret_cast<const f32x4 *>(&lds.sums[team + i][col]) * f;
      }
    }
    __syncthreads();
  }
};
// The last request b with before[b] <= v (before rises from 0), by one wave: 64
// places a step.
__device__ __forceinline__ uint32_t holder(const uint64_t *before, uint32_t batch, uint64_t v) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0;
  for (uint32_t n = batch; n > 1;) {
    const uint32_t step = (n + 63) / 64, i = lane * step;
    const uint64_t at = before[lo + min(i, n - 1)];
    const uint32_t last = __popcll(__ballot(i < n && at <= v)) - 1;   // place 0 always
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// f of the kernels K<type, blocks of 32 values of a head>, for the call's.
template <template <int, int> class K, int DT, class F>
auto by_blocks(uint32_t blocks, F f) {
  switch (blocks) {
    case 1: return f(K<DT, 1>());
    case 2: return f(K<DT, 2>());
    case 3: return f(K<DT, 3>());
    case 4: return f(K<DT, 4>());
    case 5: return f(K<DT, 5>());
    case 6: return f(K<DT, 6>());
    case 7: return f(K<DT, 7>());
    default: return f(K<DT, 8>());
  }
}
template <template <int, int> class K, class F>
auto by_kind(int dtype, uint32_t blocks, F f) {
  return dtype == BF16 ? by_blocks<K, BF16>(blocks, f) : by_blocks<K, FP32>(blocks, f);
}

// zn_attn_tall.hip
uint64_t attention_tall_scratch(int dtype, const AttnArgs &a);
hipError_t launch_attention_tall(int dtype, const AttnArgs &a, hipStream_t s);

}  // namespace zn
