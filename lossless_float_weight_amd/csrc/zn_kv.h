// zn_kv.h -- the key-value cache in 4 bits: arguments of the kernels that fill
// its block tables, write and read its rows and attend over it, and their
// launch interface.
#pragma once
#include "zn_mx.h"

namespace zn {

constexpr uint32_t kKvMaxBatch = 8192;         // requests of a step
constexpr uint32_t kKvMaxPage = 65536;         // tokens of a page (at least 16, a power of two)
constexpr uint32_t kKvMaxDim = 256;
constexpr uint32_t kKvMaxHeads = 1024;         // of keys
// strides in blocks, for products and offsets of 32 bits
constexpr uint64_t kKvMaxPageStride = 0xFFFFFFFFull, kKvMaxPlaceStride = 1ull << 20;

// Where the cache's rows lie: block i of row (page, head, place) is block
// page * page_stride + head * head_stride + place * place_stride + i.
struct KvCache {
  uint8_t *k, *ks, *v, *vs;
  uint32_t n_pages, shift;                     // page_size = 1 << shift
  uint32_t heads, blocks;                      // of keys; of a row
  uint64_t page_stride, head_stride, place_stride;
};

struct KvStepArgs {
  const int32_t *lens, *add;                   // add: NULL for a release
  const uint8_t *done;
  uint32_t batch, width, shift;
  int32_t *table;
  uint64_t table_stride;
  int32_t *free;
  uint32_t free_cap, n_pages, tokens;
  const int32_t *n_free;
  int32_t *new_lens, *starts, *slots, *positions, *n_left;
};
hipError_t launch_kv_extend(const KvStepArgs &a, hipStream_t s);
hipError_t launch_kv_release(const KvStepArgs &a, hipStream_t s);

struct KvRowsArgs {
  KvCache c;
  const uint8_t *k, *v;                        // write: plain rows
  uint64_t k_token, k_head, v_token, v_head;   // strides, elements
  uint8_t *k_out, *v_out;                      // read: dense rows
  const int32_t *slots;
  uint64_t tokens;
};
hipError_t launch_kv_write(int dtype, const KvRowsArgs &a, hipStream_t s);
hipError_t launch_kv_read(int dtype, const KvRowsArgs &a, hipStream_t s);

struct AttnArgs {
  KvCache c;
  const uint8_t *q;
  uint64_t q_token, q_head;                    // strides, elements
  uint8_t *out;
  uint64_t out_token, out_head;
  float *lse;
  const int32_t *table, *lens, *starts;        // starts: NULL for one query a request
  uint64_t table_stride;
  uint32_t width, batch, tokens, heads, group; // group: query heads of a key head
  float scale;
  uint32_t causal, window;
  uint32_t max_new;                            // 0: not known
  bool fast_weights;                           // beside BF16 queries
  uint8_t *scratch;
};
// Bytes of scratch, by the sizes alone.
uint64_t attention_scratch(int dtype, const AttnArgs &a);
// 0, 1: one launch, with many waves a workgroup or two; 2: waves of 16 rows; 3: workgroups of 128.
int attention_kernel(int dtype, const AttnArgs &a);
hipError_t launch_attention(int dtype, const AttnArgs &a, hipStream_t s);

// ------------------------------------------------------------ device side --

// Sums of v over the lanes up to this one.  32 bits where the sum surely fits.
__device__ __forceinline__ uint32_t scan32(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, false);   // a lane down, within 16
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false);   // the last of 16 to the next 16
  v += __builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false);   // the last of 32 to the next 32
  return v;
}
__device__ __forceinline__ uint64_t scan(uint64_t v) {
  if (!__any((v >> 25) != 0)) return scan32(uint32_t(v));
#pragma unroll 1
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t p = __shfl_up(v, d);
    if ((threadIdx.x & 63) >= uint32_t(d)) v += p;
  }
  return v;
}
// v of a lane that all know.
__device__ __forceinline__ uint64_t of_lane(uint64_t v, uint32_t lane) {
  return uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(v >> 32), lane))) << 32 |
         uint32_t(__builtin_amdgcn_readlane(uint32_t(v), lane));
}

}  // namespace zn
