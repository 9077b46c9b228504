// The plan of a batch of packed sequences (fa_packed_plan of fa.h): what the
// attention kernels read of it.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace fa {

// Head of the plan in device memory. Behind it lie two lists of {first row of
// the sequence, its length, index in it, 0}: the sequences' 128-row tiles, and
// their pairs of neighbouring tiles. Both are ordered by the work of a query
// tile, most first: the key tiles it sees, which are index + 1 of a causal plan
// and all the sequence's else. (A causal key tile sees what is behind it, so
// the same list read with j = last - index is ordered for them too.)
struct PackedPlan {
  uint32_t magic;
  int rows;               // rows of the tensors it was made for
  int n_tiles, n_pairs;
  int pairs_at;           // first entry of the second list
  int max_tiles;          // tiles of the longest sequence
  int row_begin, row_end; // rows that belong to a sequence
  unsigned long long causal_products, full_products;  // (query tile, key tile) pairs per head
};
constexpr uint32_t kPackedMagic = 0x46415031u;
constexpr int kPackedHead = 256;  // bytes before the lists

__device__ __forceinline__ const int4* packed_tiles(const PackedPlan* p) {
  return reinterpret_cast<const int4*>(reinterpret_cast<const uint8_t*>(p) + kPackedHead);
}
__device__ __forceinline__ const int4* packed_pairs(const PackedPlan* p) { return packed_tiles(p) + p->pairs_at; }

// A plan that was never made, or made for other tensors, has no work.
__device__ __forceinline__ bool packed_plan_ok(const PackedPlan* p, int rows) {
  return p->magic == kPackedMagic && p->rows == rows;
}

// Whole warp: rows [from, to) of a 128-byte-swizzled tile in shared memory (its
// 64-column chunks CHUNK_BYTES apart) become zeros that the tensor core sees.
template <int CHUNKS, int CHUNK_BYTES>
__device__ __forceinline__ void clear_rows(uint32_t tile, int from, int to) {
  const int units = (to - from) * 8;  // of 16 bytes, in a chunk
  for (int i = lane_id(); i < units; i += 32)
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) st_shared_v4(tile + c * CHUNK_BYTES + from * 128 + i * 16, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace fa
