// Warp-level pieces of the kernels for short packed sequences: bf16 matrix
// products of a warp, and the loads that feed them from shared memory.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace fa {

// Four 8 x 8 matrices of 16-bit values: lane 8 i + j gives the address of row j of
// matrix i; lane l receives elements (l / 4, 2 (l % 4) + {0, 1}) of each, or of
// their transposes.
__device__ __forceinline__ uint4 load_matrices(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_matrices_t(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// d (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16. Lane l holds of d rows l / 4
// and l / 4 + 8, columns 2 (l % 4) + {0, 1}; of a the same rows and columns, then
// the columns 8 further on; of b rows 2 (l % 4) + {0, 1}, and 8 further on, of column l / 4.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// A tile of rows of D bf16 in shared memory, its 16-byte units swizzled by the row
// modulo 8: rows of one column, and columns of one row, are free of bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t row, uint32_t unit) {
  return row * (D * 2) + ((unit ^ (row & 7u)) << 4);
}

}  // namespace fa
