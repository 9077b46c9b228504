// The paged 8-bit key/value cache, as its writer, its reader and the attention
// see it: e4m3 codes [pages][Hkv][page][d] and one fp32 scale per page and
// head, for keys and values each; a sequence's pages are listed in its row of
// the page table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "sm103_ptx.cuh"

namespace fa {

struct Kv8Cache {
  uint8_t* code[2];   // keys, values
  float* scale[2];
  const int* table;   // [B][max_pages]
  const int* lens;    // [B] tokens of each sequence, the newest among them
  const int* counts;  // [B] of them the call's own (new tokens, queries), or null: all n
  int B, Hkv, page_log2, num_pages, max_pages;
};

// Two e4m3 codes (low byte first) as two fp16 values: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Nearest e4m3 codes of two values (ties to even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Argument checks shared by the cache's entry points (the conventions of fa.h);
// n: rows of the call's own tensors per sequence.
fa_status_t check_kv8(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                      const int* table, const int* lens, const int* counts, int B, int Hkv, int n, int d, int page,
                      int num_pages, int max_pages, bool* empty, Kv8Cache* c);

}  // namespace fa
