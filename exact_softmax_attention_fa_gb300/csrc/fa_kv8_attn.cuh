// What the two kernels of the attention over the 8-bit cache share
// (fa_fwd_kv8.cu: few query rows per K/V head, fa_fwd_kv8_tile.cu: many).
#pragma once

#include "fa_kv8.cuh"

namespace fa {

constexpr int kMaxSms = 152;      // sizes the partial results
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kShift = 6.f;     // a reference lies this far (base 2) below its row's maximum
// l is kept times 2^-10: its terms lie between 2^(6 - 120 - 10) and
// 2^(14 + 100 - 10) for the scales a cache holds, so neither one term nor 2^22
// of them leave fp32's normal range.
constexpr float kSumBias = 10.f;
// A value scale enters the weights P_j = 2^(t_j + log2 sv_j - m) and, as 1 / sv_j, the
// sum. Its exponent is held to at least kMinScaleExp (a page of zeros has that, and
// below it the terms of l overflow) and to at most kScaleSpread below the largest one
// that the run has met in its sequence and head: with scales further apart the weights
// of the smaller one, and with them their part of l, would leave fp32's range. What is
// lost is the size of values below 2^-91, and of values below 2^-89 of the
// sequence's largest.
constexpr int kMinScaleExp = -100, kScaleSpread = 90;

// One call, as both kernels take it.
struct Kv8Call {
  Kv8Cache c;
  const __nv_bfloat16* q;  // [B][Hq][Nq][d]
  __nv_bfloat16* o;
  float* lse;              // [B][Hq][Nq]
  int Hq, Nq, g, causal;   // g query heads per K/V head
  float scale_log2;
  int fill;                // rows without a result are set to 0
};

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// What a query row is multiplied with before it is split into e4m3 pieces:
// 2^e, or NaN for a row that holds an infinity or NaN (amax: bits of its largest
// |bf16|), whose scores are infinite or NaN and whose output is NaN either way;
// the pieces would saturate.
__device__ __forceinline__ float query_factor(uint32_t amax, int e) {
  return amax >= 0x7f80u ? __int_as_float(0x7fc00000) : exp2i(e);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Tokens of sequence b, or 0 where the stored length is out of range.
__device__ __forceinline__ int seq_len(const Kv8Cache& c, int b) {
  const int len = __ldg(c.lens + b);
  return len < 0 || len > (static_cast<long long>(c.max_pages) << c.page_log2) ? 0 : len;
}
__device__ __forceinline__ int seq_count(const Kv8Cache& c, int b, int n) {
  const int count = c.counts ? __ldg(c.counts + b) : n;
  return count < 0 || count > n ? 0 : count;
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Exponent of a value scale (rounded down; -126 for all smaller ones).
__device__ __forceinline__ int scale_exponent(float sv) {
  return min(max(static_cast<int>(__float_as_uint(sv) >> 23 & 255) - 127, -126), 126);
}

// log2 of the value scales of a run's 16-key groups and 2^-kSumBias / sv, 32
// consecutive groups at a time, one a lane; `id`: the group's sequence and head.
struct ScaleRun {
  int id = -1, most = -1000;  // of the last lane's id so far: the largest exponent
  __device__ __forceinline__ void take(bool has, float sv, int group_id, float* log2_sv, float* inv) {
    const int e = scale_exponent(sv);
    if (has) {
      *log2_sv = static_cast<float>(e) + log2f(sv * exp2i(-e));  // exact for a power of two
      *inv = exp2i(-static_cast<int>(kSumBias)) / sv;
    }
    const bool near = !has || (group_id == id && e <= most && e >= max(most - kScaleSpread, kMinScaleExp));
    if (__all_sync(0xffffffffu, near)) return;
    // A new id or a larger scale, or one to hold. The later groups of an id count too:
    // one softmax step takes several of them with one reference.
    int own = __reduce_max_sync(__match_any_sync(0xffffffffu, group_id), has ? e : -1000);
    if (group_id == id) own = max(own, most);
    id = __shfl_sync(0xffffffffu, group_id, 31);
    most = __shfl_sync(0xffffffffu, own, 31);
    const int least = max(own - kScaleSpread, kMinScaleExp);
    if (has && e < least) {
      *log2_sv = static_cast<float>(least);
      *inv = exp2i(-static_cast<int>(kSumBias) - least);
    }
  }
};

// l 2^d, d <= 0 (exp2_d: 2^d): in two steps where 2^d alone would leave fp32's range; a
// sum of small value scales that meets a far larger one is as large as its factor is small.
__device__ __forceinline__ float scale_sum(float l, float d, float exp2_d) {
  if (d < -100.f && l > 0.f) {
    const float half = ex2_approx(0.5f * d);
    return l * half * half;
  }
  return l * exp2_d;
}
// a 2^da + b 2^db likewise (wa, wb: 2^da, 2^db).
__device__ __forceinline__ float add_sums(float a, float da, float wa, float b, float db, float wb) {
  if (fminf(da, db) < -100.f && a > 0.f && b > 0.f) return scale_sum(a, da, wa) + scale_sum(b, db, wb);
  return a * wa + b * wb;
}

// x / (l 2^kSumBias) and ln of the row's sum, for sums near either end of
// fp32's range; a row that saw no key has l = 0: O = 0, L = -inf.
struct RowEnd {
  float a, b, lse;
  __device__ __forceinline__ RowEnd(float m, float l) {
    const int e = min(static_cast<int>(__float_as_uint(l) >> 23 & 255) - 127, 126);  // l >= 0
    b = exp2i(-e);
    // l - l: NaN, not 0, for an infinite sum
    a = l == 0.f ? 0.f : exp2i(-static_cast<int>(kSumBias)) / (l * b) + (l - l);
    lse = l == 0.f ? -INFINITY : (m + kSumBias + log2f(l)) * kLn2;
  }
  __device__ __forceinline__ float operator()(float x) const { return a == 0.f ? 0.f : x * a * b; }
};

// fa_fwd_kv8_tile.cu
size_t kv8_tile_workspace(int d);
fa_status_t launch_kv8_tiles(const Kv8Call& call, int d, void* workspace, const DeviceInfo& dev, cudaStream_t stream);

// fa_api.cu: tensor map {d, page, slots} of the cache's codes, boxes of one page and at most 128 columns,
// swizzled by the row's bytes (64 or 128).
bool make_cache_map(CUtensorMap* m, const void* base, int d, int page, long long slots);

}  // namespace fa
