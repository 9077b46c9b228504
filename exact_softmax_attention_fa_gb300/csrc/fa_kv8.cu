// Writing the paged 8-bit key/value cache and reading it back (fa_kv8_append /
// fa_kv8_gather of fa.h).
//
// A page's scale is a power of two, the smallest 2^e with amax <= 448 * 2^e:
// value / scale and code * scale are then exact up to the one rounding to
// e4m3, the read-back is exact in bf16, and when later tokens raise a page's
// scale its earlier codes move by an exponent shift that rounds only codes
// that become subnormal. (amax / 448 itself as the scale would gain at most
// one binade of range for the smallest values, and nothing in the relative
// step of the others.)
//
// Both are HBM-bound: 2 bytes read and 1 written per value, or 1 and 2.
#include <cmath>

#include "fa_kv8.cuh"

namespace fa {
namespace {

constexpr int kGatherThreads = 64;  // 256: 70.1 instead of 68.4 us for the long cache below
// Threads of an append block: each holds eight rows' 16 bytes of a page where the
// limits allow (more threads leave the block's fixed latencies to fewer bytes: with
// 256, 8192 tokens as below took 34 us in pages of 64 and 57 in pages of 16).
constexpr int append_threads(int d, int page) { return page * d / 64 < 32 ? 32 : page * d / 64 > 512 ? 512 : page * d / 64; }
constexpr int kMinExp = -100, kMaxExp = 120;

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the smallest 2^e with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exp(float amax) {
  const int bits = __float_as_int(amax);
  // amax = 1.m * 2^x: e = x - 8, one more when 1.m > 1.75
  const int e = ((bits >> 23) & 255) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// One block writes the new tokens of one page of one head into the key (z = 0)
// or value (z = 1) cache. Every thread holds 8 columns of PASSES rows: the
// rows are read once, their maximum is reduced over the block, and the codes
// are formed from the registers. Bound: HBM, 3 bytes a value; 8192 tokens of 4
// sequences with 8 heads of 128 (ragged, pages of 64) take 30.7 us, 5.4 TB/s: a
// block's bytes are all on their way at once, but its reduction and its stores
// stand behind one another, and the other blocks of its SM fill the gap. One token
// for each of 64 sequences: 5 us, three dependent latencies (length, page number,
// codes and scale).
template <int D, int PAGE>
__global__ void __launch_bounds__(append_threads(D, PAGE)) kv8_append_kernel(const __grid_constant__ Kv8Cache c,
                                                              const __nv_bfloat16* __restrict__ k,
                                                              const __nv_bfloat16* __restrict__ v, int n, int touched,
                                                              uint32_t* status) {
  constexpr int THREADS = append_threads(D, PAGE);
  constexpr int LPR = D / 8;            // threads per row
  constexpr int ROWS = THREADS / LPR;   // rows per pass
  constexpr int PASSES = (PAGE + ROWS - 1) / ROWS;
  const int b = blockIdx.x / touched, t = blockIdx.x - b * touched, h = blockIdx.y, kv = blockIdx.z;
  const int len = __ldg(c.lens + b), count = c.counts ? __ldg(c.counts + b) : n;
  if (count < 0 || count > n || count > len || len > static_cast<long long>(c.max_pages) * PAGE) {
    if (threadIdx.x == 0) record_bad_index(status, WHERE_KV8_APPEND);
    return;
  }
  const int start = len - count;
  const int p = start / PAGE + t;  // page of the sequence
  const int first = max(start, p * PAGE), last = min(len, (p + 1) * PAGE);
  if (first >= last) return;
  const int held = first - p * PAGE, end = last - p * PAGE;  // places [held, end) are written
  const int col = (threadIdx.x % LPR) * 8, row0 = threadIdx.x / LPR;
  const __nv_bfloat16* src =
      (kv ? v : k) + ((static_cast<size_t>(b) * c.Hkv + h) * n + (first - start)) * D + col;
  const int pid = __ldg(c.table + static_cast<size_t>(b) * c.max_pages + p);
  // The rows do not wait for the page's number: two latencies less a block.
  uint4 raw[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int place = row0 + i * ROWS;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (place >= held && place < end)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(place - held) * D));
  }
  if (pid < 0 || pid >= c.num_pages) {
    if (threadIdx.x == 0) record_bad_index(status, WHERE_KV8_APPEND);
    return;
  }
  const size_t slot = static_cast<size_t>(pid) * c.Hkv + h;
  const float s_old = held > 0 ? c.scale[kv][slot] : 0.f;
  uint32_t amax = 0;  // bits of the largest finite |value| (bf16 patterns order as integers)
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
      amax = max(amax, lo < 0x7f80u ? lo : 0u);
      amax = max(amax, hi < 0x7f80u ? hi : 0u);
    }
  }
  __shared__ uint32_t red[THREADS / 32];
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) amax = max(amax, red[i]);
  const int e_new = amax ? scale_exp(__uint_as_float(amax << 16)) : kMinExp;
  const float s = held > 0 ? fmaxf(s_old, exp2i(e_new)) : exp2i(e_new);
  uint8_t* dst = c.code[kv] + slot * PAGE * D + col;
  const float inv = 1.f / s;
  const float ratio = s_old * inv;
  const bool grew = held > 0 && s > s_old;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int place = row0 + i * ROWS;
    uint2* at = reinterpret_cast<uint2*>(dst + static_cast<size_t>(place) * D);
    if (place >= held && place < end) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t two[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f = unpack_bf16x2(w[j]);
        f.x = isinf(f.x) ? NAN : f.x * inv;
        f.y = isinf(f.y) ? NAN : f.y * inv;
        two[j] = f32x2_to_e4m3x2(f.x, f.y);
      }
      *at = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
    } else if (grew && place < held) {
      const uint2 was = *at;
      const uint32_t w[4] = {was.x & 0xffffu, was.x >> 16, was.y & 0xffffu, was.y >> 16};
      uint32_t two[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_to_f32x2(w[j]);
        two[j] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
      }
      *at = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
    }
  }
  if (threadIdx.x == 0) c.scale[kv][slot] = s;
}

// Lengths for an append that refuses no sequence any more: one latency, beside which
// its few bytes do not count.
__global__ void __launch_bounds__(128) kv8_advance_kernel(int* lens, const int* counts, int* taken, int B, int n,
                                                          long long most, uint32_t* status) {
  const int b = blockIdx.x * 128 + threadIdx.x;
  if (b >= B) return;
  const int len = lens[b], count = counts ? counts[b] : n;
  const bool ok = count >= 0 && count <= n && len >= 0 && static_cast<long long>(len) + count <= most;
  if (!ok) record_bad_index(status, WHERE_KV8_APPEND);
  if (ok) lens[b] = len + count;
  taken[b] = ok ? count : 0;
}

// Reads rows [0, min(lens[b], n)) back as bf16 [B][Hkv][n][d]. A thread holds
// 16 columns (16 bytes in, 32 out) of kRows rows, whose loads are issued
// together; a page may end between any two of them. Bound: HBM, 3 bytes a value:
// 4 sequences of 16384 tokens, 8 heads of 128: 68 us, 5.9 TB/s.
constexpr int kRows = 4;

template <int D>
__global__ void __launch_bounds__(kGatherThreads) kv8_gather_kernel(const __grid_constant__ Kv8Cache c,
                                                              __nv_bfloat16* __restrict__ k,
                                                              __nv_bfloat16* __restrict__ v, int n, int tiles,
                                                              uint32_t* status) {
  constexpr int LPR = D / 16, ROWS = kGatherThreads / LPR;
  const int b = blockIdx.x / tiles, tile = blockIdx.x - b * tiles, h = blockIdx.y, kv = blockIdx.z;
  int len = __ldg(c.lens + b);
  const long long most = static_cast<long long>(c.max_pages) << c.page_log2;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) record_bad_index(status, WHERE_KV8_GATHER);
    return;
  }
  len = min(len, n);
  const int row0 = tile * (ROWS * kRows) + threadIdx.x / LPR, col = (threadIdx.x % LPR) * 16;
  const int mask = (1 << c.page_log2) - 1;
  uint4 code[kRows];
  float s[kRows];
  bool ok[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * ROWS;
    ok[i] = row < len;
    if (!ok[i]) continue;
    const int pid = __ldg(c.table + static_cast<size_t>(b) * c.max_pages + (row >> c.page_log2));
    if (pid < 0 || pid >= c.num_pages) {
      record_bad_index(status, WHERE_KV8_GATHER);
      ok[i] = false;
      continue;
    }
    const size_t slot = static_cast<size_t>(pid) * c.Hkv + h;
    s[i] = __ldg(c.scale[kv] + slot);
    code[i] = __ldg(reinterpret_cast<const uint4*>(c.code[kv] + ((slot << c.page_log2) + (row & mask)) * D + col));
  }
  __nv_bfloat16* dst = (kv ? v : k) + (static_cast<size_t>(b) * c.Hkv + h) * n * D + col;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!ok[i]) continue;
    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = e4m3x2_to_f32x2(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
      out[j] = pack_bf16x2(f.x * s[i], f.y * s[i]);
    }
    uint4* at = reinterpret_cast<uint4*>(dst + static_cast<size_t>(row0 + i * ROWS) * D);
    at[0] = make_uint4(out[0], out[1], out[2], out[3]);
    at[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <int D>
cudaError_t launch_append(const Kv8Cache& c, const void* k, const void* v, int n, uint32_t* status,
                          cudaStream_t stream) {
  const int page = 1 << c.page_log2;
  const int touched = (n + page - 2) / page + 1;  // pages that n tokens can touch
  const dim3 grid(static_cast<unsigned>(c.B) * touched, c.Hkv, 2);
  const auto* kk = static_cast<const __nv_bfloat16*>(k);
  const auto* vv = static_cast<const __nv_bfloat16*>(v);
  switch (page) {
    case 16: kv8_append_kernel<D, 16><<<grid, append_threads(D, 16), 0, stream>>>(c, kk, vv, n, touched, status); break;
    case 32: kv8_append_kernel<D, 32><<<grid, append_threads(D, 32), 0, stream>>>(c, kk, vv, n, touched, status); break;
    case 64: kv8_append_kernel<D, 64><<<grid, append_threads(D, 64), 0, stream>>>(c, kk, vv, n, touched, status); break;
    default: kv8_append_kernel<D, 128><<<grid, append_threads(D, 128), 0, stream>>>(c, kk, vv, n, touched, status); break;
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_gather(const Kv8Cache& c, void* k, void* v, int n, uint32_t* status, cudaStream_t stream) {
  constexpr int ROWS = kGatherThreads / (D / 16) * kRows;
  const long long held = static_cast<long long>(c.max_pages) << c.page_log2;
  const int rows = held < n ? static_cast<int>(held) : n;
  const int tiles = (rows + ROWS - 1) / ROWS;
  const dim3 grid(static_cast<unsigned>(c.B) * tiles, c.Hkv, 2);
  kv8_gather_kernel<D><<<grid, kGatherThreads, 0, stream>>>(c, static_cast<__nv_bfloat16*>(k),
                                                      static_cast<__nv_bfloat16*>(v), n, tiles, status);
  return cudaGetLastError();
}

}  // namespace

fa_status_t check_kv8(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                      const int* table, const int* lens, const int* counts, int B, int Hkv, int n, int d, int page,
                      int num_pages, int max_pages, bool* empty, Kv8Cache* c) {
  if (B < 0 || Hkv < 0 || n < 0 || num_pages < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FA_ERR_UNSUPPORTED;
  if (Hkv > 65535) return FA_ERR_INVALID_ARG;
  // block indexes and a sequence's token numbers are int32
  if (n > INT32_MAX - 256 || static_cast<long long>(max_pages) * page > INT32_MAX - 256) return FA_ERR_INVALID_ARG;
  if (static_cast<double>(B) * (static_cast<double>(n) / 16 + 2) >= 2147483648.0) return FA_ERR_INVALID_ARG;
  *empty = B == 0 || Hkv == 0 || n == 0;
  if (*empty) return FA_OK;
  if (num_pages == 0 || max_pages == 0) return FA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !table || !lens) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(counts, 4))
    return FA_ERR_MISALIGNED;
  c->code[0] = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  c->code[1] = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  c->scale[0] = const_cast<float*>(k_scale);
  c->scale[1] = const_cast<float*>(v_scale);
  c->table = table;
  c->lens = lens;
  c->counts = counts;
  c->B = B;
  c->Hkv = Hkv;
  c->page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  c->num_pages = num_pages;
  c->max_pages = max_pages;
  return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status_t fa_kv8_append(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                          const int* page_table, const int* lens, const int* counts, int B, int Hkv, int n, int d,
                          int page, int num_pages, int max_pages, cudaStream_t stream) {
  Kv8Cache c{};
  bool empty = false;
  fa_status_t st = check_kv8(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, B, Hkv, n, d, page,
                             num_pages, max_pages, &empty, &c);
  if (st != FA_OK || empty) return st;
  if (!k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  switch (d) {
    case 64: return from_cuda(launch_append<64>(c, k, v, n, dev.status, stream));
    case 128: return from_cuda(launch_append<128>(c, k, v, n, dev.status, stream));
    default: return from_cuda(launch_append<256>(c, k, v, n, dev.status, stream));
  }
}

fa_status_t fa_kv8_advance(int* lens, const int* counts, int* taken, int B, int n, int page, int max_pages,
                           cudaStream_t stream) {
  if (B < 0 || n < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FA_ERR_UNSUPPORTED;
  const long long most = static_cast<long long>(max_pages) * page;
  if (n > INT32_MAX - 256 || most > INT32_MAX - 256) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!lens || !taken) return FA_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(counts, 4) || !aligned(taken, 4)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  const fa_status_t st = device_info(&dev);
  if (st != FA_OK) return st;
  kv8_advance_kernel<<<(B - 1) / 128 + 1, 128, 0, stream>>>(lens, counts, taken, B, n, most, dev.status);
  return from_cuda(cudaGetLastError());
}

fa_status_t fa_kv8_gather(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                          const int* page_table, const int* lens, void* k, void* v, int B, int Hkv, int n, int d,
                          int page, int num_pages, int max_pages, cudaStream_t stream) {
  Kv8Cache c{};
  bool empty = false;
  fa_status_t st = check_kv8(k_cache, v_cache, k_scale, v_scale, page_table, lens, nullptr, B, Hkv, n, d, page,
                             num_pages, max_pages, &empty, &c);
  if (st != FA_OK || empty) return st;
  if (!k || !v) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  switch (d) {
    case 64: return from_cuda(launch_gather<64>(c, k, v, n, dev.status, stream));
    case 128: return from_cuda(launch_gather<128>(c, k, v, n, dev.status, stream));
    default: return from_cuda(launch_gather<256>(c, k, v, n, dev.status, stream));
  }
}

}  // extern "C"
