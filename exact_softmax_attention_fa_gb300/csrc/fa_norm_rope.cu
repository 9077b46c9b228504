// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, and its gradients (fa_norm_rope_fwd / _bwd of fa.h).
//
//   z = x r w, r = 1/sqrt(mean(x^2) + eps);  y = R(pos) z
//   g = R(pos)^T dy, h = g w, dx = r (h - x r^2 mean(h x)), dw = sum g x r
// The rotation is orthogonal, so the gradient turns back by the same angle.
//
// Both are HBM-bound: a row of d bf16 is read once and written once (the
// backward reads dy and x). One row is held by d / 8 lanes of a warp, 16 bytes
// a lane, so a warp's loads and stores are whole 128-byte lines and the row
// sums are shuffles inside the lane group. A lane group takes kHeads heads of
// one token: their loads are issued together (bytes in flight), and the
// token's cosines and sines are read once for all of them.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;            // heads of one token per lane group
constexpr int kMaxBwdBlocks = 608;   // partial sums of dw: 4 blocks on each of 152 SMs

struct NormRope {
  // t = 0 q, 1 k, 2 v: the strided side (the projection) and the [B][H][N][d] side
  const __nv_bfloat16* x[3];   // strided inputs (backward: q_in, k_in)
  long long xs[3][3];          // batch, head, token strides in elements
  __nv_bfloat16* y[3];         // forward: outputs; backward: unused
  const __nv_bfloat16* dy[3];  // backward: gradients of the outputs
  __nv_bfloat16* dx[3];        // backward: strided outputs
  long long ds[3][3];
  const void* w[2];
  int w_bf16;
  const float* cos_t;
  const float* sin_t;
  const int* positions;
  uint32_t* status;
  float* part;                 // backward: [2][blocks][d] partial dw
  float* dw[2];
  int N, tokens, H[3], chunks[3];  // chunks: lane groups a token needs for q, k, v
  int rot, half, table_rows;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// A lane's place in its group, the columns it holds and what turns them.
template <int D, bool INTER>
struct Lane {
  static constexpr int LPR = D / 8;  // lanes per row
  int j;             // lane within the group: columns 8j .. 8j + 7
  uint32_t mask;     // the group's lanes
  bool turned;       // its columns are rotated
  int partner;       // warp lane holding the other member of each pair (half-split pairs)
  float sign;        // half-split: -1 for the first member (y_a = z_a c - z_b s), +1 for the second
  float c[8], s[8];  // interleaved: entries 0-3

  __device__ __forceinline__ void init(const NormRope& p) {
    const int lane = threadIdx.x & 31;
    j = lane % LPR;
    mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane - j);
    turned = j * 8 < p.rot;
    const bool first = j * 8 < p.half;
    partner = turned ? lane + (first ? p.half / 8 : -(p.half / 8)) : lane;
    sign = first ? -1.f : 1.f;
  }

  __device__ __forceinline__ void load_angles(const NormRope& p, int pos) {
    if (!turned) return;
    const size_t row = static_cast<size_t>(pos) * p.half;
    if (INTER) {
      const float4 a = ldg_f4(p.cos_t + row + j * 4), b = ldg_f4(p.sin_t + row + j * 4);
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
      s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    } else {
      const int i0 = j * 8 < p.half ? j * 8 : j * 8 - p.half;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 a = ldg_f4(p.cos_t + row + i0 + 4 * q), b = ldg_f4(p.sin_t + row + i0 + 4 * q);
        c[4 * q] = a.x, c[4 * q + 1] = a.y, c[4 * q + 2] = a.z, c[4 * q + 3] = a.w;
        s[4 * q] = b.x, s[4 * q + 1] = b.y, s[4 * q + 2] = b.z, s[4 * q + 3] = b.w;
      }
    }
  }

  // z <- R z (BACK: R^T z). Every lane of the group calls it.
  template <bool BACK>
  __device__ __forceinline__ void rotate(const NormRope& p, float (&z)[8]) const {
    if (p.rot == 0) return;
    if (INTER) {
      if (!turned) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = z[2 * i], b = z[2 * i + 1], sn = BACK ? -s[i] : s[i];
        z[2 * i] = a * c[i] - b * sn;
        z[2 * i + 1] = b * c[i] + a * sn;
      }
    } else {
      const float sg = BACK ? -sign : sign;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(mask, z[i], partner);
        if (turned) z[i] = z[i] * c[i] + sg * o * s[i];
      }
    }
  }

  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
  }
};

__device__ __forceinline__ void load_weights(const NormRope& p, int kind, int j, float (&w)[8]) {
  if (p.w_bf16) {
    unpack8(__ldg(static_cast<const uint4*>(p.w[kind]) + j), w);
  } else {
    const float4 a = ldg_f4(static_cast<const float*>(p.w[kind]) + 8 * j);
    const float4 b = ldg_f4(static_cast<const float*>(p.w[kind]) + 8 * j + 4);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

__device__ __forceinline__ int position(const NormRope& p, int token, int n) {
  return p.positions ? __ldg(p.positions + token) : n;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const __grid_constant__ NormRope p) {
  Lane<D, INTER> L;
  L.init(p);
  const int upt = p.chunks[0] + p.chunks[1] + p.chunks[2];
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / L.LPR) + threadIdx.x / L.LPR;
  if (unit >= static_cast<long long>(p.tokens) * upt) return;  // whole lane groups leave
  const int token = static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(upt));
  int ch = static_cast<int>(unit) - token * upt;
  int kind = 0;
  while (ch >= p.chunks[kind]) ch -= p.chunks[kind++];
  const int b = token / p.N, n = token - b * p.N;
  const int h0 = ch * kHeads, nh = min(kHeads, p.H[kind] - h0);
  const __nv_bfloat16* src = p.x[kind] + b * p.xs[kind][0] + h0 * p.xs[kind][1] + n * p.xs[kind][2] + L.j * 8;
  uint4 raw[kHeads];
#pragma unroll
  for (int u = 0; u < kHeads; ++u)
    if (u < nh) raw[u] = __ldg(reinterpret_cast<const uint4*>(src + u * p.xs[kind][1]));
  const size_t head = static_cast<size_t>(b) * p.H[kind] + h0;
  __nv_bfloat16* dst = p.y[kind] + (head * p.N + n) * D + L.j * 8;
  const size_t step = static_cast<size_t>(p.N) * D;
  if (kind == 2) {
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (u < nh) *reinterpret_cast<uint4*>(dst + u * step) = raw[u];
    return;
  }
  if (p.rot > 0) {
    const int pos = position(p, token, n);
    if (pos < 0 || pos >= p.table_rows) {
      if (L.j == 0) record_bad_index(p.status, WHERE_NORM_ROPE);
      return;
    }
    L.load_angles(p, pos);
  }
  const bool norm = p.w[0] != nullptr;
  float w[8];
  if (norm) load_weights(p, kind, L.j, w);
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    if (u >= nh) break;
    float z[8];
    unpack8(raw[u], z);
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(z[i], z[i], ss);
      const float r = rsqrtf(L.sum(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = z[i] * r * w[i];
    }
    L.template rotate<false>(p, z);
    *reinterpret_cast<uint4*>(dst + u * step) = pack8(z);
  }
}

// Persistent: a block walks the q rows, then the k rows, then copies the v
// rows. Each lane sums dw of its 8 columns over the rows it meets; the block's
// lane groups are added in order, and norm_rope_dw_kernel adds the blocks in
// order, so dw does not depend on timing.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRope p) {
  constexpr int GROUPS = kThreads / (D / 8);
  __shared__ float red[GROUPS][D];
  griddep_launch_dependents();
  Lane<D, INTER> L;
  L.init(p);
  const int group = threadIdx.x / L.LPR;
  const bool norm = p.w[0] != nullptr;
  const size_t step = static_cast<size_t>(p.N) * D;
  for (int kind = 0; kind < 3; ++kind) {
    const long long units = static_cast<long long>(p.tokens) * p.chunks[kind];
    float dw[8] = {}, w[8];
    if (norm && kind < 2) load_weights(p, kind, L.j, w);
    for (long long unit = static_cast<long long>(blockIdx.x) * GROUPS + group; unit < units;
         unit += static_cast<long long>(gridDim.x) * GROUPS) {
      const int token = static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(p.chunks[kind]));
      const int ch = static_cast<int>(unit) - token * p.chunks[kind];
      const int b = token / p.N, n = token - b * p.N;
      const int h0 = ch * kHeads, nh = min(kHeads, p.H[kind] - h0);
      const __nv_bfloat16* gy = p.dy[kind] + ((static_cast<size_t>(b) * p.H[kind] + h0) * p.N + n) * D + L.j * 8;
      __nv_bfloat16* out = p.dx[kind] + b * p.ds[kind][0] + h0 * p.ds[kind][1] + n * p.ds[kind][2] + L.j * 8;
      const __nv_bfloat16* src =
          norm && kind < 2 ? p.x[kind] + b * p.xs[kind][0] + h0 * p.xs[kind][1] + n * p.xs[kind][2] + L.j * 8 : nullptr;
      uint4 rg[kHeads], rx[kHeads];
#pragma unroll
      for (int u = 0; u < kHeads; ++u)
        if (u < nh) {
          rg[u] = __ldg(reinterpret_cast<const uint4*>(gy + u * step));
          if (src) rx[u] = __ldg(reinterpret_cast<const uint4*>(src + u * p.xs[kind][1]));
        }
      if (kind == 2) {
#pragma unroll
        for (int u = 0; u < kHeads; ++u)
          if (u < nh) *reinterpret_cast<uint4*>(out + u * p.ds[kind][1]) = rg[u];
        continue;
      }
      if (p.rot > 0) {
        const int pos = position(p, token, n);
        if (pos < 0 || pos >= p.table_rows) {
          if (L.j == 0) record_bad_index(p.status, WHERE_NORM_ROPE_BWD);
          continue;
        }
        L.load_angles(p, pos);
      }
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        if (u >= nh) break;
        float g[8];
        unpack8(rg[u], g);
        L.template rotate<true>(p, g);
        if (norm) {
          float x[8], ss = 0.f, hx = 0.f;
          unpack8(rx[u], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[i], x[i], ss);
            hx = fmaf(g[i] * w[i], x[i], hx);
          }
          const float r = rsqrtf(L.sum(ss) * (1.f / D) + p.eps);
          const float m = L.sum(hx) * (1.f / D) * r * r;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[i] = fmaf(g[i] * r, x[i], dw[i]);
            g[i] = r * (g[i] * w[i] - x[i] * m);
          }
        }
        *reinterpret_cast<uint4*>(out + u * p.ds[kind][1]) = pack8(g);
      }
    }
    if (norm && kind < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) red[group][L.j * 8 + i] = dw[i];
      __syncthreads();
      for (int col = threadIdx.x; col < D; col += kThreads) {
        float t = 0.f;
        for (int g = 0; g < GROUPS; ++g) t += red[g][col];
        p.part[(static_cast<size_t>(kind) * gridDim.x + blockIdx.x) * D + col] = t;
      }
      __syncthreads();
    }
  }
}

// dw[kind][col] = sum over the blocks of their partial sums, in block order
// within each of 8 interleaved runs, in 64 bits. One block per 32 columns.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* __restrict__ part, float* dwq, float* dwk,
                                                           int blocks, int D) {
  __shared__ double red[8][32];
  griddep_wait();  // launched to overlap the pass that writes the partial sums
  const int col = blockIdx.x * 32 + threadIdx.x, kind = blockIdx.y;
  double t = 0.0;
  for (int i = threadIdx.y; i < blocks; i += 8) t += part[(static_cast<size_t>(kind) * blocks + i) * D + col];
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0) {
    for (int i = 1; i < 8; ++i) t += red[i][threadIdx.x];
    (kind ? dwk : dwq)[col] = static_cast<float>(t);
  }
}

template <bool BACK>
cudaError_t launch_norm_rope(const NormRope& a, int d, int interleaved, int blocks, cudaStream_t stream) {
#define FA_NORM_ROPE(D)                                                                        \
  if (d == D) {                                                                                \
    auto kern = BACK ? (interleaved ? norm_rope_bwd_kernel<D, true> : norm_rope_bwd_kernel<D, false>) \
                     : (interleaved ? norm_rope_fwd_kernel<D, true> : norm_rope_fwd_kernel<D, false>); \
    kern<<<blocks, kThreads, 0, stream>>>(a);                                                  \
    return cudaGetLastError();                                                                 \
  }
  FA_NORM_ROPE(64)
  FA_NORM_ROPE(128)
  FA_NORM_ROPE(256)
#undef FA_NORM_ROPE
  return cudaErrorInvalidValue;
}

// Do rows of d elements at these strides stay apart? Sorted by stride, each
// dimension has to step over everything the smaller ones cover.
bool rows_apart(const int (&size)[3], const long long (&stride)[3], int d) {
  int o[3] = {0, 1, 2};
  std::sort(o, o + 3, [&](int a, int b) { return stride[a] < stride[b]; });
  long long span = d;
  for (int i : o) {
    if (size[i] <= 1) continue;
    if (stride[i] < span) return false;
    span += (size[i] - 1) * stride[i];
  }
  return true;
}

// Checks and arguments shared by the two directions.
fa_status_t prepare(const long long* strides, const void* wq, const void* wk, int w_bf16, const float* cos_t,
                    const float* sin_t, int table_rows, const int* positions, int B, int Hq, int Hkv, int N, int d,
                    int rot, int interleaved, float eps, bool with_v, bool* empty, NormRope* a) {
  if (B < 0 || Hq < 0 || Hkv < 0 || N < 0 || table_rows < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (w_bf16 != 0 && w_bf16 != 1)) return FA_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return FA_ERR_INVALID_ARG;
  if (wq && (!std::isfinite(eps) || !(eps > 0.f))) return FA_ERR_INVALID_ARG;
  const double rows = static_cast<double>(B) * N * (static_cast<double>(Hq) + 2.0 * Hkv);
  if (rows >= 2147483648.0) return FA_ERR_INVALID_ARG;
  *empty = rows == 0.0;
  if (*empty) return FA_OK;
  if (rot > 0) {
    if (!cos_t || !sin_t || table_rows == 0 || (!positions && N > table_rows)) return FA_ERR_INVALID_ARG;
    if (!aligned(cos_t, 16) || !aligned(sin_t, 16) || !aligned(positions, 4)) return FA_ERR_MISALIGNED;
  }
  if (!aligned(wq, 16) || !aligned(wk, 16)) return FA_ERR_MISALIGNED;
  if (!strides) return FA_ERR_INVALID_ARG;
  a->w[0] = wq;
  a->w[1] = wk;
  a->w_bf16 = w_bf16;
  a->cos_t = cos_t;
  a->sin_t = sin_t;
  a->positions = positions;
  a->N = N;
  a->tokens = B * N;
  a->H[0] = Hq;
  a->H[1] = Hkv;
  a->H[2] = with_v ? Hkv : 0;
  for (int t = 0; t < 3; ++t) a->chunks[t] = (a->H[t] + kHeads - 1) / kHeads;
  a->rot = rot;
  a->half = rot / 2;
  a->table_rows = table_rows;
  a->eps = eps;
  return FA_OK;
}

// Strides of tensor t as the kernels use them: 0 for a dimension of size 1,
// whose stride a caller may leave at anything.
fa_status_t take_strides(const long long* s, int t, int B, int H, int N, long long (&out)[3]) {
  const int size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    out[i] = size[i] > 1 ? s[3 * t + i] : 0;
    if (out[i] < 0) return FA_ERR_INVALID_ARG;
    if (out[i] % 8 != 0) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

int bwd_blocks(const NormRope& a, int d, int num_sms) {
  const int groups = kThreads / (d / 8);
  const long long most = static_cast<long long>(a.tokens) * std::max(a.chunks[0], std::max(a.chunks[1], a.chunks[2]));
  return static_cast<int>(std::min<long long>((most + groups - 1) / groups, std::min(4 * num_sms, kMaxBwdBlocks)));
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status_t fa_norm_rope_fwd(const void* q_in, const void* k_in, const void* v_in, const long long* strides,
                             const void* wq, const void* wk, int w_bf16, const float* cos_t, const float* sin_t,
                             int table_rows, const int* positions, void* q, void* k, void* v, int B, int Hq, int Hkv,
                             int N, int d, int rot, int interleaved, float eps, cudaStream_t stream) {
  NormRope a{};
  bool empty = false;
  if ((v_in == nullptr) != (v == nullptr)) return FA_ERR_INVALID_ARG;
  fa_status_t st = prepare(strides, wq, wk, w_bf16, cos_t, sin_t, table_rows, positions, B, Hq, Hkv, N, d, rot,
                           interleaved, eps, v != nullptr, &empty, &a);
  if (st != FA_OK || empty) return st;
  const void* in[3] = {q_in, k_in, v_in};
  void* out[3] = {q, k, v};
  for (int t = 0; t < 3; ++t) {
    if (a.H[t] == 0) continue;
    if (!in[t] || !out[t]) return FA_ERR_INVALID_ARG;
    if (!aligned(in[t], 16) || !aligned(out[t], 16)) return FA_ERR_MISALIGNED;
    st = take_strides(strides, t, B, a.H[t], N, a.xs[t]);
    if (st != FA_OK) return st;
    a.x[t] = static_cast<const __nv_bfloat16*>(in[t]);
    a.y[t] = static_cast<__nv_bfloat16*>(out[t]);
  }
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  a.status = dev.status;
  const int groups = kThreads / (d / 8);
  const long long units = static_cast<long long>(a.tokens) * (a.chunks[0] + a.chunks[1] + a.chunks[2]);
  return from_cuda(launch_norm_rope<false>(a, d, interleaved, static_cast<int>((units + groups - 1) / groups), stream));
}

size_t fa_norm_rope_bwd_workspace_size(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq < 0 || Hkv < 0 || Hq + static_cast<long long>(Hkv) == 0 || N <= 0) return 0;
  if (d != 64 && d != 128 && d != 256) return 0;
  return static_cast<size_t>(2) * kMaxBwdBlocks * d * sizeof(float);
}

fa_status_t fa_norm_rope_bwd(const void* dq, const void* dk, const void* dv, const void* q_in, const void* k_in,
                             const long long* strides, const void* wq, const void* wk, int w_bf16, const float* cos_t,
                             const float* sin_t, int table_rows, const int* positions, void* dq_in, void* dk_in,
                             void* dv_in, const long long* out_strides, float* dwq, float* dwk, int B, int Hq, int Hkv,
                             int N, int d, int rot, int interleaved, float eps, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  NormRope a{};
  bool empty = false;
  if ((dv == nullptr) != (dv_in == nullptr)) return FA_ERR_INVALID_ARG;
  fa_status_t st = prepare(wq ? strides : out_strides, wq, wk, w_bf16, cos_t, sin_t, table_rows, positions, B, Hq, Hkv,
                           N, d, rot, interleaved, eps, dv != nullptr, &empty, &a);
  if (st != FA_OK) return st;
  const bool norm = wq != nullptr;
  if (norm) {  // dw of no rows is still written: 0
    if (!dwq || !dwk) return FA_ERR_INVALID_ARG;
    if (!aligned(dwq, 4) || !aligned(dwk, 4)) return FA_ERR_MISALIGNED;
  }
  if (empty && !norm) return FA_OK;
  if (!empty) {
    if (!out_strides) return FA_ERR_INVALID_ARG;
    const void* in[3] = {dq, dk, dv};
    const void* x[2] = {q_in, k_in};
    void* out[3] = {dq_in, dk_in, dv_in};
    for (int t = 0; t < 3; ++t) {
      if (a.H[t] == 0) continue;
      if (!in[t] || !out[t]) return FA_ERR_INVALID_ARG;
      if (!aligned(in[t], 16) || !aligned(out[t], 16)) return FA_ERR_MISALIGNED;
      st = take_strides(out_strides, t, B, a.H[t], N, a.ds[t]);
      if (st != FA_OK) return st;
      if (!rows_apart({B, a.H[t], N}, a.ds[t], d)) return FA_ERR_INVALID_ARG;
      a.dy[t] = static_cast<const __nv_bfloat16*>(in[t]);
      a.dx[t] = static_cast<__nv_bfloat16*>(out[t]);
      if (norm && t < 2) {
        if (!x[t]) return FA_ERR_INVALID_ARG;
        if (!aligned(x[t], 16)) return FA_ERR_MISALIGNED;
        st = take_strides(strides, t, B, a.H[t], N, a.xs[t]);
        if (st != FA_OK) return st;
        a.x[t] = static_cast<const __nv_bfloat16*>(x[t]);
      }
    }
    if (norm) {
      if (!workspace || workspace_bytes < fa_norm_rope_bwd_workspace_size(B, Hq, Hkv, N, d)) return FA_ERR_WORKSPACE;
      if (!aligned(workspace, 256)) return FA_ERR_MISALIGNED;
    }
  }
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  if (empty) {
    cudaError_t e = cudaMemsetAsync(dwq, 0, d * sizeof(float), stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, d * sizeof(float), stream);
    return from_cuda(e);
  }
  a.status = dev.status;
  a.part = static_cast<float*>(workspace);
  const int blocks = bwd_blocks(a, d, dev.num_sms);
  cudaError_t e = launch_norm_rope<true>(a, d, interleaved, blocks, stream);
  if (e != cudaSuccess || !norm) return from_cuda(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d / 32, 2);
  cfg.blockDim = dim3(32, 8);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return from_cuda(cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.part), dwq, dwk, blocks, d));
}

}  // extern "C"
