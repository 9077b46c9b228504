// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, and its gradients (fa_norm_rope_fwd / _bwd of fa.h).
//
//   z = x r w, r = 1/sqrt(mean(x^2) + eps);  y = R(pos) z
//   g = R(pos)^T dy, h = g w, dx = r (h - x r^2 mean(h x)), dw = sum g x r
// The rotation is orthogonal, so the gradient turns back by the same angle.
//
// Both are HBM-bound: a row of d bf16 is read once and written once (the
// backward reads dy and x). One row is held by d / 8 lanes of a warp, as two
// groups of four columns each: for half-split pairs the group and its partner
// half a rotation further, so that a pair is turned inside its lane with one
// sine and cosine for both members, and the row sums are the only shuffles. A
// lane group takes several heads of one token: their loads are issued together
// (bytes in flight), and the token's angles are read once for all of them.
//
// At B = 2, N = 8192, 16 heads for q, k and v, d = 128: forward 65 us, 6.3 TB/s or
// 0.92 of the copy rate; backward 111 us, 4.9 TB/s. The backward holds dy, x and the
// dw of its columns in registers, which leaves 16 warps an SM; it waits for
// loads (more rows on their way, more or fewer warps, and a unit's first rows
// fetched behind the unit before all measured within 2%).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kFwdThreads = 64;      // 256: 69.3, 128: 67.3 instead of 65.0 us (B = 2, N = 8192, 16 heads, d = 128)
constexpr int kThreads = 256;        // backward
constexpr int kHeads = 4;            // heads of one token per lane group, forward
constexpr int kBwdHeads = 8;         // heads of one token per lane group, backward: kBwdSide at a time
constexpr int kBwdSide = 2;
constexpr int kBwdPerSm = 2;         // blocks of the backward on an SM
constexpr int kMaxBwdBlocks = kBwdPerSm * 152;  // partial sums of dw, for q and k each

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
  float* part;                 // backward: partial dw [blocks[0] + blocks[1]][d]
  int blocks[3];               // backward: blocks for q, k and v, in this order
  float* dw[2];
  int N, tokens, H[3], chunks[3];  // chunks: lane groups a token needs for q, k, v
  int rot, half, table_rows;
  float eps;
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Two groups of four columns: pairs 0, 1 and pairs 2, 3 (two columns an operation).
struct Cols {
  float2 f[4];
  __device__ __forceinline__ void unpack(const uint2& a, const uint2& b) {
    f[0] = unpack_bf16x2(a.x), f[1] = unpack_bf16x2(a.y), f[2] = unpack_bf16x2(b.x), f[3] = unpack_bf16x2(b.y);
  }
  __device__ __forceinline__ uint2 pack(int g) const {
    return make_uint2(pack_bf16x2(f[2 * g].x, f[2 * g].y), pack_bf16x2(f[2 * g + 1].x, f[2 * g + 1].y));
  }
};

// A lane's place in its group, the columns it holds and what turns them.
template <int D, bool INTER>
struct Lane {
  static constexpr int LPR = D / 8;  // lanes per row
  uint32_t mask;     // the group's lanes
  int a, b;          // first column of each of its two groups of four
  bool turned;       // its columns are rotated
  int angle;         // first entry of the table's row it needs
  // half-split: cosine and sine of pairs (column a + i, column b + i), i = 0, 1 and 2, 3;
  // interleaved: of pairs (2 i, 2 i + 1) of the eight, i = 0 .. 3
  float2 c[2], s[2];

  __device__ __forceinline__ void init(const NormRope& p) {
    const int lane = threadIdx.x & 31, j = lane % LPR;
    mask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (lane - j);
    turned = 8 * j < p.rot;
    if (INTER || !turned) {  // eight neighbours; rows of rot columns are half-split over lanes 0 .. rot / 8 - 1
      a = 8 * j;
      b = a + 4;
    } else {
      a = 4 * j;
      b = a + p.half;
    }
    angle = 4 * j;
  }

  __device__ __forceinline__ void load_angles(const NormRope& p, int pos) {
    if (!turned) return;
    const size_t at = static_cast<size_t>(pos) * p.half + angle;
    const float4 x = ldg_f4(p.cos_t + at), y = ldg_f4(p.sin_t + at);
    c[0] = make_float2(x.x, x.y), c[1] = make_float2(x.z, x.w);
    s[0] = make_float2(y.x, y.y), s[1] = make_float2(y.z, y.w);
  }

  // z <- R z (BACK: R^T z)
  template <bool BACK>
  __device__ __forceinline__ void rotate(Cols& z) const {
    if (!turned) return;
    const float back = BACK ? -1.f : 1.f;
    if (INTER) {  // (x, y) -> (x, y) c + (-y, x) s
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float cc = i & 1 ? c[i / 2].y : c[i / 2].x, ss = (i & 1 ? s[i / 2].y : s[i / 2].x) * back;
        z.f[i] = fma2(z.f[i], both(cc), fmul2(make_float2(z.f[i].y, z.f[i].x), make_float2(-ss, ss)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = z.f[i], y = z.f[2 + i], ss = make_float2(s[i].x * back, s[i].y * back);
        z.f[i] = fma2(x, c[i], fmul2(y, make_float2(-ss.x, -ss.y)));
        z.f[2 + i] = fma2(y, c[i], fmul2(x, ss));
      }
    }
  }

  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
  }

  __device__ __forceinline__ void load(const __nv_bfloat16* row, uint2 (&x)[2]) const {
    x[0] = __ldg(reinterpret_cast<const uint2*>(row + a));
    x[1] = __ldg(reinterpret_cast<const uint2*>(row + b));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, const uint2& x, const uint2& y) const {
    *reinterpret_cast<uint2*>(row + a) = x;
    *reinterpret_cast<uint2*>(row + b) = y;
  }
  __device__ __forceinline__ void load_weights(const NormRope& p, int kind, float2 (&w)[4]) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int col = g ? b : a;
      if (p.w_bf16) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.w[kind]) + col));
        w[2 * g] = unpack_bf16x2(v.x), w[2 * g + 1] = unpack_bf16x2(v.y);
      } else {
        const float4 v = ldg_f4(static_cast<const float*>(p.w[kind]) + col);
        w[2 * g] = make_float2(v.x, v.y), w[2 * g + 1] = make_float2(v.z, v.w);
      }
    }
  }
};

__device__ __forceinline__ int position(const NormRope& p, int token, int n) {
  return p.positions ? __ldg(p.positions + token) : n;
}

template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kFwdThreads, 16) norm_rope_fwd_kernel(const __grid_constant__ NormRope p) {
  Lane<D, INTER> L;
  L.init(p);
  const int upt = p.chunks[0] + p.chunks[1] + p.chunks[2];
  const long long unit = static_cast<long long>(blockIdx.x) * (kFwdThreads / L.LPR) + threadIdx.x / L.LPR;
  if (unit >= static_cast<long long>(p.tokens) * upt) return;  // whole lane groups leave
  const int token = static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(upt));
  int ch = static_cast<int>(unit) - token * upt;
  int kind = 0;
  while (ch >= p.chunks[kind]) ch -= p.chunks[kind++];
  const int b = token / p.N, n = token - b * p.N;
  const int h0 = ch * kHeads, nh = min(kHeads, p.H[kind] - h0);
  const __nv_bfloat16* src = p.x[kind] + b * p.xs[kind][0] + h0 * p.xs[kind][1] + n * p.xs[kind][2];
  uint2 raw[kHeads][2];
#pragma unroll
  for (int u = 0; u < kHeads; ++u)
    if (u < nh) L.load(src + u * p.xs[kind][1], raw[u]);
  const size_t head = static_cast<size_t>(b) * p.H[kind] + h0;
  __nv_bfloat16* dst = p.y[kind] + (head * p.N + n) * D;
  const size_t step = static_cast<size_t>(p.N) * D;
  if (kind == 2) {
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (u < nh) L.store(dst + u * step, raw[u][0], raw[u][1]);
    return;
  }
  if (p.rot > 0) {
    const int pos = position(p, token, n);
    if (pos < 0 || pos >= p.table_rows) {
      if (L.angle == 0) record_bad_index(p.status, WHERE_NORM_ROPE);
      return;
    }
    L.load_angles(p, pos);
  }
  float2 w[4];
  if (NORM) L.load_weights(p, kind, w);
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    if (u >= nh) break;
    Cols z;
    z.unpack(raw[u][0], raw[u][1]);
    if (NORM) {
      float2 ss = fmul2(z.f[0], z.f[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) ss = fma2(z.f[i], z.f[i], ss);
      const float r = rsqrtf(L.sum(ss.x + ss.y) * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 4; ++i) z.f[i] = fmul2(fmul2(z.f[i], both(r)), w[i]);
    }
    L.template rotate<false>(z);
    L.store(dst + u * step, z.pack(0), z.pack(1));
  }
}

// Persistent: the blocks are shared out over q, k and v by their work, and a
// lane group takes up to kBwdHeads heads of one token, two at a time with the
// next two on their way. Each lane sums dw of its 8 columns over the rows it
// meets; the block's lane groups are added in order, and norm_rope_dw_kernel
// adds the blocks in order, so dw does not depend on timing.
template <int D, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, kBwdPerSm) norm_rope_bwd_kernel(const __grid_constant__ NormRope p) {
  constexpr int GROUPS = kThreads / (D / 8), SIDE = kBwdSide;
  __shared__ float red[GROUPS][D];
  griddep_launch_dependents();
  Lane<D, INTER> L;
  L.init(p);
  const int group = threadIdx.x / L.LPR;
  int block = blockIdx.x, kind = 0;
  while (block >= p.blocks[kind]) block -= p.blocks[kind++];
  const int chunks = p.chunks[kind], heads = p.H[kind], n_blocks = p.blocks[kind];
  const long long units = static_cast<long long>(p.tokens) * chunks;
  const long long step = static_cast<long long>(p.N) * D, x_step = p.xs[kind][1], d_step = p.ds[kind][1];
  const bool norm = NORM && kind < 2;
  float2 dw[4], w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = make_float2(0.f, 0.f);
  if (norm) L.load_weights(p, kind, w);
#pragma unroll 1
  for (long long unit = static_cast<long long>(block) * GROUPS + group; unit < units;
       unit += static_cast<long long>(n_blocks) * GROUPS) {
    const int token = static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(chunks));
    const int h0 = (static_cast<int>(unit) - token * chunks) * kBwdHeads, nh = min(kBwdHeads, heads - h0);
    const int b = token / p.N, n = token - b * p.N;
    const __nv_bfloat16* gy = p.dy[kind] + (static_cast<size_t>(b) * heads + h0) * step + static_cast<size_t>(n) * D;
    const __nv_bfloat16* src = norm ? p.x[kind] + b * p.xs[kind][0] + h0 * x_step + n * p.xs[kind][2] : nullptr;
    __nv_bfloat16* out = p.dx[kind] + b * p.ds[kind][0] + h0 * d_step + n * p.ds[kind][2];
    uint2 g_raw[SIDE][2], x_raw[SIDE][2];
    auto fetch = [&](int h) {
#pragma unroll
      for (int u = 0; u < SIDE; ++u)
        if (h + u < nh) {
          L.load(gy + (h + u) * step, g_raw[u]);
          if (norm) L.load(src + (h + u) * x_step, x_raw[u]);
        }
    };
    fetch(0);
    if (kind < 2 && p.rot > 0) {
      const int pos = position(p, token, n);
      if (pos < 0 || pos >= p.table_rows) {
        if (L.angle == 0) record_bad_index(p.status, WHERE_NORM_ROPE_BWD);
        continue;
      }
      L.load_angles(p, pos);
    }
#pragma unroll 1
    for (int h = 0; h < nh; h += SIDE) {
      uint2 g_now[SIDE][2], x_now[SIDE][2];
#pragma unroll
      for (int u = 0; u < SIDE; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          g_now[u][e] = g_raw[u][e];
          if (norm) x_now[u][e] = x_raw[u][e];
        }
      fetch(h + SIDE);
#pragma unroll
      for (int u = 0; u < SIDE; ++u) {
        if (h + u >= nh) break;
        __nv_bfloat16* row = out + (h + u) * d_step;
        if (kind == 2) {
          L.store(row, g_now[u][0], g_now[u][1]);
          continue;
        }
        Cols g;
        g.unpack(g_now[u][0], g_now[u][1]);
        L.template rotate<true>(g);
        if (NORM) {
          Cols x, gw;
          x.unpack(x_now[u][0], x_now[u][1]);
          float2 ss = fmul2(x.f[0], x.f[0]), hx = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i > 0) ss = fma2(x.f[i], x.f[i], ss);
            gw.f[i] = fmul2(g.f[i], w[i]);
            hx = fma2(gw.f[i], x.f[i], hx);
          }
          const float r = rsqrtf(L.sum(ss.x + ss.y) * (1.f / D) + p.eps);
          const float m = -L.sum(hx.x + hx.y) * (1.f / D) * r * r * r;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dw[i] = fma2(fmul2(g.f[i], both(r)), x.f[i], dw[i]);
            g.f[i] = fma2(gw.f[i], both(r), fmul2(x.f[i], both(m)));
          }
        }
        L.store(row, g.pack(0), g.pack(1));
      }
    }
  }
  if (norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float2*>(&red[group][(i < 2 ? L.a : L.b - 4) + 2 * i]) = dw[i];
    __syncthreads();
    for (int col = threadIdx.x; col < D; col += kThreads) {
      float t = 0.f;
      for (int g = 0; g < GROUPS; ++g) t += red[g][col];
      p.part[static_cast<size_t>(blockIdx.x) * D + col] = t;
    }
  }
}

// dw[kind][col] = sum over the blocks of their partial sums, in 32 interleaved
// runs of them in block order, in 64 bits. One block per 32 columns.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, float* dwq, float* dwk,
                                                            int q_blocks, int k_blocks, int D) {
  __shared__ double red[32][32];
  griddep_wait();  // launched to overlap the pass that writes the partial sums
  const int col = blockIdx.x * 32 + threadIdx.x, kind = blockIdx.y;
  const int begin = kind ? q_blocks : 0, end = kind ? q_blocks + k_blocks : q_blocks;
  double t = 0.0;
#pragma unroll 4
  for (int i = begin + threadIdx.y; i < end; i += 32) t += part[static_cast<size_t>(i) * D + col];
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0) {
    for (int i = 1; i < 32; ++i) t += red[i][threadIdx.x];
    (kind ? dwk : dwq)[col] = static_cast<float>(t);
  }
}

template <bool BACK>
cudaError_t launch_norm_rope(const NormRope& a, int d, int interleaved, int blocks, cudaStream_t stream) {
#define FA_NORM_ROPE_KERNEL(D, I, N) (BACK ? norm_rope_bwd_kernel<D, I, N> : norm_rope_fwd_kernel<D, I, N>)
#define FA_NORM_ROPE(D)                                                                                     \
  if (d == D) {                                                                                             \
    auto kern = a.w[0] ? (interleaved ? FA_NORM_ROPE_KERNEL(D, true, true) : FA_NORM_ROPE_KERNEL(D, false, true)) \
                       : (interleaved ? FA_NORM_ROPE_KERNEL(D, true, false) : FA_NORM_ROPE_KERNEL(D, false, false)); \
    kern<<<blocks, BACK ? kThreads : kFwdThreads, 0, stream>>>(a);                                          \
    return cudaGetLastError();                                                                              \
  }
  FA_NORM_ROPE(64)
  FA_NORM_ROPE(128)
  FA_NORM_ROPE(256)
#undef FA_NORM_ROPE
#undef FA_NORM_ROPE_KERNEL
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
                    int rot, int interleaved, float eps, bool with_v, int heads, bool* empty, NormRope* a) {
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
  for (int t = 0; t < 3; ++t) a->chunks[t] = (a->H[t] + heads - 1) / heads;
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

// Blocks for q, k and v: all that fit the device at once, by the bytes each
// moves (q and k three rows a head with weights, else two; v's two then count 2.2,
// its blocks else end 7 us behind the others of a 113 us call), no more than
// there are lane groups to fill. A kind without rows has none.
void share_blocks(NormRope* a, int d, int num_sms) {
  const int groups = kThreads / (d / 8), all = std::min(kBwdPerSm * num_sms, kMaxBwdBlocks);
  double work[3], sum = 0.0;
  for (int t = 0; t < 3; ++t) sum += work[t] = a->H[t] * (!a->w[0] ? 2.0 : t < 2 ? 3.0 : 2.2);
  for (int t = 0; t < 3; ++t) {
    const long long most = (static_cast<long long>(a->tokens) * a->chunks[t] + groups - 1) / groups;
    a->blocks[t] = static_cast<int>(std::min<long long>(most, std::max(1, static_cast<int>(all * work[t] / sum))));
  }
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
                           interleaved, eps, v != nullptr, kHeads, &empty, &a);
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
  const int groups = kFwdThreads / (d / 8);
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
                           N, d, rot, interleaved, eps, dv != nullptr, kBwdHeads, &empty, &a);
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
  share_blocks(&a, d, dev.num_sms);
  cudaError_t e = launch_norm_rope<true>(a, d, interleaved, a.blocks[0] + a.blocks[1] + a.blocks[2], stream);
  if (e != cudaSuccess || !norm) return from_cuda(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d / 32, 2);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return from_cuda(cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.part), dwq, dwk,
                                      a.blocks[0], a.blocks[1], d));
}

}  // extern "C"
