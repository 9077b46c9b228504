// Attention of the short sequences of a packed batch (kShortRows rows or fewer),
// for sm_103a.
//
// The tcgen05 kernel's chain of steps per query tile (a load, S, the softmax, the
// second product, O on its way out) takes about 4 us whatever the tile holds, and
// tensor memory has room for two such chains on an SM: 256 sequences of 16 rows
// with 32 heads took it 109 us, their bytes 13. Sequences this short hold too
// little for that tensor core: here a block of four warps takes one sequence and
// one K/V head, K and V (at most 32 KB at d = 128) go to shared memory once for all
// query heads of the group, and each warp takes 16 query rows at a time through
// warp-level products, S and O in registers. Rows are counted through the heads of
// the group, so that a sequence of a few rows fills the products with several
// heads. Four blocks share an SM and hide each other's loads. 256 sequences of 16
// rows, 32 + 8 heads: 31 us (2.7 TB/s); of 64 rows 105 us (3.2 TB/s), between the
// issue of instructions (0.54 of the cycles) and DRAM (0.38); d = 64, 16 heads, 44 us.
// All keys of a row are in one pass: plain softmax, statistics in fp32, the
// weights rounded to bf16 for the second product, the sum from the unrounded ones.
#include <cuda_bf16.h>

#include <algorithm>

#include "fa_internal.h"
#include "fa_packed.cuh"
#include "warp_mma.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLn2 = 0.69314718055994530942f;

template <int HD>
struct ShortCfg {
  static constexpr int UNITS = HD / 8;  // 16-byte units of a row
  static constexpr int TILE = kShortRows * HD * 2;
  static constexpr int WARP_TILE = 16 * HD * 2;
  static constexpr int SMEM = 2 * TILE + kWarps * WARP_TILE;
  static constexpr int PER_SM = HD == 64 ? 5 : (HD == 128 ? 4 : 2);
};

// A batch's rows of one head: base + row * row stride.
__device__ __forceinline__ const __nv_bfloat16* head_rows(const __nv_bfloat16* p, const long long (&st)[2], int row,
                                                          int head) {
  return p + static_cast<long long>(row) * st[0] + head * st[1];
}

template <int HD, bool CAUSAL>
__global__ void __launch_bounds__(32 * kWarps, ShortCfg<HD>::PER_SM)
    packed_short_fwd_kernel(const __grid_constant__ ShortLaunch p) {
  using C = ShortCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sK = smem_u32(smem), sV = sK + C::TILE, sQ = sV + C::TILE + warp * C::WARP_TILE;
  const int n_short = packed_plan_ok(p.plan, p.rows) ? p.plan->n_short : 0;
  const int4* list = packed_tiles(p.plan) + (p.plan->n_tiles - n_short);
  const int group = p.Hq / p.Hkv;
  for (int item = blockIdx.x; item < n_short * p.Hkv; item += gridDim.x) {
    const int e = item / p.Hkv, hk = item - e * p.Hkv;
    const int4 x = __ldg(list + e);
    const int row0 = x.x, n = x.y, n16 = (n + 15) & ~15, R = group * n;
    {
      // a row by UNITS threads, STEP rows at a time
      constexpr int STEP = 32 * kWarps / C::UNITS;
      const int r0 = threadIdx.x / C::UNITS, u = threadIdx.x % C::UNITS;
      const __nv_bfloat16 *kp = head_rows(p.k, p.k_st, row0, hk) + 8 * u, *vp = head_rows(p.v, p.v_st, row0, hk) + 8 * u;
      const __nv_bfloat16 *ks = kp + r0 * p.k_st[0], *vs = vp + r0 * p.v_st[0];
      for (int r = r0; r < n16; r += STEP, ks += STEP * p.k_st[0], vs += STEP * p.v_st[0]) {
        const bool in = r < n;
        cp_async16_or_zero(sK + tile_at<HD>(r, u), in ? ks : kp, in);
        cp_async16_or_zero(sV + tile_at<HD>(r, u), in ? vs : vp, in);
      }
    }
    cp_async_commit();
    const __nv_bfloat16* q = head_rows(p.q, p.q_st, row0, hk * group);
    __nv_bfloat16* o_rows = p.o + static_cast<long long>(row0) * p.o_st[0] + hk * group * p.o_st[1];
    bool waited = false;
    for (int blk = warp; 16 * blk < R || !waited; blk += kWarps) {
      const int first = 16 * blk;
      // Lane i knows row i of the block: 256 times its head in the group, plus its
      // place in the sequence; negative behind the last row.
      const int mine = first + (lane & 15);
      const int place = mine < R ? mine / n * 256 + mine % n : -1;
      constexpr int LPR = C::UNITS < 32 ? C::UNITS : 32, RPI = 32 / LPR;  // a row by LPR lanes
      if (first < R) {
#pragma unroll
        for (int i = 0; i < 16; i += RPI) {
          const int r = i + lane / LPR, at = __shfl_sync(0xffffffffu, place, r);
          const __nv_bfloat16* src = q + (at & 255) * p.q_st[0] + (at >> 8) * p.q_st[1];
#pragma unroll
          for (int u = lane % LPR; u < C::UNITS; u += LPR)
            cp_async16_or_zero(sQ + tile_at<HD>(r, u), (at < 0 ? q : src) + 8 * u, at >= 0);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (!waited) __syncthreads();  // K and V are in
      waited = true;
      __syncwarp();
      if (first >= R) break;

      // the thread's two rows: place in the sequence, keys they see
      int at[2], sees[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        at[i] = __shfl_sync(0xffffffffu, place, (lane >> 2) + 8 * i);
        sees[i] = at[i] < 0 ? 0 : (CAUSAL ? (at[i] & 255) + 1 : n);
      }
      // keys that some row of the block sees
      const int last = __shfl_sync(0xffffffffu, place, min(15, R - 1 - first));
      const bool wraps = last >> 8 != __shfl_sync(0xffffffffu, place, 0) >> 8;
      const int keys = CAUSAL && !wraps ? (last & 255) + 1 : n;

      float s[kShortRows / 16][2][4];
#pragma unroll
      for (int c = 0; c < kShortRows / 16; ++c)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[c][b][i] = 0.f;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        const uint4 a = load_matrices(sQ + tile_at<HD>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
        for (int c = 0; c < kShortRows / 16; ++c)
          if (16 * c < keys) {
            const uint4 b = load_matrices(
                sK + tile_at<HD>(16 * c + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
            mma_bf16(s[c][0], a, b.x, b.y);
            mma_bf16(s[c][1], a, b.z, b.w);
          }
      }
      __syncwarp();  // Q is read: its place takes O
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kShortRows / 16; ++c)
        if (16 * c < keys) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = 16 * c + 8 * b + 2 * (lane & 3) + (i & 1);
              if (col >= sees[i >> 1]) s[c][b][i] = -INFINITY;
              m[i >> 1] = fmaxf(m[i >> 1], s[c][b][i]);
            }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
        m[i] = m[i] == -INFINITY ? 0.f : m[i] * p.scale_log2;
      }
      float o[HD / 8][4];
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
#pragma unroll
      for (int c = 0; c < kShortRows / 16; ++c)
        if (16 * c < keys) {
          float e[2][4];
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[b][i] = ex2_approx(fmaf(s[c][b][i], p.scale_log2, -m[i >> 1]));
              l[i >> 1] += e[b][i];
            }
          const uint4 a = make_uint4(pack_bf16x2(e[0][0], e[0][1]), pack_bf16x2(e[0][2], e[0][3]),
                                     pack_bf16x2(e[1][0], e[1][1]), pack_bf16x2(e[1][2], e[1][3]));
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint4 b = load_matrices_t(
                sV + tile_at<HD>(16 * c + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * j + (lane >> 4)));
            mma_bf16(o[2 * j], a, b.x, b.y);
            mma_bf16(o[2 * j + 1], a, b.z, b.w);
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const int r = (lane >> 2) + 8 * i;
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
          st_shared_b32(sQ + tile_at<HD>(r, j) + 4 * (lane & 3), pack_bf16x2(o[j][2 * i] * inv, o[j][2 * i + 1] * inv));
        if (sees[i] > 0 && (lane & 3) == 0)
          p.lse[static_cast<size_t>(hk * group + (at[i] >> 8)) * p.rows + row0 + (at[i] & 255)] =
              l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; i += RPI) {
        const int r = i + lane / LPR, to = __shfl_sync(0xffffffffu, place, r);
        if (to >= 0) {
          __nv_bfloat16* dst = o_rows + (to & 255) * p.o_st[0] + (to >> 8) * p.o_st[1];
#pragma unroll
          for (int u = lane % LPR; u < C::UNITS; u += LPR)
            *reinterpret_cast<uint4*>(dst + 8 * u) = ld_shared_v4(sQ + tile_at<HD>(r, u));
        }
      }
      __syncwarp();  // O is read before the next rows' Q comes in
    }
    __syncthreads();  // every warp is done with K and V
  }
  // Launched to overlap the kernel for the other sequences: work queued after this
  // one may read what that one writes. One block that waits keeps the grid from
  // ending; the others leave their SMs to the kernels behind.
  if (blockIdx.x == 0 && threadIdx.x == 0) griddep_wait();
}

// ---------------------------------------------------------------------------
// Backward: a block of eight warps takes one sequence and one K/V head, and the
// rows of all its query heads, 64 at a time. S and dP are formed once (the tcgen05
// path forms them twice, for dK, dV and for dQ), P and dS go through shared memory,
// and dK, dV stay in registers until the group's last rows:
//   1. warp (r, h): rows 16 r, keys 32 h: S, dP, P = 2^(S scale log2e - L log2e),
//      dS = P (dP - D) scale, both to shared memory in bf16
//   2. warp (r, 0): dV of keys 16 r += P^T dO;  warp (r, 1): dK += dS^T Q;
//      both: dQ of rows 16 r = dS K, half of the columns each
// D comes from O and dO as they are loaded, so no kernel runs before this one. 256
// sequences of 16 rows, 32 + 8 heads of d = 128: 82 us (the tcgen05 kernels 345); of 64
// rows 325 us, 2.1 TB/s (438): five products from fragments in shared memory, whose
// loads and stores it waits for, at 41% of the issue slots.
// ---------------------------------------------------------------------------
constexpr int kBwdWarps = 8;
constexpr float kLog2e = 1.44269504088896340736f;

template <int HD>
struct ShortBwdCfg {
  static constexpr int UNITS = HD / 8;
  static constexpr int TILE = kShortRows * HD * 2;
  static constexpr int P_TILE = 64 * 64 * 2;
  static constexpr int SMEM = 4 * TILE + 2 * P_TILE + 3 * 64 * 4;
  static constexpr int PER_SM = HD == 256 ? 1 : 2;
};

template <int HD, bool CAUSAL>
__global__ void __launch_bounds__(32 * kBwdWarps, ShortBwdCfg<HD>::PER_SM)
    packed_short_bwd_kernel(const __grid_constant__ ShortLaunch p) {
  griddep_launch_dependents();  // the dQ kernel
  using C = ShortBwdCfg<HD>;
  constexpr int THREADS = 32 * kBwdWarps, STEP = THREADS / C::UNITS;  // a row by UNITS threads, STEP rows at a time
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rq = warp & 3, half = warp >> 2;
  const uint32_t sK = smem_u32(smem), sV = sK + C::TILE, sQ = sV + C::TILE, sO = sQ + C::TILE, sP = sO + C::TILE,
                 sS = sP + C::P_TILE;
  float* sD = reinterpret_cast<float*>(smem + 4 * C::TILE + 2 * C::P_TILE);
  float* sL = sD + 64;
  int* sAt = reinterpret_cast<int*>(sL + 64);  // 256 * head + place of each row, negative behind the last
  const int r0 = threadIdx.x / C::UNITS, u = threadIdx.x % C::UNITS;
  const int n_short = packed_plan_ok(p.plan, p.rows) ? p.plan->n_short : 0;
  const int4* list = packed_tiles(p.plan) + (p.plan->n_tiles - n_short);
  const int group = p.Hq / p.Hkv;
  for (int item = blockIdx.x; item < n_short * p.Hkv; item += gridDim.x) {
    const int e = item / p.Hkv, hk = item - e * p.Hkv;
    const int4 x = __ldg(list + e);
    const int row0 = x.x, n = x.y, n16 = (n + 15) & ~15, R = group * n;
    {
      const __nv_bfloat16 *kp = head_rows(p.k, p.k_st, row0, hk) + 8 * u, *vp = head_rows(p.v, p.v_st, row0, hk) + 8 * u;
      for (int r = r0; r < n16; r += STEP) {
        const bool in = r < n;
        cp_async16_or_zero(sK + tile_at<HD>(r, u), kp + (in ? r : 0) * p.k_st[0], in);
        cp_async16_or_zero(sV + tile_at<HD>(r, u), vp + (in ? r : 0) * p.v_st[0], in);
      }
    }
    const __nv_bfloat16* q = head_rows(p.q, p.q_st, row0, hk * group) + 8 * u;
    const __nv_bfloat16* dO = head_rows(p.dO, p.do_st, row0, hk * group) + 8 * u;
    const __nv_bfloat16* o = head_rows(p.o, p.o_st, row0, hk * group) + 8 * u;
    float acc[HD / 8][4];  // dV or dK of 16 keys
#pragma unroll
    for (int j = 0; j < HD / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

#pragma unroll 1
    for (int base = 0; base < R; base += 64) {
      const int rows = min(64, R - base), rows16 = (rows + 15) & ~15;
      if (threadIdx.x < 64) {
        const int at = base + threadIdx.x;
        sAt[threadIdx.x] = at < R ? at / n * 256 + at % n : -1;
      }
      __syncthreads();
      // this thread's rows: Q and dO on their way to shared memory, its pieces of O
      // and L to registers, all at once
      constexpr int MINE = 64 / STEP;
      uint4 o_piece[MINE];
      float L_mine[MINE];
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int r = r0 + m * STEP;
        o_piece[m] = make_uint4(0u, 0u, 0u, 0u);
        L_mine[m] = 0.f;
        if (r >= rows16) break;
        const int at = sAt[r], head = at >> 8, pos = at & 255;
        const bool in = at >= 0;
        cp_async16_or_zero(sQ + tile_at<HD>(r, u), in ? q + pos * p.q_st[0] + head * p.q_st[1] : q, in);
        cp_async16_or_zero(sO + tile_at<HD>(r, u), in ? dO + pos * p.do_st[0] + head * p.do_st[1] : dO, in);
        if (in) o_piece[m] = __ldg(reinterpret_cast<const uint4*>(o + pos * p.o_st[0] + head * p.o_st[1]));
        if (in && u == 0) L_mine[m] = __ldg(p.lse + static_cast<size_t>(hk * group + head) * p.rows + row0 + pos) * kLog2e;
      }
      cp_async_commit();
      cp_async_wait<0>();
      // D of the rows, from this thread's pieces of O and of dO (which it copied itself)
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int r = r0 + m * STEP;
        if (r >= rows16) break;
        const uint4 a = o_piece[m], b = ld_shared_v4(sO + tile_at<HD>(r, u));
        const uint32_t as[4] = {a.x, a.y, a.z, a.w}, bs[4] = {b.x, b.y, b.z, b.w};
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = unpack_bf16x2(as[i]), z = unpack_bf16x2(bs[i]);
          d = fmaf(y.x, z.x, d);
          d = fmaf(y.y, z.y, d);
        }
#pragma unroll
        for (int s = (C::UNITS < 32 ? C::UNITS : 32) / 2; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
        if (u == 0) {
          sD[r] = d;
          sL[r] = L_mine[m];
        }
      }
      __syncthreads();

      if (16 * rq < rows && 32 * half < n16) {
        float s[2][2][4], dp[2][2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[c][b][i] = dp[c][b][i] = 0.f;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t a_at = tile_at<HD>(16 * rq + (lane & 15), 2 * k + (lane >> 4));
          const uint4 a = load_matrices(sQ + a_at), g = load_matrices(sO + a_at);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (32 * half + 16 * c < n16) {
              const uint32_t b_at =
                  tile_at<HD>(32 * half + 16 * c + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1));
              const uint4 b = load_matrices(sK + b_at), v = load_matrices(sV + b_at);
              mma_bf16(s[c][0], a, b.x, b.y);
              mma_bf16(s[c][1], a, b.z, b.w);
              mma_bf16(dp[c][0], g, v.x, v.y);
              mma_bf16(dp[c][1], g, v.z, v.w);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 16 * rq + (lane >> 2) + 8 * i, at = sAt[r];
          const int sees = at < 0 ? 0 : (CAUSAL ? (at & 255) + 1 : n);
          const float L = sL[r], D = sD[r];
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (32 * half + 16 * c < n16) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float w[2], ds[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int col = 32 * half + 16 * c + 8 * b + 2 * (lane & 3) + z;
                  const bool in = col < sees;
                  w[z] = in ? ex2_approx(fmaf(s[c][b][2 * i + z], p.scale_log2, -L)) : 0.f;
                  ds[z] = in ? w[z] * (dp[c][b][2 * i + z] - D) * p.scale : 0.f;
                }
                const uint32_t to = tile_at<64>(r, 4 * half + 2 * c + b) + 4 * (lane & 3);
                st_shared_b32(sP + to, pack_bf16x2(w[0], w[1]));
                st_shared_b32(sS + to, pack_bf16x2(ds[0], ds[1]));
              }
            }
        }
      }
      __syncthreads();

      if (16 * rq < n16) {
        const uint32_t from = half ? sS : sP, with = half ? sQ : sO;
#pragma unroll 1
        for (int k = 0; k < rows16; k += 16) {
          const uint4 a = load_matrices_t(from + tile_at<64>(k + (lane & 7) + ((lane >> 4) << 3), 2 * rq + ((lane >> 3) & 1)));
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint4 b = load_matrices_t(with + tile_at<HD>(k + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * j + (lane >> 4)));
            mma_bf16(acc[2 * j], a, b.x, b.y);
            mma_bf16(acc[2 * j + 1], a, b.z, b.w);
          }
        }
      }
      float dq[HD / 16][4];
#pragma unroll
      for (int j = 0; j < HD / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[j][i] = 0.f;
      if (16 * rq < rows) {
#pragma unroll 1
        for (int k = 0; k < n16; k += 16) {
          const uint4 a = load_matrices(sS + tile_at<64>(16 * rq + (lane & 15), k / 8 + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < HD / 32; ++j) {
            const uint4 b = load_matrices_t(
                sK + tile_at<HD>(k + (lane & 7) + (((lane >> 3) & 1) << 3), half * (HD / 16) + 2 * j + (lane >> 4)));
            mma_bf16(dq[2 * j], a, b.x, b.y);
            mma_bf16(dq[2 * j + 1], a, b.z, b.w);
          }
        }
      }
      __syncthreads();  // Q is read: its place takes dQ
      if (16 * rq < rows) {
#pragma unroll
        for (int j = 0; j < HD / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            st_shared_b32(sQ + tile_at<HD>(16 * rq + (lane >> 2) + 8 * i, half * (HD / 16) + j) + 4 * (lane & 3),
                          pack_bf16x2(dq[j][2 * i], dq[j][2 * i + 1]));
      }
      __syncthreads();
      for (int r = r0; r < rows; r += STEP) {
        const int at = sAt[r], head = at >> 8, pos = at & 255;
        *reinterpret_cast<uint4*>(p.dq + static_cast<long long>(row0 + pos) * p.dq_st[0] +
                                  (hk * group + head) * p.dq_st[1] + 8 * u) = ld_shared_v4(sQ + tile_at<HD>(r, u));
      }
      __syncthreads();  // before the next rows come in
    }
    if (16 * rq < n16) {
      const uint32_t to = half ? sQ : sO;
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          st_shared_b32(to + tile_at<HD>(16 * rq + (lane >> 2) + 8 * i, j) + 4 * (lane & 3),
                        pack_bf16x2(acc[j][2 * i], acc[j][2 * i + 1]));
    }
    __syncthreads();
    for (int r = r0; r < n; r += STEP) {
      *reinterpret_cast<uint4*>(p.dk + static_cast<long long>(row0 + r) * p.dk_st[0] + hk * p.dk_st[1] + 8 * u) =
          ld_shared_v4(sQ + tile_at<HD>(r, u));
      *reinterpret_cast<uint4*>(p.dv + static_cast<long long>(row0 + r) * p.dv_st[0] + hk * p.dv_st[1] + 8 * u) =
          ld_shared_v4(sO + tile_at<HD>(r, u));
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) griddep_wait();  // as the forward
}

// Queue a kernel so that it takes SMs as the kernel before it leaves them.
template <class Kernel>
cudaError_t launch_beside(Kernel kern, const ShortLaunch& a, int threads, int smem, int per_sm, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
      std::min<long long>(static_cast<long long>(a.rows) * a.Hkv, static_cast<long long>(a.num_sms) * per_sm)));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int HD, bool CAUSAL>
cudaError_t launch_short_fwd(const ShortLaunch& a, cudaStream_t stream) {
  using C = ShortCfg<HD>;
  auto kern = packed_short_fwd_kernel<HD, CAUSAL>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, C::SMEM, a.device, done);
  if (e != cudaSuccess) return e;
  return launch_beside(kern, a, 32 * kWarps, C::SMEM, C::PER_SM, stream);
}

template <int HD, bool CAUSAL>
cudaError_t launch_short_bwd(const ShortLaunch& a, cudaStream_t stream) {
  using C = ShortBwdCfg<HD>;
  auto kern = packed_short_bwd_kernel<HD, CAUSAL>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, C::SMEM, a.device, done);
  if (e != cudaSuccess) return e;
  return launch_beside(kern, a, 32 * kBwdWarps, C::SMEM, C::PER_SM, stream);
}

}  // namespace

cudaError_t launch_fwd_short(const ShortLaunch& a, int d, int causal, cudaStream_t stream) {
  switch (d) {
    case 64: return causal ? launch_short_fwd<64, true>(a, stream) : launch_short_fwd<64, false>(a, stream);
    case 128: return causal ? launch_short_fwd<128, true>(a, stream) : launch_short_fwd<128, false>(a, stream);
    case 256: return causal ? launch_short_fwd<256, true>(a, stream) : launch_short_fwd<256, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_bwd_short(const ShortLaunch& a, int d, int causal, cudaStream_t stream) {
  switch (d) {
    case 64: return causal ? launch_short_bwd<64, true>(a, stream) : launch_short_bwd<64, false>(a, stream);
    case 128: return causal ? launch_short_bwd<128, true>(a, stream) : launch_short_bwd<128, false>(a, stream);
    case 256: return causal ? launch_short_bwd<256, true>(a, stream) : launch_short_bwd<256, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
