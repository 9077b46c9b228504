// Attention over packed sequences of different lengths (fa_packed_plan,
// fa_fwd_packed, fa_bwd_packed of fa.h): the plan, the backward's row
// statistics, the sums of split groups, and the entry points. The products are
// in the attention kernels (fa_fwd_kernel.cuh, fa_bwd*.cu), whose instantiations
// for packed sequences take their work from the plan.
//
// Sequence b is rows cu[b] .. cu[b+1] - 1 of every head. The tensors stay as the
// projection left them: a tensor map per tensor spans all rows of all heads at
// its strides, and a tile's first row is a coordinate. A sequence's last tile
// therefore ends in the next one's rows. Their scores are masked like a key
// tail's; where they stand in the summed dimension of a product, whole steps of
// 16 rows are left out of it and the rest of the last step is cleared in shared
// memory, so that nothing they hold, NaN included, reaches another sequence;
// and the last tile's results leave through plain stores.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// ---------------------------------------------------------------------------
// The plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kBins = 2048;   // of work, most first; longer sequences share bins
constexpr int kOwnTiles = 8;  // a lane lists its own sequence up to this length, the warp a longer one

struct PlanShared {
  int bin[2][kBins];
  int max_tiles, n_short;
  unsigned long long causal, full;
};

// One block: lengths checked, tiles counted by work, and listed from the most
// work to the least. Within one amount of work the order is left to chance; no
// result depends on it.
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const int* __restrict__ cu, int B, int rows,
                                                                   int causal, PackedPlan* plan, int pairs_at,
                                                                   uint32_t* status) {
  __shared__ PlanShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sh.max_tiles = sh.n_short = 0;
    sh.causal = sh.full = 0;
  }
  __syncthreads();
  bool bad = false;
  int most = 0, n_short = 0;
  unsigned long long sum_c = 0, sum_f = 0;
  for (long long b = tid; b < B; b += kPlanThreads) {
    const int from = cu[b], to = cu[b + 1];
    if (from < 0 || to < from || to > rows) {
      bad = true;
      continue;
    }
    const unsigned long long T = (static_cast<unsigned>(to - from) + 127u) >> 7;
    most = max(most, static_cast<int>(T));
    sum_c += T * (T + 1) / 2;
    sum_f += T * T;
    n_short += to > from && to - from <= kShortRows;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      record_bad_index(status, WHERE_PACKED_PLAN);
      *plan = PackedPlan{kPackedMagic, rows, 0, 0, 0, pairs_at, 0, 0, 0, 0, 0};
    }
    return;
  }
  // (one addition a warp: 64-bit ones to shared memory go round until nobody else has
  // come between, which took 1024 threads 50 us)
  most = __reduce_max_sync(0xffffffffu, most);
  n_short = __reduce_add_sync(0xffffffffu, n_short);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum_c += __shfl_xor_sync(0xffffffffu, sum_c, o);
    sum_f += __shfl_xor_sync(0xffffffffu, sum_f, o);
  }
  if (lane == 0 && sum_f) {
    atomicMax(&sh.max_tiles, most);
    atomicAdd(&sh.n_short, n_short);
    atomicAdd(&sh.causal, sum_c);
    atomicAdd(&sh.full, sum_f);
  }
  __syncthreads();
  const int longest = sh.max_tiles;
  int shift = 0;
  while (((longest + (1 << shift) - 1) >> shift) >= kBins) ++shift;
  const int bins = ((longest + (1 << shift) - 1) >> shift) + 1;
  for (int i = tid; i < 2 * bins; i += kPlanThreads) sh.bin[i >= bins][i % bins] = 0;
  __syncthreads();

  // visit(list, first row, length, index, work) for every tile (list 0) and pair of tiles (1)
  auto each = [&](auto visit) {
    // (short sequences, which have lists to themselves, count as no work)
    auto tile = [&](int row0, int n, int T, int i) { visit(0, row0, n, i, n <= kShortRows ? 0 : causal ? i + 1 : T); };
    auto pair = [&](int row0, int n, int T, int w) {
      visit(1, row0, n, w, n <= kShortRows ? 0 : causal ? min(2 * w + 2, T) : T);
    };
    for (long long b0 = 32 * warp; b0 < B; b0 += kPlanThreads) {
      const bool in = b0 + lane < B;
      const int row0 = in ? cu[b0 + lane] : 0, n = in ? cu[b0 + lane + 1] - row0 : 0;
      const int T = (n + 127) >> 7;
      if (T <= kOwnTiles) {
        for (int i = 0; i < T; ++i) tile(row0, n, T, i);
        for (int w = 0; 2 * w < T; ++w) pair(row0, n, T, w);
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, T > kOwnTiles); left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int r = __shfl_sync(0xffffffffu, row0, src), m = __shfl_sync(0xffffffffu, n, src);
        const int TT = (m + 127) >> 7;
        for (int i = lane; i < TT; i += 32) tile(r, m, TT, i);
        for (int w = lane; 2 * w < TT; w += 32) pair(r, m, TT, w);
      }
    }
  };
  each([&](int list, int, int, int, int work) { atomicAdd(&sh.bin[list][(work + (1 << shift) - 1) >> shift], 1); });
  __syncthreads();
  // first place of each bin: what the bins of more work hold
  __shared__ int count[2];
  if (warp < 2) {
    const int per = (bins + 31) / 32;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
      const int at = bins - 1 - (lane * per + i);
      if (at >= 0) mine += sh.bin[warp][at];
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    if (lane == 31) count[warp] = upto;
    int place = upto - mine;
    for (int i = 0; i < per; ++i) {
      const int at = bins - 1 - (lane * per + i);
      if (at < 0) continue;
      const int held = sh.bin[warp][at];
      sh.bin[warp][at] = place;
      place += held;
    }
  }
  __syncthreads();
  int4* list0 = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(plan) + kPackedHead);
  each([&](int list, int row0, int n, int index, int work) {
    const int at = atomicAdd(&sh.bin[list][(work + (1 << shift) - 1) >> shift], 1);
    list0[(list ? pairs_at : 0) + at] = make_int4(row0, n, index, 0);
  });
  if (tid == 0)
    *plan = PackedPlan{kPackedMagic, rows,    count[0],            count[1],            sh.n_short,
                       pairs_at,     longest, B > 0 ? cu[0] : 0,   B > 0 ? cu[B] : 0,   sh.causal,
                       sh.full};
}

// ---------------------------------------------------------------------------
// Backward: row statistics before, sums of split groups after
// ---------------------------------------------------------------------------
struct PackedRows {
  const __nv_bfloat16* o;
  const __nv_bfloat16* dO;
  long long o_st[2], do_st[2];
  const float* lse;
  float *D, *lse2;
  uint32_t* sched;
  const PackedPlan* plan;
  uint32_t* status;
  int rows, Hq, Hkv, d, causal, max_chunks, num_sms;
};

// Into how many chunks the heads of a group are split (see choose_kv_chunks of
// fa_api.cu, whose estimate this is with the batch's own products and longest
// sequence, which only the device knows): the longest item against the work of
// an SM, and the partial sums' bytes.
__device__ int packed_chunks(const PackedRows& a) {
  const int g = a.Hq / a.Hkv;
  const double t_prod = 2.0 * 128 * 128 * a.d / 6.0e12;
  const double pairs = static_cast<double>(a.Hq) * (a.causal ? a.plan->causal_products : a.plan->full_products);
  const double part = 8.0 * a.Hkv * (a.plan->row_end - a.plan->row_begin) * a.d;
  int best = 1;
  double best_t = 1e300;
  for (int c = 1; c <= a.max_chunks; ++c) {
    if (g % c != 0) continue;
    const double work = fmax(4.0 * (g / c) * a.plan->max_tiles, 7.0 * pairs / a.num_sms);
    const double t = work * t_prod + (c > 1 ? 2.0 * c * part / 6.0e12 : 0.0);
    if (t < best_t * 0.98) {
      best_t = t;
      best = c;
    }
  }
  return best;
}

// D = rowsum(dO o O) from the stored bf16, and L * log2(e), of the tiles' rows (the
// short sequences' kernel forms its own): d / 8 lanes a row, kPreRows rows of one
// head at a time. HBM-bound (reads 4 d + 4 bytes a row and head).
constexpr int kPreRows = 4;

template <int HD>
__global__ void __launch_bounds__(256) packed_pre_kernel(const __grid_constant__ PackedRows a) {
  constexpr int LPR = HD / 8, STEP = 256 / LPR, PARTS = 128 / (STEP * kPreRows);
  griddep_launch_dependents();
  const bool ok = packed_plan_ok(a.plan, a.rows);
  if (blockIdx.x == 0) {
    if (threadIdx.x < 4) a.sched[threadIdx.x] = 0u;
    if (threadIdx.x == 0) {
      a.sched[4] = ok ? packed_chunks(a) : 1;
      if (!ok) record_bad_index(a.status, WHERE_PACKED);
    }
  }
  if (!ok) return;
  const int sub = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const long long items = static_cast<long long>(a.plan->n_tiles - a.plan->n_short) * a.Hq * PARTS;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t part = static_cast<uint32_t>(item % PARTS), t = static_cast<uint32_t>(item / PARTS);
    const int4 x = __ldg(packed_tiles(a.plan) + t / a.Hq);
    const int h = t % a.Hq, first = 128 * x.z + part * STEP * kPreRows + r0;
    const __nv_bfloat16* po = a.o + static_cast<long long>(x.x) * a.o_st[0] + h * a.o_st[1] + 8 * sub;
    const __nv_bfloat16* pd = a.dO + static_cast<long long>(x.x) * a.do_st[0] + h * a.do_st[1] + 8 * sub;
    const size_t at = static_cast<size_t>(h) * a.rows + x.x;
    uint4 y[kPreRows], z[kPreRows];
#pragma unroll
    for (int i = 0; i < kPreRows; ++i) {
      const int n = first + i * STEP;
      if (n >= x.y) continue;
      y[i] = __ldg(reinterpret_cast<const uint4*>(po + n * a.o_st[0]));
      z[i] = __ldg(reinterpret_cast<const uint4*>(pd + n * a.do_st[0]));
    }
#pragma unroll
    for (int i = 0; i < kPreRows; ++i) {
      const int n = first + i * STEP;
      const uint32_t* ys = reinterpret_cast<const uint32_t*>(&y[i]);
      const uint32_t* zs = reinterpret_cast<const uint32_t*>(&z[i]);
      float acc = 0.f;
      if (n < x.y) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack_bf16x2(ys[k]), w = unpack_bf16x2(zs[k]);
          acc = fmaf(v.x, w.x, acc);
          acc = fmaf(v.y, w.y, acc);
        }
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if (n < x.y && sub == 0) {
        a.D[at + n] = acc;
        a.lse2[at + n] = a.lse[at + n] * kLog2e;
      }
    }
  }
}

// Where a group was split, dK, dV = bf16 of the sum of the chunks' fp32 partials
// in chunk order (bitwise reproducible): a tile's rows of one head at a time, 8
// elements a thread. (Ordinary loads: this grid is resident while the partials are
// still being written, which the read-only path does not allow.)
__global__ void __launch_bounds__(256) packed_kv_sum_kernel(const __grid_constant__ BwdLaunch p) {
  griddep_wait();
  if (!packed_plan_ok(p.plan, p.N)) return;
  const int chunks = static_cast<int>(p.sched[4]);
  if (chunks == 1) return;
  const int units = p.d / 8, heads = 2 * p.BHkv, items = (p.plan->n_tiles - p.plan->n_short) * heads;
  const size_t len = static_cast<size_t>(p.BHkv) * p.N * p.d;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int4 x = __ldg(packed_tiles(p.plan) + item / heads);
    const int hh = item % heads, first = x.x + 128 * x.z, rows = min(128, x.y - 128 * x.z);
    const bool is_v = hh >= p.BHkv;
    const int h = is_v ? hh - p.BHkv : hh;
    const long long* st = is_v ? p.dv_strides : p.dk_strides;
    for (int i = threadIdx.x; i < rows * units; i += 256) {
      const int row = first + i / units, col = i % units * 8;
      const float* src = p.kv_part + (is_v ? chunks * len : 0) + (static_cast<size_t>(h) * p.N + row) * p.d + col;
      auto part = [&](size_t at) { return *reinterpret_cast<const float4*>(src + at); };
      float4 a = part(0), b = part(4);
      for (int c = 1; c < chunks; ++c) {
        const float4 a2 = part(c * len), b2 = part(c * len + 4);
        a.x += a2.x, a.y += a2.y, a.z += a2.z, a.w += a2.w;
        b.x += b2.x, b.y += b2.y, b.z += b2.z, b.w += b2.w;
      }
      *reinterpret_cast<uint4*>((is_v ? p.dv : p.dk) + row * st[0] + h * st[1] + col) =
          make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
    }
  }
}

// Zeros in the rows that belong to no sequence: a row of a head by d / 8 threads. (A
// plan that was not made for these rows names none, and the call writes nothing.)
struct PackedFill {
  __nv_bfloat16* x[3];
  long long st[3][2];
  int heads[3];
  float* lse;
  const PackedPlan* plan;
  int rows, d;
};

__global__ void __launch_bounds__(256) packed_fill_kernel(const __grid_constant__ PackedFill a) {
  if (!packed_plan_ok(a.plan, a.rows)) return;
  const int begin = a.plan->row_begin, end = a.plan->row_end;
  const int empty = a.rows - (end - begin), units = a.d / 8;
  const int heads = a.heads[0] + a.heads[1] + a.heads[2];
  const long long all = static_cast<long long>(empty) * heads * units, step = static_cast<long long>(gridDim.x) * 256;
  for (long long v = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; v < all; v += step) {
    const int unit = static_cast<int>(v % units);
    const long long r = v / units;
    int h = static_cast<int>(r % heads), t = 0, row = static_cast<int>(r / heads);
    if (row >= begin) row += end - begin;
    if (a.lse && unit == 0) a.lse[static_cast<size_t>(h) * a.rows + row] = 0.f;
    while (h >= a.heads[t]) h -= a.heads[t++];
    *reinterpret_cast<uint4*>(a.x[t] + row * a.st[t][0] + h * a.st[t][1] + 8 * unit) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Entries that a plan has room for: full tiles, and one begun tile (and pair) a
// sequence. Their places are counted in 32 bits.
long long plan_tiles(int B, int rows) { return static_cast<long long>(rows / 128) + std::min(B, rows); }
long long plan_pairs(int B, int rows) { return static_cast<long long>(rows / 256) + std::min(B, rows); }
bool plan_fits(int B, int rows) {
  return B >= 0 && rows >= 0 && plan_tiles(B, rows) + plan_pairs(B, rows) < (1ll << 31);
}

constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Sizes common to the two directions; *empty when there are no rows.
fa_status_t check_packed(int rows, int Hq, int Hkv, int d, int causal, float scale, bool* empty) {
  fa_status_t st = check_common(1, Hq, rows, d, causal, scale, empty);
  if (st == FA_OK) st = check_heads(Hq, Hkv);
  if (st == FA_OK && Hq > 65535) st = FA_ERR_INVALID_ARG;  // a head's number shares a register with a count
  // work items are counted in 32 bits
  if (st == FA_OK && static_cast<long long>(rows) * Hq >= (1ll << 31)) st = FA_ERR_INVALID_ARG;
  return st;
}

// Strides (a row's, a head's) of tensor t: positive multiples of 8 that a tensor
// map takes; 0 for a dimension of size 1, whose stride a caller may leave at anything.
fa_status_t take_rows(const long long* strides, int t, int rows, int heads, const void* p, long long (&out)[2]) {
  if (!p) return FA_ERR_INVALID_ARG;
  if (!aligned(p, 16)) return FA_ERR_MISALIGNED;
  const int size[2] = {rows, heads};
  for (int i = 0; i < 2; ++i) {
    out[i] = size[i] > 1 ? strides[2 * t + i] : 0;
    if (size[i] > 1 && (out[i] <= 0 || out[i] >= (1ll << 38))) return FA_ERR_INVALID_ARG;
    if (out[i] % 8 != 0) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

// fp32 partial dK, dV of one chunk of the groups; how many chunks a workspace is
// made for (a split pays only for short batches, whose partials are small).
size_t part_bytes(int rows, int Hkv, int d) { return static_cast<size_t>(rows) * Hkv * d * 8; }
constexpr size_t kMostPartBytes = 512u << 20;

int chunk_room(int rows, int Hq, int Hkv, int d, size_t room) {
  const int g = Hq / Hkv;
  if (d == 256) return 1;  // as the dense backward at this head dimension
  for (int c = g; c > 1; --c)
    if (g % c == 0 && c * part_bytes(rows, Hkv, d) <= std::min(room, kMostPartBytes)) return c;
  return 1;
}

cudaError_t launch_fill(const PackedFill& f, int num_sms, cudaStream_t stream) {
  const long long all = static_cast<long long>(f.rows) * (f.heads[0] + f.heads[1] + f.heads[2]) * (f.d / 8);
  packed_fill_kernel<<<static_cast<unsigned>(std::min<long long>((all + 255) / 256, 2 * num_sms)), 256, 0, stream>>>(f);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_packed_pre(const PackedRows& a, cudaStream_t stream) {
  // four blocks an SM: the rows on their way at once
  const long long most = static_cast<long long>(a.rows) * a.Hq;
  packed_pre_kernel<HD><<<static_cast<unsigned>(std::min<long long>(most, 4 * a.num_sms)), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_packed_plan_size(int B, int rows) {
  if (!plan_fits(B, rows)) return 0;
  return kPackedHead + static_cast<size_t>(plan_tiles(B, rows) + plan_pairs(B, rows)) * sizeof(int4);
}

fa_status_t fa_packed_plan(const int* cu_seqlens, int B, int rows, int causal, void* plan, size_t plan_bytes,
                           cudaStream_t stream) {
  if (!plan_fits(B, rows) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (B > 0 && !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4)) return FA_ERR_MISALIGNED;
  if (!plan || plan_bytes < fa_packed_plan_size(B, rows)) return FA_ERR_WORKSPACE;
  if (!aligned(plan, 256)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  const fa_status_t st = device_info(&dev);
  if (st != FA_OK) return st;
  packed_plan_kernel<<<1, kPlanThreads, 0, stream>>>(cu_seqlens, B, rows, causal, static_cast<PackedPlan*>(plan),
                                                    static_cast<int>(plan_tiles(B, rows)), dev.status);
  return from_cuda(cudaGetLastError());
}

fa_status_t fa_fwd_packed(const void* q, const void* k, const void* v, const long long* strides, void* o, float* lse,
                          const void* plan, int rows, int Hq, int Hkv, int d, int causal, float scale, int fill,
                          cudaStream_t stream) {
  bool empty = false;
  fa_status_t st = check_packed(rows, Hq, Hkv, d, causal, scale, &empty);
  if (st != FA_OK) return st;
  if (fill != 0 && fill != 1) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (!strides || !lse || !plan) return FA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(plan, 256)) return FA_ERR_MISALIGNED;
  const void* t[4] = {q, k, v, o};
  long long s[4][2];
  for (int i = 0; i < 4; ++i) {
    st = take_rows(strides, i, rows, i == 1 || i == 2 ? Hkv : Hq, t[i], s[i]);
    if (st != FA_OK) return st;
  }
  if (!rows_apart<2>({rows, Hq}, s[3], d)) return FA_ERR_INVALID_ARG;
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  FwdLaunch a{};
  if (!make_rows_map(&a.tmQ, q, rows, Hq, d, s[0], 128) || !make_rows_map(&a.tmK, k, rows, Hkv, d, s[1], 128) ||
      !make_rows_map(&a.tmV, v, rows, Hkv, d, s[2], 128) || !make_rows_map(&a.tmO, o, rows, Hq, d, s[3], 32))
    return FA_ERR_CUDA;
  a.lse = lse;
  a.o = static_cast<__nv_bfloat16*>(o);
  std::copy(s[3], s[3] + 2, a.o_strides);
  a.plan = static_cast<const PackedPlan*>(plan);
  a.Nq = a.Nk = rows;
  a.BH = Hq;
  a.group = Hq / Hkv;
  a.pair_heads = a.group % 2 == 0;
  a.device = dev.device;
  a.pack = 1;
  a.rph = 128;
  a.splits = 1;
  a.d = d;
  a.causal = causal;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  a.status = dev.status;
  a.wait_limit_ns = dev.wait_limit_ns;
  a.num_sms = dev.num_sms;
  a.debug_skip = dev.debug_skip;
  cudaError_t e = launch_fwd_ragged(a, stream);
  ShortLaunch sl{};
  sl.q = static_cast<const __nv_bfloat16*>(q);
  sl.k = static_cast<const __nv_bfloat16*>(k);
  sl.v = static_cast<const __nv_bfloat16*>(v);
  sl.o = a.o;
  sl.lse = lse;
  std::copy(s[0], s[0] + 2, sl.q_st);
  std::copy(s[1], s[1] + 2, sl.k_st);
  std::copy(s[2], s[2] + 2, sl.v_st);
  std::copy(s[3], s[3] + 2, sl.o_st);
  sl.plan = a.plan;
  sl.rows = rows;
  sl.Hq = Hq;
  sl.Hkv = Hkv;
  sl.device = dev.device;
  sl.num_sms = dev.num_sms;
  sl.scale_log2 = a.scale_log2;
  if (e == cudaSuccess) e = launch_fwd_short(sl, d, causal, stream);
  if (e == cudaSuccess && fill) {
    PackedFill f{};
    f.x[0] = a.o;
    std::copy(s[3], s[3] + 2, f.st[0]);
    f.heads[0] = Hq;
    f.lse = lse;
    f.plan = a.plan;
    f.rows = rows;
    f.d = d;
    e = launch_fill(f, dev.num_sms, stream);
  }
  return from_cuda(e);
}

size_t fa_bwd_packed_workspace_size(int rows, int Hq, int Hkv, int d) {
  bool empty = false;
  if (check_packed(rows, Hq, Hkv, d, 0, 1.f, &empty) != FA_OK || empty) return 0;
  const int chunks = chunk_room(rows, Hq, Hkv, d, ~size_t(0));
  return 256 + 2 * up256(static_cast<size_t>(rows) * Hq * 4) + (chunks > 1 ? chunks * part_bytes(rows, Hkv, d) : 0);
}

fa_status_t fa_bwd_packed(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                          const long long* strides, void* dq, void* dk, void* dv, const long long* grad_strides,
                          const void* plan, int rows, int Hq, int Hkv, int d, int causal, float scale, int fill,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  bool empty = false;
  fa_status_t st = check_packed(rows, Hq, Hkv, d, causal, scale, &empty);
  if (st != FA_OK) return st;
  if (fill != 0 && fill != 1) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (!strides || !grad_strides || !lse || !plan) return FA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(plan, 256)) return FA_ERR_MISALIGNED;
  const void* in[5] = {q, k, v, o, dO};
  void* out[3] = {dq, dk, dv};
  long long s[5][2], gs[3][2];
  for (int i = 0; i < 5; ++i) {
    st = take_rows(strides, i, rows, i == 1 || i == 2 ? Hkv : Hq, in[i], s[i]);
    if (st != FA_OK) return st;
  }
  for (int i = 0; i < 3; ++i) {
    const int heads = i == 0 ? Hq : Hkv;
    st = take_rows(grad_strides, i, rows, heads, out[i], gs[i]);
    if (st != FA_OK) return st;
    if (!rows_apart<2>({rows, heads}, gs[i], d)) return FA_ERR_INVALID_ARG;
  }
  const size_t stats = up256(static_cast<size_t>(rows) * Hq * 4), fixed = 256 + 2 * stats;
  if (!workspace || workspace_bytes < fixed) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  BwdLaunch a{};
  const unsigned q_rows = d == 256 ? 64 : 128;  // the d = 256 kernel's query tiles
  if (!make_rows_map(&a.tmQ, q, rows, Hq, d, s[0], q_rows) || !make_rows_map(&a.tmK, k, rows, Hkv, d, s[1], 128) ||
      !make_rows_map(&a.tmV, v, rows, Hkv, d, s[2], 128) || !make_rows_map(&a.tmdO, dO, rows, Hq, d, s[4], q_rows))
    return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.sched = reinterpret_cast<uint32_t*>(ws);
  a.D = reinterpret_cast<float*>(ws + 256);
  a.lse2 = reinterpret_cast<float*>(ws + 256 + stats);
  a.kv_part = reinterpret_cast<float*>(ws + fixed);
  a.lse = lse;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  std::copy(gs[0], gs[0] + 2, a.dq_strides);
  std::copy(gs[1], gs[1] + 2, a.dk_strides);
  std::copy(gs[2], gs[2] + 2, a.dv_strides);
  a.plan = static_cast<const PackedPlan*>(plan);
  a.deterministic = 1;
  a.device = dev.device;
  a.status = dev.status;
  a.N = rows;
  a.BH = Hq;
  a.BHkv = Hkv;
  a.group = Hq / Hkv;
  a.d = d;
  a.causal = causal;
  a.scale = scale;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  a.wait_limit_ns = dev.wait_limit_ns;
  a.num_sms = dev.num_sms;
  a.debug_skip = dev.debug_skip;
  PackedRows r{};
  r.o = static_cast<const __nv_bfloat16*>(o);
  r.dO = static_cast<const __nv_bfloat16*>(dO);
  std::copy(s[3], s[3] + 2, r.o_st);
  std::copy(s[4], s[4] + 2, r.do_st);
  r.lse = lse;
  r.D = a.D;
  r.lse2 = a.lse2;
  r.sched = a.sched;
  r.plan = a.plan;
  r.status = dev.status;
  r.rows = rows;
  r.Hq = Hq;
  r.Hkv = Hkv;
  r.d = d;
  r.causal = causal;
  r.max_chunks = chunk_room(rows, Hq, Hkv, d, workspace_bytes - fixed);
  r.num_sms = dev.num_sms;
  cudaError_t e = d == 64    ? launch_packed_pre<64>(r, stream)
                  : d == 128 ? launch_packed_pre<128>(r, stream)
                             : launch_packed_pre<256>(r, stream);
  if (e == cudaSuccess) e = launch_bwd_main(a, stream);  // dK, dV
  ShortLaunch sl{};
  sl.q = static_cast<const __nv_bfloat16*>(q);
  sl.k = static_cast<const __nv_bfloat16*>(k);
  sl.v = static_cast<const __nv_bfloat16*>(v);
  sl.o = const_cast<__nv_bfloat16*>(r.o);
  sl.dO = r.dO;
  sl.lse = const_cast<float*>(lse);
  sl.dq = a.dq;
  sl.dk = a.dk;
  sl.dv = a.dv;
  long long* to[8] = {sl.q_st, sl.k_st, sl.v_st, sl.o_st, sl.do_st, sl.dq_st, sl.dk_st, sl.dv_st};
  for (int i = 0; i < 8; ++i) std::copy(i < 5 ? s[i] : gs[i - 5], (i < 5 ? s[i] : gs[i - 5]) + 2, to[i]);
  sl.plan = a.plan;
  sl.rows = rows;
  sl.Hq = Hq;
  sl.Hkv = Hkv;
  sl.device = dev.device;
  sl.num_sms = dev.num_sms;
  sl.scale = scale;
  sl.scale_log2 = a.scale_log2;
  // Each of the three starts where the one before leaves SMs: short sequences before
  // dQ, whose items are the larger and handed out one by one (256 sequences of up to
  // 256 rows 856 us, the other way round 880), and a single one of 57 rows beside one
  // of 129 no longer ends behind both (36 -> 26 us, with the blocks that leave early).
  if (e == cudaSuccess) e = launch_bwd_short(sl, d, causal, stream);
  a.overlap_prev = 1;
  if (e == cudaSuccess) e = launch_bwd_dq(a, stream);
  if (e == cudaSuccess && r.max_chunks > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4 * dev.num_sms);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, packed_kv_sum_kernel, a);
  }
  if (e == cudaSuccess && fill) {
    PackedFill f{};
    for (int i = 0; i < 3; ++i) {
      f.x[i] = static_cast<__nv_bfloat16*>(out[i]);
      std::copy(gs[i], gs[i] + 2, f.st[i]);
      f.heads[i] = i == 0 ? Hq : Hkv;
    }
    f.plan = a.plan;
    f.rows = rows;
    f.d = d;
    e = launch_fill(f, dev.num_sms, stream);
  }
  return from_cuda(e);
}

}  // extern "C"
