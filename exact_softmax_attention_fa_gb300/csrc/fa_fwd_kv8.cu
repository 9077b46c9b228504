// Attention over the paged 8-bit cache (fa_fwd_kv8 of fa.h), for few query
// rows per K/V head: decoding and short blocks of new tokens.
//
// Mathematics. With codes k8, v8, page scales sk, sv and c = scale * log2(e):
//   t_j = c sk_j (q . k8_j),  u_j = t_j + log2 sv_j,
//   P_j = 2^(u_j - m),  l = sum_j P_j / sv_j,  O = sum_j P_j v8_j / l,
//   L = ln2 (m + log2 l)
// for any reference m: the value scale rides in the exponent, so the codes are
// multiplied as they are stored and one reference m = max u_j keeps every P_j
// in fp16's range however the pages' scales differ.
//
// Precision. e4m3 codes are exact in fp16. A query row is moved by a power of
// two so that its largest |value| lies in [2^14, 2^15): its bf16 values are then
// exact in fp16 down to 2^-28 of the largest. P_j (0 .. 2^14) is rounded to
// fp16, 2^-11 relative and never coarser than 2^-30 of the row's largest; l
// sums the unrounded values. All sums are fp32.
//
// Bound: HBM, one byte per cached value. Each warp owns a run of consecutive
// 16-key steps of the flattened list of (sequence, K/V head, row chunk) and
// streams them through a ring of its own in shared memory: every lane copies
// (cp.async) exactly the 16-byte pieces it will read back, so the ring needs no
// barrier, has no bank conflicts and keeps (stages - 1) * 32 d bytes per warp
// in flight. Runs are of equal length whatever the sequences' lengths are; a
// row whose keys are shared between warps is joined by kv8_combine_kernel.
//
// Products are m16n8k16 with the cache as the 16-row operand and 8 query rows
// as columns (S^T = K Q^T, O^T = V^T P^T), the shape with the least padding for
// the 1-16 rows of a K/V head that decoding has; the tensor pipe is a small
// share of the time at one byte per value. The order of d within the product
// is free, so a lane's 16 contiguous codes of a key are its fragments as they
// are; V needs pairs of keys side by side, which one byte permute per word
// gives on the way to fp16.
#include <algorithm>
#include <cmath>

#include "fa_kv8.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStepKeys = 16;
constexpr int kMinSteps = 4;      // a warp's share is not cut below this
constexpr int kMaxSms = 152;      // sizes the partials
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;     // growth of a reference (base 2) absorbed without rescaling
constexpr float kShift = 6.f;     // P <= 2^(kShift + kSlack) = 2^14
// l is kept times 2^-10: its terms lie between 2^(6 - 120 - 10) and
// 2^(14 + 100 - 10) for the scales a cache holds, so neither one term nor 2^24
// of them leave fp32's normal range.
constexpr float kSumBias = 10.f;

struct Kv8Attn {
  Kv8Cache c;
  const __nv_bfloat16* q;  // [B][Hq][Nq][d]
  __nv_bfloat16* o;
  float* lse;              // [B][Hq][Nq]
  float* part;             // [2 * warps][part_rows][d] unnormalised O of a run's part of a row
  float2* part_ml;         // [2 * warps][part_rows] its m and l
  uint32_t* status;
  int Hq, Nq, g, rows, chunks, part_rows;  // rows = g * Nq per K/V head, in `chunks` of 8 NT
  int causal;
  float scale_log2;
};

template <int D, int NT>
struct Cfg {
  static constexpr int CTAS = D <= 128 && NT == 1 ? 2 : 1;  // per SM
  static constexpr int STAGE = 32 * D;                      // 16 keys and values
  static constexpr int STAGES = (CTAS == 2 ? 12288 : 24576) / STAGE;
  static constexpr int HEADER = 16;
  static constexpr int WARP_BYTES = STAGES * (STAGE + HEADER);
  static constexpr int SMEM = kWarps * WARP_BYTES;
};

// Tokens of sequence b, or 0 where the stored length is out of range.
__device__ __forceinline__ int seq_len(const Kv8Cache& c, int b) {
  const int len = __ldg(c.lens + b);
  return len < 0 || len > (static_cast<long long>(c.max_pages) << c.page_log2) ? 0 : len;
}
__device__ __forceinline__ int seq_count(const Kv8Cache& c, int b, int n) {
  const int count = c.counts ? __ldg(c.counts + b) : n;
  return count < 0 || count > n ? 0 : count;
}
__device__ __forceinline__ int seq_steps(const Kv8Cache& c, int b) {
  return (seq_len(c, b) + kStepKeys - 1) / kStepKeys;
}

// Every lane: the steps of sequences [0, B) summed, and of those before `b`.
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void step_totals(const Kv8Cache& c, int pairs, int b, long long* total, long long* before) {
  long long t = 0, u = 0;
  for (int i = threadIdx.x & 31; i < c.B; i += 32) {
    const long long s = static_cast<long long>(seq_steps(c, i)) * pairs;
    t += s;
    if (i < b) u += s;
  }
  *total = warp_sum(t);
  *before = warp_sum(u);
}

// Warps that share `total` steps, and the first step of warp w of them.
__device__ __forceinline__ int used_warps(long long total, int warps) {
  const long long most = (total + kMinSteps - 1) / kMinSteps;
  return most < warps ? static_cast<int>(most) : warps;
}
__device__ __forceinline__ long long first_step(long long total, int used, int w) { return total * w / used; }

// A place in the flattened list of steps: (sequence, pair of K/V head and row
// chunk, step of its keys).
struct Cursor {
  int b, pair, s, steps;
  __device__ __forceinline__ void settle(const Kv8Cache& c, int pairs) {
    while (b < c.B && s >= steps) {
      s -= steps;
      if (steps == 0 || ++pair == pairs) {
        pair = 0;
        ++b;
        steps = b < c.B ? seq_steps(c, b) : 0;
      }
    }
  }
};

// The cursor at step x, found by all lanes together.
__device__ Cursor find_cursor(const Kv8Cache& c, int pairs, long long x) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int b = b0 + lane;
    const int steps = b < c.B ? seq_steps(c, b) : 0;
    long long incl = static_cast<long long>(steps) * pairs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > x);
    if (past) {
      const int l = __ffs(past) - 1;
      const int st = __shfl_sync(0xffffffffu, steps, l);
      const long long rem = x - (__shfl_sync(0xffffffffu, incl, l) - static_cast<long long>(st) * pairs);
      const int pair = static_cast<int>(rem / st);
      return Cursor{b0 + l, pair, static_cast<int>(rem - static_cast<long long>(pair) * st), st};
    }
    x -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return Cursor{c.B, 0, 0, 0};
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// D[16][8] += A[16][16] B[16][8], fp16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// x / (l 2^kSumBias) and ln of the row's sum, for sums near either end of
// fp32's range; a row that saw no key has l = 0: O = 0, L = -inf.
struct RowEnd {
  float a, b, lse;
  __device__ __forceinline__ RowEnd(float m, float l) {
    const int e = static_cast<int>(__float_as_uint(l) >> 23 & 255) - 127;  // l >= 0
    a = l == 0.f ? 0.f : 1.f;
    b = 1.f;
    if (l != 0.f && e < 127) {  // not infinite, not NaN
      b = exp2i(-e);
      a = exp2i(-static_cast<int>(kSumBias)) / (l * b);
    } else if (l != 0.f) {
      a = 1.f / l;
    }
    lse = l == 0.f ? -INFINITY : (m + kSumBias + log2f(l)) * kLn2;
  }
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::CTAS) kv8_attn_kernel(const __grid_constant__ Kv8Attn p) {
  using C = Cfg<D, NT>;
  constexpr int KU = D / 64;                  // 16-byte pieces a lane reads of a key
  constexpr int VB = D == 64 ? 8 : 16;        // bytes of a value row per lane and piece
  constexpr int VU = D / (8 * VB);            // such pieces
  constexpr int MT = D / 16;                  // 16-row tiles of O^T
  constexpr int V_AT = 16 * D;                // values' place in a stage
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 2, c4 = lane & 3;
  const int pairs = p.c.Hkv * p.chunks;
  const int warps = gridDim.x * kWarps;
  const int gid = warp * gridDim.x + blockIdx.x;  // few runs spread over the SMs
  long long total, before;
  step_totals(p.c, pairs, 0, &total, &before);
  const int used = used_warps(total, warps);
  if (gid >= used) return;
  const long long x0 = first_step(total, used, gid);
  const int n_steps = static_cast<int>(first_step(total, used, gid + 1) - x0);

  const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
  const uint32_t headers = ring + C::STAGES * C::STAGE;

  // Issue side: lane l looks up step 32 k + l of the run, one batch ahead of
  // the copies (page numbers two batches ahead, as the scales depend on them).
  Cursor cur = find_cursor(p.c, pairs, x0);
  cur.s += lane;
  cur.settle(p.c, pairs);
  struct Meta {
    int slot, s, where;  // slot: page * Hkv + head, -1 for a bad page; where: b * pairs + pair
    float sk, sv;
  };
  auto look_page = [&](Meta& m) {
    m.slot = -2;
    if (cur.b < p.c.B) {
      m.s = cur.s;
      m.where = cur.b * pairs + cur.pair;
      const int pid = __ldg(p.c.table + static_cast<size_t>(cur.b) * p.c.max_pages +
                            (cur.s * kStepKeys >> p.c.page_log2));
      m.slot = pid < 0 || pid >= p.c.num_pages ? -1 : pid * p.c.Hkv + cur.pair / p.chunks;
      cur.s += 32;
      cur.settle(p.c, pairs);
    }
  };
  auto look_scales = [&](Meta& m) {
    m.sk = m.sv = 1.f;
    if (m.slot >= 0) {
      m.sk = __ldg(p.c.scale[0] + m.slot);
      m.sv = __ldg(p.c.scale[1] + m.slot);
    }
  };
  Meta now{}, next{};
  look_page(next);
  int issued = 0;
  auto issue = [&]() {
    if (issued < n_steps) {
      const int l = issued & 31;
      if (l == 0) {
        now = next;
        look_scales(now);
        look_page(next);
      }
      const int slot = __shfl_sync(0xffffffffu, now.slot, l);
      const int s = __shfl_sync(0xffffffffu, now.s, l);
      const bool live = slot >= 0;
      const size_t row = (static_cast<size_t>(live ? slot : 0) << p.c.page_log2) +
                         (s * kStepKeys & ((1 << p.c.page_log2) - 1));
      const uint8_t* kp = p.c.code[0] + row * D;
      const uint8_t* vp = p.c.code[1] + row * D;
      const int st = issued % C::STAGES;
      const uint32_t at = ring + st * C::STAGE;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        cp_async16(at + (2 * u * 32 + lane) * 16, kp + i * D + u * 64 + c4 * 16, live);
        cp_async16(at + ((2 * u + 1) * 32 + lane) * 16, kp + (i + 8) * D + u * 64 + c4 * 16, live);
      }
#pragma unroll
      for (int u = 0; u < VU; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * c4 + (k & 1) + (k >> 1) * 8;
          const uint32_t dst = at + V_AT + ((u * 4 + k) * 32 + lane) * VB;
          const uint8_t* src = vp + key * D + u * 128 + i * VB;
          if constexpr (VB == 16) cp_async16(dst, src, live); else cp_async8(dst, src, live);
        }
      if (lane == l) {
        if (!live) record_bad_index(p.status, WHERE_FWD_KV8);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(headers + st * C::HEADER),
                     "r"(__float_as_uint(now.sk)), "r"(__float_as_uint(now.sv)), "r"(live ? now.s : ~now.s),
                     "r"(now.where)
                     : "memory");
      }
      ++issued;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int k = 0; k < C::STAGES - 1; ++k) issue();

  // Compute side.
  uint32_t qf[NT][KU][8];                     // the row chunk's queries as the B operand
  float acc[NT][MT][4];                       // O^T
  float m[NT][2], l[NT][2], qfac[NT][2];      // columns 2 c4, 2 c4 + 1: reference - kShift, sum, query's power of two
  int limit[NT][2];                           // keys the row sees
  int where = -1, seg_first = 0, seg_last = 0, seg_len = 0, seg_index = -1;

  auto row_place = [&](int w, int r, int* b, int* qi) -> size_t {  // row r of chunk `w`: its place in [B][Hq][Nq]
    *b = w / pairs;
    const int pair = w - *b * pairs, h = pair / p.chunks;
    const int row = (pair - h * p.chunks) * 8 * NT + r;
    *qi = row < p.rows ? row / p.g : INT_MAX;
    return row < p.rows ? (static_cast<size_t>(*b) * p.Hq + h * p.g + row % p.g) * p.Nq + *qi : 0;
  };

  auto begin_rows = [&](int w, int s) {
    where = w;
    seg_first = s;
    ++seg_index;
    int b, qi;
    const int b0 = w / pairs;
    seg_len = seq_len(p.c, b0);
    const int count = seq_count(p.c, b0, p.Nq);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const size_t at = row_place(w, nt * 8 + i, &b, &qi);
      const bool live = qi < count;
      uint4 raw[KU][2];
      uint32_t amax = 0;
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          raw[u][e] = live ? __ldg(reinterpret_cast<const uint4*>(p.q + at * D + u * 64 + c4 * 16) + e)
                           : make_uint4(0, 0, 0, 0);
          const uint32_t w4[4] = {raw[u][e].x, raw[u][e].y, raw[u][e].z, raw[u][e].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) amax = max(amax, max(w4[k] & 0x7fffu, (w4[k] >> 16) & 0x7fffu));
        }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // exponent of the largest value; 2^-100 and below are left as they are
      const int x = max(static_cast<int>(amax >> 7) - 127, -100);
      const float mul = exp2i(14 - x);
#pragma unroll
      for (int u = 0; u < KU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w4[4] = {raw[u][e].x, raw[u][e].y, raw[u][e].z, raw[u][e].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack_bf16x2(w4[k]);
            qf[nt][u][e * 4 + k] = pack_f16x2(f.x * mul, f.y * mul);
          }
        }
      const float fac = exp2i(x - 14);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        qfac[nt][j] = __shfl_sync(0xffffffffu, fac, (2 * c4 + j) * 4);
        row_place(w, nt * 8 + 2 * c4 + j, &b, &qi);
        limit[nt][j] = qi >= count ? 0 : p.causal ? min(seg_len, seg_len - count + qi + 1) : seg_len;
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][t][k] = 0.f;
    }
  };

  // The lane's columns of O^T: 2 consecutive d per 16-row tile.
  auto d_of = [&](int t) { return D == 256 ? (t >> 3) * 128 + i * 16 + 2 * (t & 7) : i * (D / 8) + 2 * t; };

  auto end_rows = [&]() {
    const bool whole = seg_first == 0 && seg_last + 1 == (seg_len + kStepKeys - 1) / kStepKeys;
    const int b0 = where / pairs;
    const int count = seq_count(p.c, b0, p.Nq);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[nt][j];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = nt * 8 + 2 * c4 + j;
        int b, qi;
        const size_t at = row_place(where, r, &b, &qi);
        if (qi >= count) continue;
        if (whole) {
          const RowEnd end(m[nt][j], sum);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            *reinterpret_cast<uint32_t*>(p.o + at * D + d_of(t)) =
                pack_bf16x2(end(acc[nt][t][j]), end(acc[nt][t][2 + j]));
          if (i == 0) p.lse[at] = end.lse;
        } else {
          const size_t slot = (static_cast<size_t>(gid) * 2 + (seg_index > 0)) * p.part_rows + r;
#pragma unroll
          for (int t = 0; t < MT; ++t)
            *reinterpret_cast<float2*>(p.part + slot * D + d_of(t)) = make_float2(acc[nt][t][j], acc[nt][t][2 + j]);
          if (i == 0) p.part_ml[slot] = make_float2(m[nt][j], sum);
        }
      }
  };

#pragma unroll 1
  for (int k = 0; k < n_steps; ++k) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();  // the step's header is written, the last step's has been read
    issue();
    const int st = k % C::STAGES;
    const uint32_t at = ring + st * C::STAGE;
    const uint4 head = ld_shared_v4(headers + st * C::HEADER);
    const bool bad = static_cast<int>(head.z) < 0;
    const int s = bad ? ~static_cast<int>(head.z) : static_cast<int>(head.z);
    if (static_cast<int>(head.w) != where) {
      if (where >= 0) end_rows();
      begin_rows(static_cast<int>(head.w), s);
    }
    seg_last = s;
    const float kf = __uint_as_float(head.x) * p.scale_log2;
    // sv = 2^ev * mant
    const int ev = min(max(static_cast<int>(head.y >> 23 & 255) - 127, -126), 126);
    const float mant = __uint_as_float(head.y) * exp2i(-ev);
    const float inv_sv = exp2i(-static_cast<int>(kSumBias)) / __uint_as_float(head.y);

    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const uint4 ka = ld_shared_v4(at + (2 * u * 32 + lane) * 16);
      const uint4 kb = ld_shared_v4(at + ((2 * u + 1) * 32 + lane) * 16);
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = e4m3x2_to_f16x2(wa[w] & 0xffffu), a2 = e4m3x2_to_f16x2(wa[w] >> 16);
        const uint32_t a1 = e4m3x2_to_f16x2(wb[w] & 0xffffu), a3 = e4m3x2_to_f16x2(wb[w] >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(sc[nt], a0, a1, a2, a3, qf[nt][u][2 * w], qf[nt][u][2 * w + 1]);
      }
    }

    const int key = s * kStepKeys + i;
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool seen = !bad && key + (e >> 1) * 8 < limit[nt][e & 1];
        sc[nt][e] = seen ? fmaf(sc[nt][e] * qfac[nt][e & 1], kf, static_cast<float>(ev)) : -INFINITY;
        grow |= sc[nt][e] > m[nt][e & 1] + (kSlack + kShift);
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = fmaxf(sc[nt][j], sc[nt][2 + j]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) - kShift;
          const float to = fmaxf(m[nt][j], mx);
          const float alpha = to == -INFINITY ? 1.f : ex2_approx(m[nt][j] - to);
          m[nt][j] = to;
          l[nt][j] *= alpha;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            acc[nt][t][j] *= alpha;
            acc[nt][t][2 + j] *= alpha;
          }
        }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
        pr[e] = ex2_approx(sc[nt][e] - ref);
        l[nt][e & 1] = fmaf(pr[e], inv_sv, l[nt][e & 1]);
      }
      pf[nt][0] = transpose8(pack_f16x2(pr[0] * mant, pr[1] * mant));
      pf[nt][1] = transpose8(pack_f16x2(pr[2] * mant, pr[3] * mant));
    }

    const bool tail = (s + 1) * kStepKeys > seg_len;
#pragma unroll
    for (int u = 0; u < VU; ++u) {
      uint32_t v[4][VB / 4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t addr = at + V_AT + ((u * 4 + q) * 32 + lane) * VB;
        if constexpr (VB == 16) {
          const uint4 x = ld_shared_v4(addr);
          v[q][0] = x.x, v[q][1] = x.y, v[q][2] = x.z, v[q][3] = x.w;
        } else {
          const uint2 x = ld_shared_v2(addr);
          v[q][0] = x.x, v[q][1] = x.y;
        }
        // What lies behind the last token may be any bytes, NaN codes among
        // them, and 0 * NaN is not 0.
        if (tail && s * kStepKeys + 2 * c4 + (q & 1) + (q >> 1) * 8 >= seg_len) {
#pragma unroll
          for (int w = 0; w < VB / 4; ++w) v[q][w] = 0;
        }
      }
#pragma unroll
      for (int w = 0; w < VB / 4; ++w) {
        const uint32_t x0_ = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
        const int t = (u * (VB / 4) + w) * 2;
        const uint32_t a0 = e4m3x2_to_f16x2(x0_ & 0xffffu), a1 = e4m3x2_to_f16x2(x0_ >> 16);
        const uint32_t a2 = e4m3x2_to_f16x2(y0 & 0xffffu), a3 = e4m3x2_to_f16x2(y0 >> 16);
        const uint32_t b0 = e4m3x2_to_f16x2(x1 & 0xffffu), b1 = e4m3x2_to_f16x2(x1 >> 16);
        const uint32_t b2 = e4m3x2_to_f16x2(y1 & 0xffffu), b3 = e4m3x2_to_f16x2(y1 >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[nt][t], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          mma_f16(acc[nt][t + 1], b0, b1, b2, b3, pf[nt][0], pf[nt][1]);
        }
      }
    }
  }
  if (where >= 0) end_rows();
  cp_async_wait<0>();
}

// Joins the parts of a query row whose keys several warps shared, and writes
// the rows of sequences without keys. One block per row; a row that one warp
// had whole is already final.
template <int D>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const __grid_constant__ Kv8Attn p, int warps, int per_chunk) {
  constexpr int LANES = D / 4, GROUPS = 128 / LANES;
  __shared__ float4 red[128];
  __shared__ float red_l[GROUPS];
  const int row = blockIdx.x % p.rows;
  const int bh = blockIdx.x / p.rows, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const int qi = row / p.g;
  griddep_wait();  // launched to overlap the kernel that writes the parts
  const bool bad_len = seq_len(p.c, b) != __ldg(p.c.lens + b);
  const bool bad_count = p.c.counts && seq_count(p.c, b, p.Nq) != __ldg(p.c.counts + b);
  if ((bad_len || bad_count) && threadIdx.x == 0) record_bad_index(p.status, WHERE_FWD_KV8);
  if (bad_len || bad_count || qi >= seq_count(p.c, b, p.Nq)) return;
  const int pairs = p.c.Hkv * p.chunks, steps = seq_steps(p.c, b);
  const size_t at = (static_cast<size_t>(b) * p.Hq + h * p.g + row % p.g) * p.Nq + qi;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  if (steps == 0) {
    if (group == 0) *reinterpret_cast<uint2*>(p.o + at * D + lane * 4) = make_uint2(0, 0);
    if (threadIdx.x == 0) p.lse[at] = -INFINITY;
    return;
  }
  long long total, before;
  step_totals(p.c, pairs, b, &total, &before);
  const int used = used_warps(total, warps);
  const int chunk = row / per_chunk, r = row - chunk * per_chunk;
  const long long s0 = before + static_cast<long long>(h * p.chunks + chunk) * steps, s1 = s0 + steps - 1;
  // the warp that holds step x: the largest w with first_step(w) <= x
  const int w0 = static_cast<int>(((s0 + 1) * used - 1) / total), w1 = static_cast<int>(((s1 + 1) * used - 1) / total);
  if (w0 == w1) return;
  auto slot = [&](int w) {
    return (static_cast<size_t>(w) * 2 + (w == w0 && s0 > first_step(total, used, w) ? 1 : 0)) * p.part_rows + r;
  };
  float m = -INFINITY;
  for (int w = w0 + (threadIdx.x & 31); w <= w1; w += 32) m = fmaxf(m, p.part_ml[slot(w)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int w = w0 + group; w <= w1; w += GROUPS) {
    const size_t sl = slot(w);
    const float2 ml = p.part_ml[sl];
    const float wt = ex2_approx(ml.x - ref);
    const float4 x = *reinterpret_cast<const float4*>(p.part + sl * D + lane * 4);
    l = fmaf(wt, ml.y, l);
    a.x = fmaf(wt, x.x, a.x), a.y = fmaf(wt, x.y, a.y), a.z = fmaf(wt, x.z, a.z), a.w = fmaf(wt, x.w, a.w);
  }
  red[threadIdx.x] = a;
  if (lane == 0) red_l[group] = l;
  __syncthreads();
  if (group > 0) return;
  for (int u = 1; u < GROUPS; ++u) {
    const float4 x = red[u * LANES + lane];
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    l += red_l[u];
  }
  const RowEnd end(m, l);
  *reinterpret_cast<uint2*>(p.o + at * D + lane * 4) =
      make_uint2(pack_bf16x2(end(a.x), end(a.y)), pack_bf16x2(end(a.z), end(a.w)));
  if (lane == 0) p.lse[at] = end.lse;
}

int row_tiles(int d, long long rows) { return d <= 128 && rows > 8 ? 2 : 1; }

size_t part_bytes(int d, long long rows, size_t* ml_off) {
  const int nt = row_tiles(d, rows);
  const int ctas = d <= 128 && nt == 1 ? 2 : 1;
  const size_t slots = static_cast<size_t>(2) * kMaxSms * ctas * kWarps * std::min<long long>(rows, 8 * nt);
  *ml_off = slots * d * sizeof(float);
  return *ml_off + slots * sizeof(float2);
}

template <int D, int NT>
cudaError_t launch_t(Kv8Attn& a, int num_sms, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  auto kern = kv8_attn_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // no more blocks than runs that the longest sequences the table allows could have
  const double most = static_cast<double>(a.c.B) * a.c.Hkv * a.chunks *
                      ((static_cast<long long>(a.c.max_pages) << a.c.page_log2) / kStepKeys) / kMinSteps;
  const int full = std::min(num_sms, kMaxSms) * C::CTAS;
  const int grid = most < full ? std::max(1, static_cast<int>(most)) : full;
  kern<<<grid, kThreads, C::SMEM, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.c.B) * a.c.Hkv * a.rows);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_combine_kernel<D>, a, grid * kWarps, 8 * NT);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_kv8_workspace_size(int B, int Hq, int Hkv, int Nq, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Hq % Hkv != 0) return 0;
  if (d != 64 && d != 128 && d != 256) return 0;
  size_t off;
  return part_bytes(d, static_cast<long long>(Hq / Hkv) * Nq, &off);
}

fa_status_t fa_fwd_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int* page_table, const int* lens, const int* counts, void* o,
                       float* lse, int B, int Hq, int Hkv, int Nq, int d, int page, int num_pages, int max_pages,
                       int causal, float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  Kv8Attn a{};
  bool empty = false;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (Hq < 0 || Hkv < 0 || (Hq > 0 && (Hkv == 0 || Hq % Hkv != 0))) return FA_ERR_INVALID_ARG;
  if (Hq == 0 && B >= 0 && Nq >= 0) return FA_OK;
  fa_status_t st = check_kv8(k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, B, Hkv, Nq, d, page,
                             num_pages, max_pages, &empty, &a.c);
  if (st != FA_OK || empty) return st;
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return FA_ERR_MISALIGNED;
  // block indexes, pages of heads and row chunks are int32
  if (static_cast<double>(B) * Hq * Nq >= 2147483648.0 || static_cast<double>(num_pages) * Hkv >= 2147483648.0)
    return FA_ERR_INVALID_ARG;
  size_t ml_off;
  if (!workspace || workspace_bytes < fa_fwd_kv8_workspace_size(B, Hq, Hkv, Nq, d)) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_MISALIGNED;
  DeviceInfo dev;
  st = device_info(&dev);
  if (st != FA_OK) return st;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.status = dev.status;
  a.Hq = Hq;
  a.Nq = Nq;
  a.g = Hq / Hkv;
  a.rows = a.g * Nq;
  const int nt = row_tiles(d, a.rows);
  a.chunks = (a.rows + 8 * nt - 1) / (8 * nt);
  a.part_rows = std::min(a.rows, 8 * nt);
  part_bytes(d, a.rows, &ml_off);
  a.part = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ml_off);
  a.causal = causal;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  if (d == 64) return from_cuda(nt == 1 ? launch_t<64, 1>(a, dev.num_sms, stream) : launch_t<64, 2>(a, dev.num_sms, stream));
  if (d == 128)
    return from_cuda(nt == 1 ? launch_t<128, 1>(a, dev.num_sms, stream) : launch_t<128, 2>(a, dev.num_sms, stream));
  return from_cuda(launch_t<256, 1>(a, dev.num_sms, stream));
}

}  // extern "C"
