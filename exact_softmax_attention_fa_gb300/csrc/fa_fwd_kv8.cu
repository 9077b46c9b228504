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
// Products. The codes are the tensor core's operands as they are stored (e4m3,
// fp32 sums: measured within 2^-23 of the sum of absolute products); what is
// multiplied with them is split into e4m3 pieces that occupy columns of their
// own, since a decoding call leaves most of an MMA's 8 columns empty anyway:
//   a query value q 2^a (row maximum in [2^7, 2^8)) = qh + 2^-4 ql, exact down to
//   2^-13 of the row's largest value, and within 2^-21 of it below;
//   P (at most 448), rounded to fp16, = ph + 2^-4 pm + 2^-8 pl: 2^-11 relative, and
//   never coarser than 2^-24 of the row's largest weight (fp16 so that the pieces
//   are taken two at a time; l sums the unrounded weights).
// (Converting the codes to fp16 for m16n8k16 products was measured first: 519
// instructions per 16 keys at d = 128, most of them unpacking bytes, and 0.61 of
// the HBM rate at B = 8, Hkv = 8, 32768 keys. The counters show an e4m3 product
// as two fp16 ones and unpacking on the ALU, 27% and 37% of those pipes there.)
//
// Bound: HBM, one byte per cached value. Each warp owns a run of consecutive
// 32-key steps of the flattened list of (sequence, K/V head, row chunk) and
// streams them (cp.async, 16 keys of a page are 16 d contiguous bytes) through a
// ring of its own in shared memory, so no warp waits for another and
// (stages - 1) * 64 d bytes per warp are in flight. Runs are of equal length
// whatever the sequences' lengths are; a row whose keys are shared between
// warps is joined by kv8_combine_kernel. Measured: B = 8, 32 heads on 8, 32768 keys,
// d = 128, pages of 64: 90 us, 6.0 TB/s; B = 16, 32 heads, ragged up to 8192 keys,
// d = 64, pages of 32: 55 us, 5.1 TB/s (a step of d = 64 has half the bytes
// for the same instructions); one sequence of 1000 keys: 9.6 us, two launches and
// the walk length, page number, codes.
//
// Products are m16n8k32 with the cache as the 16-row operand and the rows'
// pieces as columns (S^T = K Q^T, O^T = V^T P^T). A matrix load gives K's
// fragments as they are. V is loaded transposed in 16-bit units, which leaves
// two adjacent columns of a key together; one byte permute a word parts them.
#include <algorithm>
#include <cmath>

#include "fa_kv8_attn.cuh"

namespace fa {
namespace {

constexpr int kStepKeys = 32;
constexpr int kHalfKeys = 16;     // a page ends at a multiple of this
constexpr int kMinSteps = 2;      // a warp's share is not cut below this
constexpr float kSlack = 2.8f;    // growth of a reference (base 2) absorbed: P <= 2^(kShift + kSlack) < 448

struct Kv8Attn : Kv8Call {
  float* part;     // [2 * warps][part_rows][d] unnormalised O of a run's part of a row
  float2* part_ml; // [2 * warps][part_rows] its m and l
  uint32_t* status;
  int rows, chunks, part_rows;  // rows = g * Nq per K/V head, in `chunks` of 4 NQ
};

// Warps of a CTA, one CTA per SM; their stages fill its shared memory. More warps
// hide more of a step's instructions, fewer leave fewer parts to join: at d = 64
// 12 of four stages instead of 16 of three take 55 instead of 54 us for the ragged
// batch above and 16 instead of 20 for one sequence of 19098 keys and 16 heads; at
// d = 128 6 of four instead of 8 of three take 95 instead of 89 for the long one.
constexpr int warps_per_cta(int d) { return d == 64 ? 12 : 1024 / d; }

// NQ: 8-column tiles of queries, 4 rows of two pieces each.
template <int D, int NQ>
struct Cfg {
  static constexpr int WARPS = warps_per_cta(D);
  static constexpr int STAGE = 2 * kStepKeys * D;
  static constexpr int STAGES = D == 64 ? 4 : 3;
  static constexpr int TABLE = 2 * 32 * 16;    // two batches of half steps: what look_up and the scales gave
  static constexpr int WARP_BYTES = STAGES * STAGE + TABLE;
  static constexpr int SMEM = WARPS * WARP_BYTES;
  // Registers a thread. At d = 128 with one column tile 232 leave the SM 6144, in which a block
  // of the joining kernel waits for its parts: with 240 four sequences of 3000 keys and 16 heads
  // take 15.3 instead of 11.5 us.
  static constexpr int REGS = D == 64 ? 168 : (D == 128 && NQ == 1 ? 232 : 255);
};

__device__ __forceinline__ int steps_of(int len) { return (len + kStepKeys - 1) / kStepKeys; }
__device__ __forceinline__ int seq_steps(const Kv8Cache& c, int b) { return steps_of(seq_len(c, b)); }

// Every lane: the steps of all sequences summed, and of those before `b`; how
// many sequences have any.
__device__ __forceinline__ void step_totals(const Kv8Cache& c, int pairs, int b, long long* total, long long* before,
                                            int* live) {
  long long t = 0, u = 0;
  int n = 0;
  for (int i = threadIdx.x & 31; i < c.B; i += 32) {
    const int one = seq_steps(c, i);
    const long long s = static_cast<long long>(one) * pairs;
    t += s;
    if (i < b) u += s;
    n += one > 0;
  }
  *total = warp_sum(t);
  *before = warp_sum(u);
  *live = __reduce_add_sync(0xffffffffu, n);
}

// Warps that share `total` steps of `pieces` row chunks (a chunk's start and end
// cost several steps: the shortest get a warp each, 13 sequences of two keys at
// d = 256 11.5 instead of 18.5 us), and the first step of warp w.
__device__ __forceinline__ int used_warps(long long total, long long pieces, int warps) {
  const long long most = max((total + kMinSteps - 1) / kMinSteps, min(total, pieces));
  return most < warps ? static_cast<int>(most) : warps;
}
__device__ __forceinline__ long long first_step(long long total, int used, int w) { return total * w / used; }

// A place in the flattened list of steps: (sequence, pair of K/V head and row
// chunk, step of its keys).
struct Cursor {
  int b, pair, s, len;
  __device__ __forceinline__ void settle(const Kv8Cache& c, int pairs) {
    while (b < c.B && s >= steps_of(len)) {
      s -= steps_of(len);
      if (len == 0 || ++pair == pairs) {
        pair = 0;
        ++b;
        len = b < c.B ? seq_len(c, b) : 0;
      }
    }
  }
};

// The cursor at step x, found by all lanes together.
__device__ Cursor find_cursor(const Kv8Cache& c, int pairs, long long x) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int b = b0 + lane;
    const int len = b < c.B ? seq_len(c, b) : 0;
    long long incl = static_cast<long long>(steps_of(len)) * pairs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > x);
    if (past) {
      const int l = __ffs(past) - 1;
      const int len_l = __shfl_sync(0xffffffffu, len, l), st = steps_of(len_l);
      const long long rem = x - (__shfl_sync(0xffffffffu, incl, l) - static_cast<long long>(st) * pairs);
      const int pair = static_cast<int>(rem / st);
      return Cursor{b0 + l, pair, static_cast<int>(rem - static_cast<long long>(pair) * st), len_l};
    }
    x -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return Cursor{c.B, 0, 0, 0};
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// Four 8 x 8 matrices of 16-bit values; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ uint4 ldmatrix4(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 ldmatrix4_trans(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// D[16][8] += A[16][32] B[32][8], e4m3 in, fp32 sums.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// The next e4m3 piece of two fp16 values: v <- 16 times what it leaves of them
// (exact: the piece and the rest together hold the value's 11 bits).
__device__ __forceinline__ uint32_t take_piece(__half2& v) {
  const uint32_t two = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&v));
  const uint32_t back = e4m3x2_to_f16x2(two);
  v = __hmul2(__hsub2(v, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(16.f));
  return two;
}
__device__ __forceinline__ uint32_t last_piece(const __half2& v) {
  return f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&v));
}

template <int D, int NQ>
__global__ void __maxnreg__((Cfg<D, NQ>::REGS)) kv8_attn_kernel(const __grid_constant__ Kv8Attn p) {
  using C = Cfg<D, NQ>;
  constexpr int MT = D / 16;                  // 16-byte column blocks; 16-row tiles of O^T
  constexpr int V_AT = kStepKeys * D;         // values' place in a stage
  constexpr int ROWS = 4 * NQ;
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane >> 2, c4 = lane & 3;
  const int pairs = p.c.Hkv * p.chunks;
  const int warps = gridDim.x * C::WARPS;
  const int gid = warp * gridDim.x + blockIdx.x;  // few runs spread over the SMs
  long long total, before;
  int live;
  step_totals(p.c, pairs, 0, &total, &before, &live);
  const int used = used_warps(total, static_cast<long long>(live) * pairs, warps);
  if (gid >= used) return;
  const long long x0 = first_step(total, used, gid);
  const int n_steps = static_cast<int>(first_step(total, used, gid + 1) - x0);

  const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
  const uint32_t table = ring + C::STAGES * C::STAGE;

  // Issue side: lane 2 j + h looks up half h of step 16 k + j of the run, its
  // page one batch of 16 steps ahead of the copies, its scales with the batch's
  // first copy; they go to the table when that step's data has come.
  Cursor cur = find_cursor(p.c, pairs, x0);
  cur.s += lane >> 1;
  cur.settle(p.c, pairs);
  struct Meta {
    int slot, s, where;  // slot: page * Hkv + head; -1: a bad page, -2: behind the sequence; where: b * pairs + pair
  };
  auto look_up = [&](Meta& m) {
    m.slot = -2;
    if (cur.b < p.c.B) {
      m.s = cur.s;
      m.where = cur.b * pairs + cur.pair;
      const int key = cur.s * kStepKeys + (lane & 1) * kHalfKeys;
      if (key < cur.len) {
        const int pid = __ldg(p.c.table + static_cast<size_t>(cur.b) * p.c.max_pages + (key >> p.c.page_log2));
        m.slot = pid < 0 || pid >= p.c.num_pages ? -1 : pid * p.c.Hkv + cur.pair / p.chunks;
      }
      cur.s += 16;
      cur.settle(p.c, pairs);
    }
  };
  Meta now{}, next{};
  float sk = 1.f, sv = 1.f;
  bool fresh = false;  // the batch's scales are on their way
  ScaleRun scales;
  look_up(next);
  // A stage holds rows of D bytes, keys then values; the 16-byte pieces of a row
  // are XORed with its key, so that eight keys' pieces of one block lie in
  // different banks. Pass q of a half step brings its bytes 512 q + 16 lane.
  auto swizzle = [](int key) -> uint32_t { return (D == 64 ? key >> 1 & 3 : key & 7) << 4; };
  auto place = [&](int q) -> uint32_t { return (lane * 16 + q * 512) ^ swizzle(lane / MT + q * (512 / D)); };
  int issued = 0, in_stage = 0;
  auto issue = [&]() {
    if (issued < n_steps) {
      const int j = 2 * (issued & 15);
      if (j == 0) {
        now = next;
        fresh = true;
        if (now.slot >= 0) {
          sk = __ldg(p.c.scale[0] + now.slot);
          sv = __ldg(p.c.scale[1] + now.slot);
        }
        look_up(next);
      }
      const int s = __shfl_sync(0xffffffffu, now.s, j);
      const int st = in_stage;
      in_stage = in_stage + 1 == C::STAGES ? 0 : in_stage + 1;
      const uint32_t at = ring + st * C::STAGE;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int slot = __shfl_sync(0xffffffffu, now.slot, j + h);
        if (slot >= 0) {
          const size_t row = (static_cast<size_t>(slot) << p.c.page_log2) +
                             (s * kStepKeys + h * kHalfKeys & ((1 << p.c.page_log2) - 1));
          const uint8_t* kp = p.c.code[0] + row * D + lane * 16;
          const uint8_t* vp = p.c.code[1] + row * D + lane * 16;
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            const uint32_t dst = at + h * kHalfKeys * D + place(q);
            cp_async16(dst, kp + q * 512);
            cp_async16(dst + V_AT, vp + q * 512);
          }
        } else {  // a bad page or places behind the sequence: codes of 0
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            const uint32_t dst = at + h * kHalfKeys * D + place(q);
            st_shared_v4(dst, 0, 0, 0, 0);
            st_shared_v4(dst + V_AT, 0, 0, 0, 0);
          }
        }
      }
      ++issued;
    }
    cp_async_commit();
  };
  // c sk, log2 sv (-inf hides a bad page's keys), 2^-kSumBias / sv, and s or where
  auto write_table = [&]() {
    float kf = 0.f, ev = 0.f, inv = 0.f;
    scales.take(now.slot >= 0, sv, now.where, &ev, &inv);
    if (now.slot >= 0) {
      kf = sk * p.scale_log2;
    } else if (now.slot == -1) {
      ev = -INFINITY;
      record_bad_index(p.status, WHERE_FWD_KV8);
    }
    st_shared_v4(table + ((issued - 1 & 16) * 2 + lane) * 16, __float_as_uint(kf), __float_as_uint(ev),
                 __float_as_uint(inv), lane & 1 ? now.where : now.s);
    fresh = false;
  };
#pragma unroll 1
  for (int k = 0; k < C::STAGES - 1; ++k) issue();

  // Compute side. Lane (i, c4) holds row c4 + 4 nt of the chunk for keys i,
  // i + 8 of each half step, and columns 16 t + 2 i, + 1 of its output.
  uint32_t qf[NQ][D / 16];             // pieces of the chunk's queries: column 2 r + piece
  float acc[MT][NQ + 1][4];            // O^T: tile nt has pm beside ph of rows 4 nt .., the last tile every pl
  float m[NQ], l[NQ], qfac[NQ];        // reference - kShift, sum, the query's power of two
  int limit[NQ];                       // keys the row sees
  int where = -1, seg_first = 0, seg_last = 0, seg_len = 0, seg_index = -1;
  int seg_open = 0;                    // keys that every row of the chunk sees

  auto row_place = [&](int w, int r, int* qi) -> size_t {  // row r of chunk `w`: its place in [B][Hq][Nq]
    const int b = w / pairs, pair = w - b * pairs, h = pair / p.chunks;
    const int row = (pair - h * p.chunks) * ROWS + r;
    *qi = row < p.rows ? row / p.g : INT_MAX;
    return row < p.rows ? (static_cast<size_t>(b) * p.Hq + h * p.g + row % p.g) * p.Nq + *qi : 0;
  };

  auto begin_rows = [&](int w, int s) {
    where = w;
    seg_first = s;
    ++seg_index;
    const int b = w / pairs;
    seg_len = seq_len(p.c, b);
    const int count = seq_count(p.c, b, p.Nq);
    seg_open = seg_len;
#pragma unroll
    for (int nt = 0; nt < NQ; ++nt) {
      int qi;
      const size_t at = row_place(w, nt * 4 + (i >> 1), &qi);
      const bool live = qi < p.Nq;  // rows past the count too: their loads then wait for no other
      uint2 raw[MT];  // columns 16 t + 4 c4 .. + 3
      uint32_t amax = 0;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        raw[t] = live ? __ldg(reinterpret_cast<const uint2*>(p.q + at * D + t * 16 + c4 * 4)) : make_uint2(0, 0);
      }
      // The warp's references move together, so a row past the count would show in the others' last bits.
      const bool past = qi >= count;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (past) raw[t] = make_uint2(0, 0);
        amax = max(amax, max(raw[t].x & 0x7fffu, (raw[t].x >> 16) & 0x7fffu));
        amax = max(amax, max(raw[t].y & 0x7fffu, (raw[t].y >> 16) & 0x7fffu));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // exponent of the largest value; 2^-100 and below are left as they are
      const int x = min(max(static_cast<int>(amax >> 7) - 127, -100), 127);
      const float mul = query_factor(amax, 7 - x);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint32_t w2[2] = {raw[t].x, raw[t].y};
        uint32_t word = 0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float2 f = unpack_bf16x2(w2[y]);
          __half2 v = __floats2half2_rn(f.x * mul, f.y * mul);
          const uint32_t hi = take_piece(v);
          word |= (i & 1 ? last_piece(v) : hi) << (16 * y);
        }
        qf[nt][t] = word;
      }
      qfac[nt] = __shfl_sync(0xffffffffu, exp2i(x - 7), 8 * c4);
      row_place(w, nt * 4 + c4, &qi);
      limit[nt] = p.causal && qi < count ? min(seg_len, seg_len - count + qi + 1) : seg_len;
      seg_open = min(seg_open, __reduce_min_sync(0xffffffffu, limit[nt]));
      m[nt] = -INFINITY;
      l[nt] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int nt = 0; nt <= NQ; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][nt][k] = 0.f;
  };

  // One value of O^T: its three pieces' sums. y: the second of the lane's two columns.
  auto joined = [&](int t, int nt, int y) {
    const float pl = acc[t][NQ][2 * y + (nt & 1)];
    return fmaf(pl, 1.f / 256.f, fmaf(acc[t][nt][2 * y + 1], 1.f / 16.f, acc[t][nt][2 * y]));
  };

  auto end_rows = [&]() {
    const bool whole = seg_first == 0 && seg_last + 1 == steps_of(seg_len);
    const int count = seq_count(p.c, where / pairs, p.Nq);
#pragma unroll
    for (int nt = 0; nt < NQ; ++nt) {
      float sum = l[nt];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int r = nt * 4 + c4;
      int qi;
      const size_t at = row_place(where, r, &qi);
      if (qi >= count) continue;
      if (whole) {
        const RowEnd end(m[nt], sum);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          *reinterpret_cast<uint32_t*>(p.o + at * D + t * 16 + 2 * i) =
              pack_bf16x2(end(joined(t, nt, 0)), end(joined(t, nt, 1)));
        if (i == 0) p.lse[at] = end.lse;
      } else {
        const size_t slot = (static_cast<size_t>(gid) * 2 + (seg_index > 0)) * p.part_rows + r;
#pragma unroll
        for (int t = 0; t < MT; ++t)
          *reinterpret_cast<float2*>(p.part + slot * D + t * 16 + 2 * i) =
              make_float2(joined(t, nt, 0), joined(t, nt, 1));
        if (i == 0) p.part_ml[slot] = make_float2(m[nt], sum);
      }
    }
  };

  // rows of the matrix loads: K's four are (keys 0-7, 8-15) x (block, next one), V's four groups of 8 keys
  const int mat = lane >> 3, mrow = lane & 7;
  const uint32_t k_row = ((mat & 1) * 8 + mrow) * D + (((mat >> 1) << 4) ^ swizzle(mrow));
  const uint32_t v_row = (mat * 8 + mrow) * D + swizzle(mrow);
  auto block = [](int j) -> uint32_t { return (j & 7) << 4; };  // its place in a row: XORed; every eighth: 128 bytes on

  // the first rows' queries, while the first copies are under way
  begin_rows(__shfl_sync(0xffffffffu, now.where, 0), __shfl_sync(0xffffffffu, now.s, 0));
  int out_stage = 0;
#pragma unroll 1
  for (int k = 0; k < n_steps; ++k) {
    cp_async_wait<C::STAGES - 2>();
    if (fresh) write_table();
    __syncwarp();  // every lane's copies of the step are there, and the last step has been read
    issue();
    const int st = out_stage;
    out_stage = out_stage + 1 == C::STAGES ? 0 : out_stage + 1;
    const uint32_t at = ring + st * C::STAGE;
    const uint32_t entry = table + (k & 31) * 32;
    const uint4 head[2] = {ld_shared_v4(entry), ld_shared_v4(entry + 16)};
    const int s = static_cast<int>(head[0].w);
    if (static_cast<int>(head[1].w) != where) {
      end_rows();
      begin_rows(static_cast<int>(head[1].w), s);
    }
    seg_last = s;

    // The matrix loads stand in groups ahead of the products that use them: they
    // are ordered against the copies, so the compiler moves none of them.
    constexpr int KG = MT < 8 ? MT / 2 : 4;  // column block pairs a group
    float sc[2][NQ][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[h][nt][e] = 0.f;
#pragma unroll
    for (int j0 = 0; j0 < MT; j0 += 2 * KG) {
      uint4 kb[KG][2];
#pragma unroll
      for (int j = 0; j < KG; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          kb[j][h] = ldmatrix4(at + h * kHalfKeys * D + (j0 + 2 * j) / 8 * 128 + (k_row ^ block(j0 + 2 * j)));
#pragma unroll
      for (int j = 0; j < KG; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NQ; ++nt)
            mma_e4m3(sc[h][nt], kb[j][h].x, kb[j][h].y, kb[j][h].z, kb[j][h].w, qf[nt][j0 + 2 * j],
                     qf[nt][j0 + 2 * j + 1]);
    }
    // What lies behind the last token may be any bytes, NaN codes among them,
    // and 0 * NaN is not 0.
    if ((s + 1) * kStepKeys > seg_len) {
#pragma unroll 1
      for (int q = 0; q < 2 * (D / 32); ++q) {
        const int key = (q & 1) * kHalfKeys + lane / MT + (q >> 1) * (512 / D);
        if (s * kStepKeys + key >= seg_len) st_shared_v4(at + V_AT + (q & 1) * kHalfKeys * D + place(q >> 1), 0, 0, 0, 0);
      }
      __syncwarp();
    }
    constexpr int VG = 4;  // column blocks a group
    uint4 vb[2][VG];
    auto load_v = [&](int j0, uint4 (&v)[VG]) {
#pragma unroll
      for (int j = 0; j < VG; ++j)
        v[j] = ldmatrix4_trans(at + V_AT + (j0 + j) / 8 * 128 + (v_row ^ block(j0 + j)));
    };
    load_v(0, vb[0]);

    float t[2][NQ][2];  // u of keys i, i + 8 of each half
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float dot = fmaf(sc[h][nt][2 * y + 1], 1.f / 16.f, sc[h][nt][2 * y]) * qfac[nt];
          t[h][nt][y] = fmaf(dot, __uint_as_float(head[h].x), __uint_as_float(head[h].y));
        }
    if ((s + 1) * kStepKeys > seg_open) {  // some row does not see every key of this step
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NQ; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (s * kStepKeys + h * kHalfKeys + i + 8 * y >= limit[nt]) t[h][nt][y] = -INFINITY;
    }
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NQ; ++nt)
      grow |= fmaxf(fmaxf(t[0][nt][0], t[0][nt][1]), fmaxf(t[1][nt][0], t[1][nt][1])) > m[nt] + (kSlack + kShift);
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt) {
        float mx = fmaxf(fmaxf(t[0][nt][0], t[0][nt][1]), fmaxf(t[1][nt][0], t[1][nt][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) - kShift;
        const float to = fmaxf(m[nt], mx);
        const float alpha = to == -INFINITY ? 1.f : ex2_approx(m[nt] - to);
        l[nt] = to == -INFINITY ? l[nt] : scale_sum(l[nt], m[nt] - to, alpha);
        m[nt] = to;
#pragma unroll
        for (int q = 0; q < MT; ++q) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[q][nt][e] *= alpha;
          acc[q][NQ][nt] *= alpha;
          acc[q][NQ][2 + nt] *= alpha;
        }
      }
    }

    uint32_t pf[NQ + 1][2];  // pieces of the weights as the B operand: keys 2 c4, + 8, + 1, + 9 of column i
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t small = 0;
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt) {
        const float ref = m[nt] == -INFINITY ? 0.f : m[nt];
        const float a = ex2_approx(t[h][nt][0] - ref), b = ex2_approx(t[h][nt][1] - ref);
        l[nt] = fmaf(a + b, __uint_as_float(head[h].z), l[nt]);
        __half2 v = __floats2half2_rn(a, b);
        const uint32_t hi = take_piece(v);
        const uint32_t mid = take_piece(v);
        pf[nt][h] = transpose8(hi | mid << 16);
        small |= last_piece(v) << (16 * nt);
      }
      pf[NQ][h] = transpose8(small);
    }

#pragma unroll
    for (int j0 = 0; j0 < MT; j0 += VG) {
      if (j0 + VG < MT) load_v(j0 + VG, vb[(j0 / VG + 1) & 1]);
#pragma unroll
      for (int j = 0; j < VG; ++j) {
        // word q: keys 8 q + 2 c4, + 1 of columns 16 (j0 + j) + 2 i, + 1
        const uint4 v = vb[(j0 / VG) & 1][j];
        const uint32_t a0 = __byte_perm(v.x, v.y, 0x6240), a1 = __byte_perm(v.x, v.y, 0x7351);
        const uint32_t a2 = __byte_perm(v.z, v.w, 0x6240), a3 = __byte_perm(v.z, v.w, 0x7351);
#pragma unroll
        for (int nt = 0; nt <= NQ; ++nt) mma_e4m3(acc[j0 + j][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
      }
    }
  }
  end_rows();
  cp_async_wait<0>();
}

// Joins the parts of a query row whose keys several warps shared, and writes
// the rows of sequences without keys. One block per row; a row that one warp
// had whole is already final.
template <int D>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const __grid_constant__ Kv8Attn p, int warps, int per_chunk) {
  constexpr int LANES = D / 4, GROUPS = 128 / LANES;
  __shared__ float4 red[128];
  __shared__ float2 red_ml[GROUPS];
  const int row = blockIdx.x % p.rows;
  const int bh = blockIdx.x / p.rows, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const int qi = row / p.g;
  // Lengths and counts are inputs of the kernel this one overlaps, so they can
  // be read before its parts are there.
  const bool bad_len = seq_len(p.c, b) != __ldg(p.c.lens + b);
  const bool bad_count = p.c.counts && seq_count(p.c, b, p.Nq) != __ldg(p.c.counts + b);
  const int pairs = p.c.Hkv * p.chunks, steps = seq_steps(p.c, b);
  const size_t at = (static_cast<size_t>(b) * p.Hq + h * p.g + row % p.g) * p.Nq + qi;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const bool live = !bad_len && !bad_count && qi < seq_count(p.c, b, p.Nq);
  long long total, before;
  int some;
  step_totals(p.c, pairs, b, &total, &before, &some);
  const int used = max(1, used_warps(total, static_cast<long long>(some) * pairs, warps));
  const int chunk = row / per_chunk, r = row - chunk * per_chunk;
  const long long s0 = before + static_cast<long long>(h * p.chunks + chunk) * steps, s1 = s0 + steps - 1;
  if (!live && p.fill) {  // no other kernel of the call writes the row
    if (group == 0) *reinterpret_cast<uint2*>(p.o + at * D + lane * 4) = make_uint2(0, 0);
    if (threadIdx.x == 0) p.lse[at] = 0.f;
  }
  griddep_wait();
  if ((bad_len || bad_count) && threadIdx.x == 0) record_bad_index(p.status, WHERE_FWD_KV8);
  if (!live) return;
  if (steps == 0) {
    if (group == 0) *reinterpret_cast<uint2*>(p.o + at * D + lane * 4) = make_uint2(0, 0);
    if (threadIdx.x == 0) p.lse[at] = -INFINITY;
    return;
  }
  // the warp that holds step x: the largest w with first_step(w) <= x
  const int w0 = static_cast<int>(((s0 + 1) * used - 1) / total), w1 = static_cast<int>(((s1 + 1) * used - 1) / total);
  if (w0 == w1) return;
  // Each group of threads joins every GROUPS-th part as it comes, then the
  // groups are joined in order.
  const int late = s0 > first_step(total, used, w0) ? 1 : 0;  // the row's first part is its warp's last
  float m = -INFINITY, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float low = INFINITY;  // smallest reference of a part that saw keys
  auto join = [&](float mx, float lx, const float4& x) {
    const float to = fmaxf(m, mx);
    const float ref = to == -INFINITY ? 0.f : to;
    const float wa = ex2_approx(m - ref), wx = ex2_approx(mx - ref);
    l = l * wa + lx * wx;
    low = fminf(low, lx > 0.f ? mx : INFINITY);
    m = to;
    a.x = a.x * wa + x.x * wx, a.y = a.y * wa + x.y * wx, a.z = a.z * wa + x.z * wx, a.w = a.w * wa + x.w * wx;
  };
  for (int w = w0 + group; w <= w1; w += 4 * GROUPS) {  // four on their way at a time
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int v = min(w + e * GROUPS, w1);
      const size_t slot = (static_cast<size_t>(v) * 2 + (v == w0 ? late : 0)) * p.part_rows + r;
      ml[e] = p.part_ml[slot];
      x[e] = *reinterpret_cast<const float4*>(p.part + slot * D + lane * 4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (w + e * GROUPS <= w1) join(ml[e].x, ml[e].y, x[e]);
  }
  if (m - low > 100.f) {  // a part's factor may have left fp32's range, its sum is added again
    l = 0.f;
#pragma unroll 1
    for (int w = w0 + group; w <= w1; w += GROUPS) {
      const float2 ml = p.part_ml[(static_cast<size_t>(w) * 2 + (w == w0 ? late : 0)) * p.part_rows + r];
      l += scale_sum(ml.y, ml.x - m, ex2_approx(ml.x - m));
    }
  }
  red[threadIdx.x] = a;
  if (lane == 0) red_ml[group] = make_float2(m, l);
  __syncthreads();
  if (group > 0) return;
  const float l0 = l, m0 = m;
  low = l > 0.f ? m : INFINITY;
  for (int u = 1; u < GROUPS; ++u) join(red_ml[u].x, red_ml[u].y, red[u * LANES + lane]);
  if (m - low > 100.f) {
    l = scale_sum(l0, m0 - m, ex2_approx(m0 - m));
#pragma unroll 1
    for (int u = 1; u < GROUPS; ++u) l += scale_sum(red_ml[u].y, red_ml[u].x - m, ex2_approx(red_ml[u].x - m));
  }
  const RowEnd end(m, l);
  *reinterpret_cast<uint2*>(p.o + at * D + lane * 4) =
      make_uint2(pack_bf16x2(end(a.x), end(a.y)), pack_bf16x2(end(a.z), end(a.w)));
  if (lane == 0) p.lse[at] = end.lse;
}

// More query rows per K/V head than this take the 128-row tiles of
// fa_fwd_kv8_tile.cu. This kernel reads the cache once per chunk of rows; the
// tiles' time hardly depends on the rows below 128. B = 8, Hkv = 8, 16384 keys
// (and B = 1, Hkv = 8, 4096 keys), rows: this kernel / tiles, us:
//   d =  64: 8: 39 / 73 (13.9 / 19.0)    16: 62 / 73 (14.3 / 19.1)    24: 87 / 73 (16.5 / 19.1)
//   d = 128: 8: 57 / 89 (17.4 / 20.6)    12: 97 / 89 (19.0 / 20.0)    16: 99 / 89 (19.5 / 20.3)
//            24: 142 / 89 (22.0 / 20.7)
//   d = 256: 8: 178 / 174 (17.5 / 24.9)  12: 260 / 174 (20.6 / 25.0)  16: 339 / 174 (20.5 / 25.2)
// At d = 128 the tiles would be a tenth faster on the long caches from 9 rows on; up to
// 16 stay here for the short calls and because the tiles hold a query's small
// columns 16 times as coarsely. So do 8 at d = 256.
constexpr int tile_rows(int d) { return d == 256 ? 8 : 16; }

// 8-column tiles of a row chunk: two (8 rows) where the rows fill more than one
// and the sums of both fit the registers.
int query_tiles(int d, long long rows) { return d <= 128 && rows > 4 ? 2 : 1; }

size_t part_bytes(int d, long long rows, size_t* ml_off) {
  const size_t slots = static_cast<size_t>(2) * kMaxSms * warps_per_cta(d) * std::min<long long>(rows, 4 * query_tiles(d, rows));
  *ml_off = slots * d * sizeof(float);
  return *ml_off + slots * sizeof(float2);
}

template <int D, int NQ>
cudaError_t launch_t(Kv8Attn& a, const DeviceInfo& dev, cudaStream_t stream) {
  using C = Cfg<D, NQ>;
  auto kern = kv8_attn_kernel<D, NQ>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, C::SMEM, dev.device, allowed);
  if (e != cudaSuccess) return e;
  // no more blocks than runs that the longest sequences the table allows could have
  const double most = static_cast<double>(a.c.B) * a.c.Hkv * a.chunks *
                      ((static_cast<long long>(a.c.max_pages) << a.c.page_log2) / kStepKeys + 1) / kMinSteps;
  const int full = std::min(dev.num_sms, kMaxSms);
  const int grid = most < full ? std::max(1, static_cast<int>(most)) : full;
  kern<<<grid, C::WARPS * 32, C::SMEM, stream>>>(a);
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
  return cudaLaunchKernelEx(&cfg, kv8_combine_kernel<D>, a, grid * C::WARPS, 4 * NQ);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_kv8_workspace_size(int B, int Hq, int Hkv, int Nq, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Hq % Hkv != 0) return 0;
  if (d != 64 && d != 128 && d != 256) return 0;
  const long long rows = static_cast<long long>(Hq / Hkv) * Nq;
  size_t off;
  return rows > tile_rows(d) ? kv8_tile_workspace(d) : part_bytes(d, rows, &off);
}

static fa_status_t run_fwd_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                               const float* v_scale, const int* page_table, const int* lens, const int* counts,
                               void* o, float* lse, int B, int Hq, int Hkv, int Nq, int d, int page, int num_pages,
                               int max_pages, int causal, float scale, void* workspace, size_t workspace_bytes,
                               int fill, cudaStream_t stream) {
  Kv8Attn a{};
  a.fill = fill;
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
  a.Hq = Hq;
  a.Nq = Nq;
  a.g = Hq / Hkv;
  a.causal = causal;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  a.rows = a.g * Nq;
  if (a.rows > tile_rows(d)) return launch_kv8_tiles(a, d, workspace, dev, stream);
  a.status = dev.status;
  const int nq = query_tiles(d, a.rows);
  a.chunks = (a.rows + 4 * nq - 1) / (4 * nq);
  a.part_rows = std::min(a.rows, 4 * nq);
  part_bytes(d, a.rows, &ml_off);
  a.part = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ml_off);
  if (d == 64) return from_cuda(nq == 1 ? launch_t<64, 1>(a, dev, stream) : launch_t<64, 2>(a, dev, stream));
  if (d == 128) return from_cuda(nq == 1 ? launch_t<128, 1>(a, dev, stream) : launch_t<128, 2>(a, dev, stream));
  return from_cuda(launch_t<256, 1>(a, dev, stream));
}

fa_status_t fa_fwd_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int* page_table, const int* lens, const int* counts, void* o,
                       float* lse, int B, int Hq, int Hkv, int Nq, int d, int page, int num_pages, int max_pages,
                       int causal, float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_fwd_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, o, lse, B, Hq, Hkv, Nq, d, page,
                     num_pages, max_pages, causal, scale, workspace, workspace_bytes, 0, stream);
}

fa_status_t fa_fwd_kv8_filled(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                              const float* v_scale, const int* page_table, const int* lens, const int* counts, void* o,
                              float* lse, int B, int Hq, int Hkv, int Nq, int d, int page, int num_pages,
                              int max_pages, int causal, float scale, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  return run_fwd_kv8(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, counts, o, lse, B, Hq, Hkv, Nq, d, page,
                     num_pages, max_pages, causal, scale, workspace, workspace_bytes, 1, stream);
}

}  // extern "C"
