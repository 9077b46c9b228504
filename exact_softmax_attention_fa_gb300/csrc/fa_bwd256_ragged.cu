// dK and dV over packed sequences for head dimension 256 on sm_103a.
//
// P = exp(S - L), dV = P^T dO, dP = dO V^T, dS = P o (dP - D), dK = dS^T Q, keys on
// the TMEM lanes as in fa_bwd256.cu. There a work item owns half of the columns of
// dK and dV and forms S^T and dP^T for them, so both are formed twice. Here an item
// owns all of dV or all of dK (256 columns of TMEM): a dV item forms S^T alone, a dK
// item both, three products of 64 queries a tile instead of four, and three phases
// of the softmax warps instead of four.
//   - K_j and (dK items) V_j stay in shared memory for the item, 64 KB each. Query
//     tiles of 64 rows stream through two slots of Q and one of dO (32 KB each), for
//     dV items two of dO: the second is V_j's place (with one, each tile waited for
//     its dO, and a dV item took longer than a dK item). That leaves no room for dS^T,
//     which goes to TMEM as the A operand of dK += dS^T Q, as P^T does for dV += P^T dO.
//   - P stays in registers in fp32 between the phases of a dK item.
//   - MMA order per query tile n: S^T(n+1) once phase A(n) has S^T(n) in registers;
//     dV(n) after phase A(n), or dK(n) after phase B(n) and then dP^T(n+1). A commit covers all that
//     was issued before it: s_full(n) says that dV(n-2) has read its P^T, dp_full(n)
//     that dK(n-1) has read its dS^T.
// Three sequences of up to 2501 rows, 8 + 2 heads, no mask: 486 us with its dQ kernel
// instead of 610 with halves. A dK tile takes 1.6 us, of which its products 1.3 (those
// of 64 queries take the pipe as long as those of 128 do), a dV tile 1.45.
// TMEM columns (512 allocated): dV or dK [0, 256), S^T [256, 320), dP^T [320, 384),
// P^T or dS^T in two buffers [384, 416) and [416, 448) (tile n in buffer n & 1).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kTailWarp = 10;
constexpr int kThreads = 352;
constexpr int kItemConsumers = 1 + 256;  // the MMA thread and the softmax threads

struct Cfg {
  static constexpr int BQ = 64;                    // query rows per tile
  static constexpr int KV_CHUNK = 128 * 128;       // [128 keys][64 d] bf16
  static constexpr int KV_BYTES = 4 * KV_CHUNK;    // 64 KB
  static constexpr int Q_CHUNK = BQ * 128;         // [64 rows][64 d] bf16, 8 KB
  static constexpr int Q_BYTES = 4 * Q_CHUNK;      // 32 KB
  static constexpr int Q_SLOTS = 2;
  static constexpr int LD_BYTES = 2 * 64 * 4;      // per warpgroup: 32 base-2 L + 32 scaled D
  static constexpr uint32_t ACC_COL = 0, S_COL = 256, DP_COL = 320;
  __host__ __device__ static constexpr uint32_t x_col(int b) { return 384u + 32u * uint32_t(b); }
  // smem: K_j, V_j, two Q_i, one dO_i, L/D staging
  static constexpr int SMEM_BYTES = 2 * KV_BYTES + (Q_SLOTS + 1) * Q_BYTES + LD_BYTES + 1024;
};

struct Shared {
  uint64_t kv_full;
  uint64_t q_full[2], q_empty[2];  // slot n % 2
  uint64_t do_full[2], do_empty[2];  // dO: slot n % 2 of a dV item's tile n, slot 0 of a dK item's
  TailShared tail;
  uint64_t s_full, s_read;     // S^T is there, and in registers
  // P^T (dV items) or dS^T (dK items) is in its buffer, tile n in n & 1. Two barriers,
  // because a dV item's softmax can finish tile n + 1 (S^T(n+1) is issued before the
  // MMA thread waits for P^T(n)) before that wait starts, and on one barrier the wait
  // would then see two completed phases. Tile n + 2 needs S^T(n+2), issued after it.
  uint64_t x_ready[2];
  uint64_t dp_full;            // tiles of dK items
  uint64_t acc_done, acc_free;
  uint64_t mma_drain;  // the MMA thread's last commit: all its MMAs done before the CTA exits
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  int item_ring[kItemSlots];
  uint32_t tmem_base;
  int abort_flag;
};

// Work item: key tile j of K/V head bh, its dK or its dV. Its query stream is, for
// each of the g query heads that share the K/V head, the 64-row query tiles i0 ..
// T64-1 (causal: i0 = 2j). An entry of the plan's list has its dK items, which are
// the longer ones, before its dV items.
template <bool CAUSAL>
struct Work {
  int bh, j, i0, T64, g, row0, n;
  bool dk;
  __device__ Work(int item, const BwdLaunch& p) {
    const uint32_t units = 2 * p.BHkv;
    const int e = static_cast<int>(static_cast<uint32_t>(item) / units);
    const int rem = item - e * static_cast<int>(units);
    const int4 x = __ldg(packed_tiles(p.plan) + e);
    row0 = x.x;
    n = x.y;
    T64 = (n + 63) >> 6;
    j = CAUSAL ? ((n + 127) >> 7) - 1 - x.z : x.z;
    dk = rem < p.BHkv;
    bh = dk ? rem : rem - p.BHkv;
    i0 = CAUSAL ? 2 * j : 0;
    g = p.group;
  }
  __device__ int n_iter() const { return g * (T64 - i0); }
  struct Pos {
    int bh, i;  // query head, 64-row query tile
  };
  __device__ Pos first() const { return Pos{bh * g, i0}; }
  __device__ void advance(Pos& p) const {
    if (++p.i == T64) {
      p.i = i0;
      ++p.bh;
    }
  }
};

__device__ __forceinline__ int total_items(const BwdLaunch& p) {
  return packed_plan_ok(p.plan, p.N) ? (p.plan->n_tiles - p.plan->n_short) * p.BHkv * 2 : 0;
}

// TMA producer (one thread): per query tile Q_i and dO_i as their slots free up; per
// item K_j and, for dK, V_j once every MMA of the previous item has completed.
template <bool CAUSAL>
__device__ void load_role(const BwdLaunch& p, Shared& sh, uint8_t* sK, uint8_t* sV, uint8_t* sQ, uint8_t* sdO) {
  using C = Cfg;
  tma_prefetch_desc(&p.tmQ);
  tma_prefetch_desc(&p.tmK);
  tma_prefetch_desc(&p.tmV);
  tma_prefetch_desc(&p.tmdO);
  const int total = total_items(p);
  const uint64_t lim = p.wait_limit_ns;
  int g = 0, items = 0, kv_issued = 0;
  int q_issued = 0, do_issued[2] = {0, 0};  // loads into the slots
  bool aborted = false;
  auto load = [&](uint64_t* bar, uint8_t* dst, const CUtensorMap* map, int row, int bh) {
    mbar_arrive_expect_tx(bar, C::Q_BYTES);
#pragma unroll
    for (int c = 0; c < 4; ++c) tma_load_3d(dst + c * C::Q_CHUNK, map, bar, c * 64, row, bh);
  };
  auto load_do = [&](int s, int row, int bh) -> bool {
    if (do_issued[s] > 0 && !mbar_wait(&sh.do_empty[s], (do_issued[s] - 1) & 1, &sh.abort_flag, lim)) return false;
    load(&sh.do_full[s], s ? sV : sdO, &p.tmdO, row, bh);
    ++do_issued[s];
    return true;
  };
  auto load_q = [&](int n, int row, int bh) -> bool {  // n: the tile's number
    const int s = n % C::Q_SLOTS;
    if (n >= C::Q_SLOTS && !mbar_wait(&sh.q_empty[s], ((n / C::Q_SLOTS) - 1) & 1, &sh.abort_flag, lim)) return false;
    load(&sh.q_full[s], sQ + s * C::Q_BYTES, &p.tmQ, row, bh);
    ++q_issued;
    return true;
  };
  int item = blockIdx.x;
  while (!aborted) {
    if (!publish_item(sh, items, item, lim)) {
      aborted = true;
      break;
    }
    if (item >= total) break;
    const Work<CAUSAL> wk(item, p);
    const int n_iter = wk.n_iter();
    typename Work<CAUSAL>::Pos pos = wk.first(), q_pos = pos;
    auto row_of = [&](const typename Work<CAUSAL>::Pos& at) { return wk.row0 + at.i * C::BQ; };
    // (a first tile uses slot 0 of dO: slot 1 is V_j's place until then)
    if (!load_q(g, row_of(pos), pos.bh) || !load_do(0, row_of(pos), pos.bh) ||
        (items > 0 && !mbar_wait(&sh.acc_done, (items - 1) & 1, &sh.abort_flag, lim))) {
      aborted = true;
      break;
    }
    if (!debug_skip_here(p.debug_skip, WHERE_BWD_LOAD, items == 0)) {  // test hook
      mbar_arrive_expect_tx(&sh.kv_full, (wk.dk ? 2 : 1) * C::KV_BYTES);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tma_load_3d(sK + c * C::KV_CHUNK, &p.tmK, &sh.kv_full, c * 64, wk.row0 + wk.j * 128, wk.bh);
        if (wk.dk) tma_load_3d(sV + c * C::KV_CHUNK, &p.tmV, &sh.kv_full, c * 64, wk.row0 + wk.j * 128, wk.bh);
      }
      ++kv_issued;
    }
    // In the order in which the slots free up: dO_n after dP^T(n-1) and Q_(n+1) after
    // dK(n-1); for dV Q_(n+1) after S^T(n-1) and dO_n after dV(n-2).
    int q_next = 1;
    auto next_q = [&]() -> bool {
      if (q_next >= n_iter) return true;
      wk.advance(q_pos);
      return load_q(g + q_next++, row_of(q_pos), q_pos.bh);
    };
    if (!next_q()) aborted = true;
    for (int n = 1; n < n_iter && !aborted; ++n) {
      wk.advance(pos);
      aborted = wk.dk ? !load_do(0, row_of(pos), pos.bh) || !next_q()
                      : !next_q() || !((n & 1) ? load_do(1, row_of(pos), pos.bh) : load_do(0, row_of(pos), pos.bh));
    }
    if (aborted) break;
    g += n_iter;
    ++items;
    item = claim_item(p.sched);
  }
  finish_claiming(p.sched);
  if (aborted) record_timeout(p.status, &sh.abort_flag, WHERE_BWD_LOAD);
  // The copies already issued land before the CTA can exit (after an abort no consumer
  // may wait for them): the latest phase issued into each slot.
  for (int n = std::max(0, q_issued - C::Q_SLOTS); n < q_issued; ++n)
    drain_wait(&sh.q_full[n % C::Q_SLOTS], (n / C::Q_SLOTS) & 1, lim);
  for (int s = 0; s < 2; ++s)
    if (do_issued[s] > 0) drain_wait(&sh.do_full[s], (do_issued[s] - 1) & 1, lim);
  if (kv_issued > 0) drain_wait(&sh.kv_full, (kv_issued - 1) & 1, lim);
}

// One thread issues every MMA (order in the file header).
template <bool CAUSAL>
__device__ void mma_role(const BwdLaunch& p, Shared& sh, uint8_t* sK, uint8_t* sV, uint8_t* sQ, uint8_t* sdO,
                         uint32_t tmem) {
  using C = Cfg;
  constexpr uint32_t kIdescS = make_idesc_bf16_f32(128, 64, false, false);   // S^T, dP^T: 128 keys x 64 queries
  constexpr uint32_t kIdescAcc = make_idesc_bf16_f32(128, 256, false, true);  // dV, dK
  const uint32_t k_addr = smem_u32(sK), v_addr = smem_u32(sV), q_addr = smem_u32(sQ), do_addr = smem_u32(sdO);
  const uint64_t lim = p.wait_limit_ns;
  const int total = total_items(p);
  auto fail = [&]() {
    record_timeout(p.status, &sh.abort_flag, WHERE_BWD_MMA);
    drain_mmas(&sh.mma_drain, lim);
  };
  // D[tmem] = A (128 keys x 256, K-major, resident) * B (64 queries x 256, K-major)^T
  auto issue_sq = [&](uint32_t d_col, uint32_t a_addr, uint32_t b_addr) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint64_t ad = make_smem_desc_sw128(a_addr + c * C::KV_CHUNK, 16, 1024);
      const uint64_t bd = make_smem_desc_sw128(b_addr + c * C::Q_CHUNK, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        umma_ss(tmem + d_col, desc_add(ad, ks * 32), desc_add(bd, ks * 32), kIdescS, (c > 0 || ks > 0) ? 1u : 0u);
    }
  };
  // dV or dK += A (TMEM: 128 keys x 64 queries, buffer b) * B (64 queries x 256, MN-major)
  auto issue_acc = [&](int steps, int b, uint32_t b_addr, bool first) {
    const uint64_t bd = make_smem_desc_sw128(b_addr, C::Q_CHUNK, 1024);
    issue_steps<4, true>(steps, [&](int ks) {
      umma_ts(tmem + C::ACC_COL, tmem + C::x_col(b) + ks * 8, desc_add(bd, ks * 2048), kIdescAcc,
              (!first || ks > 0) ? 1u : 0u);
    });
  };

  int g = 0, items = 0;  // tiles
  int d0 = 0, d1 = 0;    // tiles of dO in slot 0 and 1
  TailCalls<false> tail;
  while (true) {
    const int item = take_item(sh, items, lim);
    if (item < 0) return fail();
    if (item >= total) break;
    const Work<CAUSAL> wk(item, p);
    const int n_iter = wk.n_iter();
    const bool dk = wk.dk;
    // steps of 16 queries that a product over the last query tile takes, and tiles of
    // the stream until the next such tile (as in fa_bwd.cu)
    const int held = wk.n - (wk.T64 - 1) * C::BQ;
    int until = held < C::BQ ? wk.T64 - 1 - wk.i0 : INT_MAX;
    auto clean = [&](uint32_t tile) -> bool {
      tail.ask(sh.tail, held, tile);
      return tail.wait(sh.tail, &sh.abort_flag, lim);
    };
    // S^T(n): the S region is free, phase A(n - 1) has read it (s_read)
    auto issue_s = [&](int n, bool cut) -> bool {
      const int s = n % C::Q_SLOTS;
      if (!mbar_wait(&sh.q_full[s], (n / C::Q_SLOTS) & 1, &sh.abort_flag, lim)) return false;
      if (cut && dk && !clean(q_addr + s * C::Q_BYTES)) return false;
      tc_fence_after_sync();
      issue_sq(C::S_COL, k_addr, q_addr + s * C::Q_BYTES);
      umma_commit(&sh.s_full);
      if (!dk) umma_commit(&sh.q_empty[s]);
      return true;
    };
    // the next dP^T: phase B(n - 1) has read the last one (x_ready)
    auto issue_dp = [&]() -> bool {
      if (!mbar_wait(&sh.do_full[0], d0++ & 1, &sh.abort_flag, lim)) return false;
      tc_fence_after_sync();
      issue_sq(C::DP_COL, v_addr, do_addr);
      umma_commit(&sh.dp_full);
      umma_commit(&sh.do_empty[0]);
      return true;
    };
    if (!mbar_wait(&sh.kv_full, items & 1, &sh.abort_flag, lim) || !issue_s(g, until == 0)) return fail();
    if (dk && !issue_dp()) return fail();
    for (int n = 0; n < n_iter; ++n, ++g) {
      const bool has_next = n + 1 < n_iter, cut = until == 0;
      const int steps = cut ? (held + 15) >> 4 : 4;
      if (!mbar_wait(&sh.s_read, g & 1, &sh.abort_flag, lim)) return fail();
      if (has_next && !issue_s(g + 1, (cut ? until = wk.T64 - 1 - wk.i0 : --until) == 0)) return fail();
      // the first product of an item overwrites the accumulator: the previous item's
      // epilogue must have read it
      if (n == 0 && items > 0 && !mbar_wait(&sh.acc_free, (items - 1) & 1, &sh.abort_flag, lim)) return fail();
      if (!mbar_wait(&sh.x_ready[g & 1], (g >> 1) & 1, &sh.abort_flag, lim)) return fail();
      if (dk) {
        tc_fence_after_sync();
        issue_acc(steps, g & 1, q_addr + (g % C::Q_SLOTS) * C::Q_BYTES, n == 0);
        umma_commit(&sh.q_empty[g % C::Q_SLOTS]);
        if (has_next && !issue_dp()) return fail();
      } else {
        const int s = n & 1;
        const uint32_t from = s ? v_addr : do_addr;
        if (!mbar_wait(&sh.do_full[s], (s ? d1++ : d0++) & 1, &sh.abort_flag, lim)) return fail();
        if (cut && !clean(from)) return fail();
        tc_fence_after_sync();
        issue_acc(steps, g & 1, from, n == 0);
        umma_commit(&sh.do_empty[s]);
      }
    }
    umma_commit(&sh.acc_done);
    ++items;
  }
  // Normally the epilogues have waited for the last products; if a softmax
  // warpgroup gave up, nothing has.
  tail.finish(sh.tail);
  drain_mmas(&sh.mma_drain, lim);
}

// Warpgroup w (w = 0, 1) owns queries [32w, 32w + 32) of every tile; thread r owns key
// r (TMEM lane r). Order per tile n of a dK item: B(n), A(n+1). After an item's last
// tile each warpgroup writes half of its columns straight from TMEM.
template <bool CAUSAL>
__device__ void softmax_role(const BwdLaunch& p, Shared& sh, float* sLD, uint32_t tmem, int w) {
  using C = Cfg;
  const int r = threadIdx.x & 127;
  const uint32_t lane_base = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
  const float c2 = p.scale_log2;
  const float sc = p.scale;
  const uint64_t lim = p.wait_limit_ns;
  float* ld_l2 = sLD + w * 64;  // 32 base-2 logsumexps, then 32 scaled D values
  float* ld_d = ld_l2 + 32;
  const uint32_t bar_id = 1 + w;
  const uint32_t tS = tmem + lane_base + C::S_COL + 32 * w;
  const uint32_t tDP = tmem + lane_base + C::DP_COL + 32 * w;
  const uint32_t tX = tmem + lane_base + C::x_col(0) + 16 * w;  // + 32 for buffer 1
  const int total = total_items(p);
  bool alive = true;
  float pv[32];  // P^T of the current tile

  // thread r < 32 loads L2 of query 32w + r of the tile, 32 <= r < 64 its scaled D.
  // Queries behind the sequence's last one get L2 = +inf (weight 0) and D = 0.
  // (Ordinary loads: this grid is resident while the kernel before still writes them.)
  auto fetch_ld = [&](const Work<CAUSAL>& wk, int bh, int i) -> float {
    if (r >= 64) return 0.f;
    const int q = i * C::BQ + 32 * w + (r & 31);
    const float* from = (r < 32 ? p.lse2 : p.D) + static_cast<size_t>(bh) * p.N + wk.row0;
    const float x = from[min(q, wk.n - 1)];
    return r < 32 ? (q < wk.n ? x : INFINITY) : (q < wk.n ? x * sc : 0.f);
  };
  auto wait_all = [&](uint64_t* bar, int parity, int where) {
    alive = alive && __all_sync(0xffffffffu, mbar_wait(bar, parity, &sh.abort_flag, lim));
    if (!alive) record_timeout(p.status, &sh.abort_flag, where);
    tc_fence_after_sync();
  };

  // ---- phase A of query tile i (global tile g): P^T in registers, and for dV in TMEM
  // (bf16). The next S^T may come as soon as this one is in registers (where dV's came
  // after P^T was stored, 503 us instead of 491).
  auto phase_a = [&](const Work<CAUSAL>& wk, int i, int g) {
    wait_all(&sh.s_full, g & 1, WHERE_BWD_SOFTMAX);
    if (!alive) return;
    uint32_t a[32];
    tmem_ld32(tS, a);
    tmem_ld_wait();
    tc_fence_before_sync();
    mbar_arrive(&sh.s_read);
    // key 128j + r is seen by query 64i + 32w + c if (causal) it is not after the
    // query: c >= c_lo. (A key behind the sequence's last one stays: its row of P^T
    // and dS^T reaches only its own row of dV and dK, which is not written.)
    const int c_lo = CAUSAL ? wk.j * 128 + r - i * C::BQ - 32 * w : 0;
#pragma unroll
    for (int c4 = 0; c4 < 32; c4 += 4) {
      const float4 l = *reinterpret_cast<const float4*>(ld_l2 + c4);
      const float2 x01 = ffma2_bcast_mul(__uint_as_float(a[c4]), __uint_as_float(a[c4 + 1]), c2, -l.x, -l.y);
      const float2 x23 = ffma2_bcast_mul(__uint_as_float(a[c4 + 2]), __uint_as_float(a[c4 + 3]), c2, -l.z, -l.w);
      pv[c4] = x01.x;
      pv[c4 + 1] = x01.y;
      pv[c4 + 2] = x23.x;
      pv[c4 + 3] = x23.y;
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) pv[c] = ex2_approx(pv[c]);
    if ((CAUSAL && c_lo > 0) || i == wk.T64 - 1) {
      // queries of this warpgroup that the sequence has (S of those behind may be anything)
      const int c_hi = wk.n - i * C::BQ - 32 * w;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c < c_lo || c >= c_hi) pv[c] = 0.f;
    }
    if (!wk.dk) {
      uint32_t pb[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) pb[c] = pack_bf16x2(pv[2 * c], pv[2 * c + 1]);
      tmem_st16(tX + 32 * (g & 1), pb);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&sh.x_ready[g & 1]);
    }
  };

  // ---- phase B (dK items): dS^T = P^T o (dP^T - D) * scale into TMEM, bf16
  // CUT: a sequence's last query tile. (One test a tile, around the whole phase:
  // inside it keeps the compiler from overlapping the TMEM loads.)
  auto phase_b = [&](const Work<CAUSAL>& wk, int i, int g, int gk, auto cut) {
    wait_all(&sh.dp_full, gk & 1, WHERE_BWD_SOFTMAX);
    if (!alive) return;
    uint32_t dpv[32];
    tmem_ld32(tDP, dpv);
    tmem_ld_wait();
    uint32_t dk[16];
#pragma unroll
    for (int c4 = 0; c4 < 32; c4 += 4) {
      const float4 dd = *reinterpret_cast<const float4*>(ld_d + c4);
      const float2 g01 = ffma2_bcast_mul(__uint_as_float(dpv[c4]), __uint_as_float(dpv[c4 + 1]), sc, -dd.x, -dd.y);
      const float2 g23 = ffma2_bcast_mul(__uint_as_float(dpv[c4 + 2]), __uint_as_float(dpv[c4 + 3]), sc, -dd.z, -dd.w);
      const float2 ds01 = fmul2(make_float2(pv[c4], pv[c4 + 1]), g01);
      const float2 ds23 = fmul2(make_float2(pv[c4 + 2], pv[c4 + 3]), g23);
      dk[c4 / 2] = pack_bf16x2(ds01.x, ds01.y);
      dk[c4 / 2 + 1] = pack_bf16x2(ds23.x, ds23.y);
    }
    if constexpr (decltype(cut)::value) {
      // dP of queries behind the sequence's last may be infinite or NaN
      const int held = wk.n - i * C::BQ - 32 * w;
#pragma unroll
      for (int c = 0; c < 16; ++c) dk[c] &= (2 * c < held ? 0xFFFFu : 0u) | (2 * c + 1 < held ? 0xFFFF0000u : 0u);
    }
    tmem_st16(tX + 32 * (g & 1), dk);
    tmem_st_wait();
    tc_fence_before_sync();
    mbar_arrive(&sh.x_ready[g & 1]);
  };

  // ---- item epilogue: columns [128w, 128w + 128) of dK or dV; thread r writes key row
  // r (rows behind the sequence's last are skipped)
  auto epilogue = [&](const Work<CAUSAL>& wk, int items) {
    wait_all(&sh.acc_done, items & 1, WHERE_BWD_SOFTMAX);
    if (!alive) return;
    const int key = wk.j * 128 + r;
    const uint32_t t = tmem + lane_base + C::ACC_COL + 128 * w;
    const long long* st = wk.dk ? p.dk_strides : p.dv_strides;
    __nv_bfloat16* dst =
        (wk.dk ? p.dk : p.dv) + static_cast<long long>(wk.row0 + key) * st[0] + wk.bh * st[1] + 128 * w;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      tmem_ld32(t + c, v);
      tmem_ld_wait();
      if (c + 32 == 128) {  // the next item may overwrite the accumulator
        tc_fence_before_sync();
        mbar_arrive(&sh.acc_free);
      }
      if (key < wk.n) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(dst + c + 8 * u) =
              make_uint4(pack_bf16x2(__uint_as_float(v[8 * u + 0]), __uint_as_float(v[8 * u + 1])),
                         pack_bf16x2(__uint_as_float(v[8 * u + 2]), __uint_as_float(v[8 * u + 3])),
                         pack_bf16x2(__uint_as_float(v[8 * u + 4]), __uint_as_float(v[8 * u + 5])),
                         pack_bf16x2(__uint_as_float(v[8 * u + 6]), __uint_as_float(v[8 * u + 7])));
      }
    }
  };

  // The next work item, agreed on by the whole warpgroup (as in fa_bwd.cu).
  auto next_item = [&](int u) -> int {
    const int it = alive ? take_item(sh, u, lim) : -1;
    if (!named_barrier_and(bar_id, 128, it >= 0)) {
      if (alive) record_timeout(p.status, &sh.abort_flag, WHERE_BWD_SOFTMAX);
      alive = false;
      return total;
    }
    return it;
  };

  int g = 0, gk = 0, items = 0;
  int item = next_item(0);
  float ld = 0.f;
  if (item < total) {
    const Work<CAUSAL> wk0(item, p);
    const typename Work<CAUSAL>::Pos f0 = wk0.first();
    ld = fetch_ld(wk0, f0.bh, f0.i);
  }
  while (item < total) {
    const Work<CAUSAL> wk(item, p);
    const int n_iter = wk.n_iter();
    if (items > 0) named_barrier_sync(bar_id, 128);  // the previous item's L2 / D reads are done
    if (r < 64) ld_l2[r] = ld;
    named_barrier_sync(bar_id, 128);
    // the next tile's L2 and D land during phase A (a dV item has no phase B)
    typename Work<CAUSAL>::Pos cur = wk.first(), nxt = cur;
    wk.advance(nxt);
    float next_ld = n_iter > 1 ? fetch_ld(wk, nxt.bh, nxt.i) : 0.f;
    phase_a(wk, cur.i, g);
    for (int n = 0; n < n_iter; ++n) {
      const bool has_next = n + 1 < n_iter;
      if (wk.dk) {
        if (cur.i == wk.T64 - 1)
          phase_b(wk, cur.i, g + n, gk + n, std::true_type());
        else
          phase_b(wk, cur.i, g + n, gk + n, std::false_type());
      }
      if (has_next) {
        named_barrier_sync(bar_id, 128);  // every thread is done reading this tile's L2 / D
        if (r < 64) ld_l2[r] = next_ld;
        named_barrier_sync(bar_id, 128);
        cur = nxt;
        wk.advance(nxt);
        if (n + 2 < n_iter) next_ld = fetch_ld(wk, nxt.bh, nxt.i);
        phase_a(wk, cur.i, g + n + 1);
      }
    }
    const int item_next = next_item(items + 1);
    if (item_next < total) {
      const Work<CAUSAL> wk1(item_next, p);
      const typename Work<CAUSAL>::Pos f1 = wk1.first();
      ld = fetch_ld(wk1, f1.bh, f1.i);  // lands during the epilogue
    }
    epilogue(wk, items);
    g += n_iter;
    if (wk.dk) gk += n_iter;
    ++items;
    item = item_next;
  }
}

template <bool CAUSAL>
__global__ void __launch_bounds__(kThreads, 1) fa_bwd256_ragged_kernel(const __grid_constant__ BwdLaunch p) {
  using C = Cfg;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::KV_BYTES;
  uint8_t* sQ = sV + C::KV_BYTES;
  uint8_t* sdO = sQ + C::Q_SLOTS * C::Q_BYTES;
  float* sLD = reinterpret_cast<float*>(sdO + C::Q_BYTES);
  const int warp = threadIdx.x >> 5;
  // Launched to overlap the end of the kernel that forms D and L; lets the next one
  // start only when that is complete. It writes nothing the dQ kernel reads.
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= total_items(p)) return;  // no item is left for this CTA

  if (threadIdx.x == 0) {
    mbar_init(&sh.kv_full, 1);
    for (int s = 0; s < C::Q_SLOTS; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
      mbar_init(&sh.do_full[s], 1);
      mbar_init(&sh.do_empty[s], 1);
    }
    // test hook: the S or P barrier waits for one arrival too many
    mbar_init(&sh.s_full, 1 + debug_extra(p.debug_skip, WHERE_BWD_MMA));
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.s_read, 256);
    for (int b = 0; b < 2; ++b)
      mbar_init(&sh.x_ready[b], 256 + (b == 0 ? debug_extra(p.debug_skip, WHERE_BWD_SOFTMAX) : 0u));
    mbar_init(&sh.acc_done, 1);
    mbar_init(&sh.acc_free, 256);
    tail_init(sh.tail);
    mbar_init(&sh.mma_drain, 1);
    for (int s = 0; s < kItemSlots; ++s) {
      mbar_init(&sh.item_full[s], 1);
      mbar_init(&sh.item_empty[s], kItemConsumers);
    }
    sh.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem_base;

  if (warp == kLoadWarp) {
    if (lane_id() == 0) load_role<CAUSAL>(p, sh, sK, sV, sQ, sdO);
  } else if (warp == kMmaWarp) {
    if (lane_id() == 0) mma_role<CAUSAL>(p, sh, sK, sV, sQ, sdO, tmem);
  } else if (warp == kTailWarp) {
    tail_role<4, C::Q_CHUNK>(sh.tail, &sh.abort_flag, p.wait_limit_ns);
  } else {
    softmax_role<CAUSAL>(p, sh, sLD, tmem, warp >> 2);
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <bool CAUSAL>
cudaError_t launch_t(const BwdLaunch& a, cudaStream_t stream) {
  auto kern = fa_bwd256_ragged_kernel<CAUSAL>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, Cfg::SMEM_BYTES, a.device, done);
  if (e != cudaSuccess) return e;
  // The plan, on the device, knows how many items there are. Persistent: one CTA per SM.
  const long long items = static_cast<long long>(a.BHkv) * a.N * 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(items, a.num_sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_bwd_main_ragged256(const BwdLaunch& a, cudaStream_t stream) {
  return a.causal ? launch_t<true>(a, stream) : launch_t<false>(a, stream);
}

}  // namespace fa
