// dQ of the backward pass without atomics, for sm_103a.
//
// Method (web pages on FlashAttention-2): the reading note (papers.chlience.com)
// 5.3-5.4 and the paper-graph-ui summary, "The Backward Pass", accumulate
// dQ_i += dS_ij K_j across key blocks with atomic adds, so dQ is not bitwise
// reproducible. This kernel is the deterministic alternative: one work item
// owns query tile i of one head and loops over the key tiles itself, so dQ_i
// is summed on chip in a fixed order:
//   S = Q_i K_j^T, P = 2^(S scale log2e - L_i log2e), dP = dO_i V_j^T,
//   dS = P o (dP - D_i) * scale, dQ_i += dS K_j,
// with L and D from the preprocess kernel. The backward main kernel then runs
// without its dQ products and reductions, and computes only dK and dV.
//
// GB300 mapping: persistent, one CTA (320 threads) per SM taking items from a
// counter in the workspace (causal: the query tiles that see the most keys
// first). Warp 8 streams Q_i, dO_i once per item and K_j, V_j through two
// rings (K deeper: K_j is read by S(j) and, late, by the dQ product);
// warp 9 issues the MMAs (S and dP into TMEM, dQ accumulated in TMEM);
// warpgroups 0 and 1 own key columns [64w, 64w + 64) of every tile, thread r
// = query row r = TMEM lane r, so the row statistics L_r and D_r are
// per-thread scalars. P (bf16, the rounding the dV product of the main kernel
// uses) stays in registers; dS (bf16) is written back into the columns of
// its own tile's S buffer, already read, and is the TMEM A operand of
// dQ += dS K_j, with K_j as the MN-major B operand.
//
// TMEM columns (512 allocated): S buffers [0, 128) and [128, 256), dP
// [256, 384), dQ [384, 384 + d).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "fa_internal.h"
#include "fa_kernel_common.cuh"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 320;
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kTailWarp = 10;  // packed sequences alone; registers are dealt out for 12 warps either way
template <bool RAG>
constexpr int kernel_threads() {
  return RAG ? kThreads + 32 : kThreads;
}
constexpr int kItemConsumers = 1 + 256;  // the MMA thread and the softmax threads

template <int HD>
struct DqCfg {
  static constexpr int CHUNKS = HD / 64;
  static constexpr int TILE_BYTES = 128 * HD * 2;
  static constexpr int CHUNK_BYTES = 128 * 128;
  // K_j is read by S(j) early and by the dQ product late; V_j only by dP(j).
  // A deeper K ring lets S(j+1) start while K_j is still in use. d = 128:
  // 4 K stages and 1 V stage (the smem of 3 + 2 measured 1 % slower).
  static constexpr int KST = 4;                 // K_j ring stages
  static constexpr int VST = HD == 64 ? 2 : 1;  // V_j ring stages
  // S is double-buffered (tile t in buffer t & 1), so S(t+1) is computed
  // while the softmax still works on tile t.
  static constexpr uint32_t S_COL = 0, DP_COL = 256, DQ_COL = 384;
  __host__ __device__ static constexpr uint32_t s_col(int b) { return S_COL + 128u * uint32_t(b); }
  // smem: Q_i, dO_i, KST x K_j, VST x V_j (dS lives in TMEM)
  static constexpr int SMEM_BYTES = (2 + KST + VST) * TILE_BYTES + 1024;
};

struct DqShared {
  uint64_t q_full, q_free;
  uint64_t k_full[4], k_empty[4], v_full[2], v_empty[2];
  TailShared tail;  // packed sequences
  uint64_t s_full[2];  // per S buffer
  // ds_ready[t & 1]: dS(t) is in TMEM. Two barriers, because the softmax can
  // finish tile t+1 (it needs only dP(t+1), issued before the MMA thread
  // waits for dS(t)) before that wait starts: on one barrier the wait would
  // then see two completed phases and take the pending third for its own.
  // Tile t+2 needs dP(t+2), issued after the wait, so one barrier per tile
  // parity can be at most one phase ahead of its waiter.
  uint64_t dp_full, dp_free, ds_ready[2], dq_done, acc_done, acc_free;
  uint64_t mma_drain;  // the MMA thread's last commit: all its MMAs done before the CTA exits
  uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  int item_ring[kItemSlots];
  uint32_t tmem_base;
  int abort_flag;
};

// Work item: query tile i of query head bh; key tiles 0 .. nkv-1 (causal:
// the tiles up to the diagonal). Causal items are numbered most-work-first;
// non-causal items of one head are adjacent (K/V reuse in L2).
template <bool CAUSAL, bool RAG>
struct DqWork {
  int bh, i, nkv;
  static constexpr int row0 = 0;  // the sequence's first row
  __device__ __forceinline__ int len(const BwdLaunch& p) const { return p.N; }
  __device__ DqWork(int item, const BwdLaunch& p) {
    const int BH = p.BH, N = p.N;
    const int T = (N + 127) / 128;
    if (CAUSAL) {
      i = T - 1 - item / BH;
      bh = item % BH;
      nkv = i + 1;
    } else {
      bh = item / T;
      i = item % T;
      nkv = T;
    }
  }
};

// The same over packed sequences: an entry of the plan's list is a sequence's
// query tile, every query head of it an item.
template <bool CAUSAL>
struct DqWork<CAUSAL, true> {
  int bh, i, nkv, row0, n;
  __device__ __forceinline__ int len(const BwdLaunch&) const { return n; }
  __device__ DqWork(int item, const BwdLaunch& p) {
    const int e = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(p.BH));
    const int4 x = __ldg(packed_tiles(p.plan) + e);
    bh = item - e * p.BH;
    row0 = x.x;
    n = x.y;
    i = x.z;
    nkv = CAUSAL ? i + 1 : (n + 127) >> 7;
  }
};

template <bool RAG>
__device__ __forceinline__ int dq_total_items(const BwdLaunch& p) {
  if constexpr (RAG)
    return packed_plan_ok(p.plan, p.N) ? (p.plan->n_tiles - p.plan->n_short) * p.BH : 0;
  else
    return p.BH * ((p.N + 127) / 128);
}

// TMA producer (one thread): Q_i and dO_i once per item, after the previous
// item's last S and dP products have read them; K_j, V_j through the ring.
template <int HD, bool CAUSAL, bool RAG>
__device__ void dq_load_role(const BwdLaunch& p, DqShared& sh, uint8_t* sQ, uint8_t* sdO, uint8_t* sK,
                             uint8_t* sV) {
  using C = DqCfg<HD>;
  tma_prefetch_desc(&p.tmQ);
  tma_prefetch_desc(&p.tmdO);
  tma_prefetch_desc(&p.tmK);
  tma_prefetch_desc(&p.tmV);
  const int total = dq_total_items<RAG>(p);
  const uint64_t lim = p.wait_limit_ns;
  int u = 0, kv = 0, q_issued = 0;  // kv: K/V tiles loaded
  bool k_extra = false;              // K of tile kv issued, its V not (abort in between)
  bool aborted = false;
  auto load_kv = [&](int row, int kvh) -> bool {
    const int ks = kv % C::KST, vs = kv % C::VST;
    if (kv >= C::KST && !mbar_wait(&sh.k_empty[ks], ((kv / C::KST) - 1) & 1, &sh.abort_flag, lim)) return false;
    mbar_arrive_expect_tx(&sh.k_full[ks], C::TILE_BYTES);
#pragma unroll
    for (int c = 0; c < C::CHUNKS; ++c)
      tma_load_3d(sK + ks * C::TILE_BYTES + c * C::CHUNK_BYTES, &p.tmK, &sh.k_full[ks], c * 64, row, kvh);
    k_extra = true;
    if (kv >= C::VST && !mbar_wait(&sh.v_empty[vs], ((kv / C::VST) - 1) & 1, &sh.abort_flag, lim)) return false;
    mbar_arrive_expect_tx(&sh.v_full[vs], C::TILE_BYTES);
#pragma unroll
    for (int c = 0; c < C::CHUNKS; ++c)
      tma_load_3d(sV + vs * C::TILE_BYTES + c * C::CHUNK_BYTES, &p.tmV, &sh.v_full[vs], c * 64, row, kvh);
    ++kv;
    k_extra = false;
    return true;
  };
  int item = blockIdx.x;
  while (!aborted) {
    if (!publish_item(sh, u, item, lim)) {
      aborted = true;
      break;
    }
    if (item >= total) break;
    const DqWork<CAUSAL, RAG> wk(item, p);
    const int kvh = wk.bh / p.group;  // grouped K/V heads
    // The first K/V tile loads while the previous item still reads Q_i, dO_i.
    if (!load_kv(wk.row0, kvh) || (u > 0 && !mbar_wait(&sh.q_free, (u - 1) & 1, &sh.abort_flag, lim))) {
      aborted = true;
      break;
    }
    if (!debug_skip_here(p.debug_skip, WHERE_BWD_LOAD, u == 0)) {  // test hook
      mbar_arrive_expect_tx(&sh.q_full, 2 * C::TILE_BYTES);
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c) {
        tma_load_3d(sQ + c * C::CHUNK_BYTES, &p.tmQ, &sh.q_full, c * 64, wk.row0 + wk.i * 128, wk.bh);
        tma_load_3d(sdO + c * C::CHUNK_BYTES, &p.tmdO, &sh.q_full, c * 64, wk.row0 + wk.i * 128, wk.bh);
      }
      ++q_issued;
    }
    for (int j = 1; j < wk.nkv && !aborted; ++j) aborted = !load_kv(wk.row0 + j * 128, kvh);
    ++u;
    if (!aborted) item = claim_item(p.sched + 2);
  }
  finish_claiming(p.sched + 2);
  if (aborted) record_timeout(p.status, &sh.abort_flag, WHERE_BWD_LOAD);
  // The copies already issued land before the CTA can exit (after an abort
  // no consumer may wait for them). An aborted load_kv may have issued K_j
  // without V_j: kv counts only tiles whose K and V were both issued. Each
  // slot waits for the latest phase issued into it only (an older phase of a
  // slot can no longer be told apart once a newer one has completed).
  const int k_last = k_extra ? kv : kv - 1;
  for (int n = std::max(0, k_last - C::KST + 1); n <= k_last; ++n)
    drain_wait(&sh.k_full[n % C::KST], (n / C::KST) & 1, lim);
  for (int n = std::max(0, kv - C::VST); n < kv; ++n) drain_wait(&sh.v_full[n % C::VST], (n / C::VST) & 1, lim);
  if (q_issued > 0) drain_wait(&sh.q_full, (q_issued - 1) & 1, lim);
}

// One thread issues every MMA. Per key tile j (global tile t):
//   S(t+1)   into the other S buffer once K_{j+1} is in and the dQ product
//            of tile t-1 (whose dS sat there) is done (overlaps A(t), B(t))
//   dP(t+1)  once phase B(t) has read dP(t)        (overlaps the rest of B(t))
//   dQ += dS(t) K_j   once phase B(t) wrote dS(t)  (overlaps phase A(t+1))
template <int HD, bool CAUSAL, bool RAG>
__device__ void dq_mma_role(const BwdLaunch& p, DqShared& sh, uint8_t* sQ, uint8_t* sdO, uint8_t* sK, uint8_t* sV,
                            uint32_t tmem) {
  using C = DqCfg<HD>;
  constexpr uint32_t kIdescSq = make_idesc_bf16_f32(128, 128, false, false);  // S, dP: A, B K-major
  constexpr uint32_t kIdescDq = make_idesc_bf16_f32(128, HD, false, true);    // A = dS (TMEM), B = K_j MN-major
  const uint32_t q_addr = smem_u32(sQ), do_addr = smem_u32(sdO), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
  const uint64_t lim = p.wait_limit_ns;
  const int total = dq_total_items<RAG>(p);

  // D[tmem] = A (128 x HD, K-major) * B (128 x HD, K-major)^T
  auto issue_sq = [&](uint32_t d_col, uint32_t a_addr, uint32_t b_addr) {
    const uint64_t ad = make_smem_desc_sw128(a_addr, 16, 1024), bd = make_smem_desc_sw128(b_addr, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks) {
      const uint32_t off = (ks >> 2) * C::CHUNK_BYTES + (ks & 3) * 32;
      umma_ss(tmem + d_col, desc_add(ad, off), desc_add(bd, off), kIdescSq, ks > 0 ? 1u : 0u);
    }
  };
  auto fail = [&]() {
    record_timeout(p.status, &sh.abort_flag, WHERE_BWD_MMA);
    drain_mmas(&sh.mma_drain, lim);
  };

  // S(t) into buffer t & 1, which tile t - 2 used.
  // done_tile: the latest dQ product issued (tile t - 2 inside an item, t - 1
  // at an item's start); its completion implies that of every earlier one,
  // including the product of tile t - 2 whose dS sat in buffer t & 1.
  auto issue_s = [&](int t, int kvi, int done_tile) -> bool {  // kvi: the tile's index in the K/V stream
    const int stage = kvi % C::KST;
    if (!mbar_wait(&sh.k_full[stage], (kvi / C::KST) & 1, &sh.abort_flag, lim)) return false;
    if (t >= 2 && !mbar_wait(&sh.dq_done, done_tile & 1, &sh.abort_flag, lim)) return false;
    tc_fence_after_sync();
    issue_sq(C::s_col(t & 1), q_addr, k_addr + stage * C::TILE_BYTES);
    umma_commit(&sh.s_full[t & 1]);
    return true;
  };
  // dP(t) over dP(t - 1): wait until phase B(t - 1) loaded it.
  auto issue_dp = [&](int t, int kvi) -> bool {
    const int stage = kvi % C::VST;
    if (!mbar_wait(&sh.v_full[stage], (kvi / C::VST) & 1, &sh.abort_flag, lim)) return false;
    if (t >= 1 && !mbar_wait(&sh.dp_free, (t - 1) & 1, &sh.abort_flag, lim)) return false;
    tc_fence_after_sync();
    issue_sq(C::DP_COL, do_addr, v_addr + stage * C::TILE_BYTES);
    umma_commit(&sh.dp_full);
    umma_commit(&sh.v_empty[stage]);  // V_j is read by dP(j) only
    return true;
  };

  int u = 0, kv = 0, t = 0;
  TailCalls<false> tail;
  while (true) {
    const int item = take_item(sh, u, lim);
    if (item < 0) return fail();
    if (item >= total) break;
    const DqWork<CAUSAL, RAG> wk(item, p);
    if (!mbar_wait(&sh.q_full, u & 1, &sh.abort_flag, lim) || !issue_s(t, kv, t - 1) ||
        !issue_dp(t, kv))
      return fail();
    if (wk.nkv == 1) umma_commit(&sh.q_free);
    // Per tile t: S(t+1) as soon as its K tile is in, dP(t+1) once phase B(t)
    // has read dP(t), dQ += dS(t) K once phase B(t) has written dS(t).
    // LAST: the item's last tile, which over packed sequences may end in rows of the
    // next sequence (see the forward).
    auto step = [&](int j, auto last_tile) -> bool {
      constexpr bool LAST = decltype(last_tile)::value;
      const int s = kv % C::KST;
      if (RAG ? !LAST : j + 1 < wk.nkv) {
        if (!issue_s(t + 1, kv + 1, t - 1) || !issue_dp(t + 1, kv + 1)) return false;
        if (j + 2 == wk.nkv) umma_commit(&sh.q_free);  // the item's last S and dP are issued
      }
      int steps = 8;  // of 16 keys
      if (RAG && LAST && wk.len(p) - j * 128 < 128) {  // once S(t) has read K_j
        steps = (wk.len(p) - j * 128 + 15) >> 4;
        if (!mbar_wait(&sh.s_full[t & 1], (t >> 1) & 1, &sh.abort_flag, lim)) return false;
        tail.ask(sh.tail, wk.len(p) - j * 128, k_addr + s * C::TILE_BYTES);
      }
      if (!mbar_wait(&sh.ds_ready[t & 1], (t >> 1) & 1, &sh.abort_flag, lim)) return false;
      if (RAG && LAST && !tail.wait(sh.tail, &sh.abort_flag, lim)) return false;
      // the first dQ product of an item overwrites the accumulator: the
      // previous item's epilogue must have read it
      if (j == 0 && u > 0 && !mbar_wait(&sh.acc_free, (u - 1) & 1, &sh.abort_flag, lim)) return false;
      tc_fence_after_sync();
      // dS (bf16 pairs) sits in columns [0, 32) and [64, 96) of S buffer t & 1:
      // keys 16 ks .. 16 ks + 15 are 8 columns at 64 (ks / 4) + 8 (ks % 4)
      const uint64_t kd = make_smem_desc_sw128(k_addr + s * C::TILE_BYTES, C::CHUNK_BYTES, 1024);
      issue_steps<8, RAG && LAST>(steps, [&](int ks) {
        umma_ts(tmem + C::DQ_COL, tmem + C::s_col(t & 1) + (ks >> 2) * 64 + (ks & 3) * 8, desc_add(kd, ks * 2048),
                kIdescDq, (j > 0 || ks > 0) ? 1u : 0u);
      });
      umma_commit(&sh.dq_done);
      umma_commit(&sh.k_empty[s]);
      return true;
    };
    for (int j = 0; j < wk.nkv; ++j, ++kv, ++t)
      if (!(RAG && j + 1 < wk.nkv ? step(j, std::false_type()) : step(j, std::true_type()))) return fail();
    umma_commit(&sh.acc_done);
    ++u;
  }
  // Normally the epilogues have waited for the last products; if a softmax
  // warpgroup gave up, nothing has.
  if (RAG) tail.finish(sh.tail);
  drain_mmas(&sh.mma_drain, lim);
}

// Warpgroup w owns key columns [64w, 64w + 64) of every tile; thread r owns
// query row r. Phase A: P = 2^(S scale log2e - L2_r) (bf16-rounded, kept in
// registers). Phase B: dS = P o (dP scale - D_r scale) into the dS tile. At
// the end of an item warpgroup w writes dQ columns [w d/2, (w+1) d/2).
template <int HD, bool CAUSAL, bool RAG>
__device__ void dq_softmax_role(const BwdLaunch& p, DqShared& sh, uint32_t tmem, int w) {
  using C = DqCfg<HD>;
  const int r = threadIdx.x & 127;
  const uint32_t lane_base = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
  const float c2 = p.scale_log2;
  const float sc = p.scale;
  const uint64_t lim = p.wait_limit_ns;
  const uint32_t tS0 = tmem + lane_base + C::S_COL + 64 * w;  // + 128 for buffer 1
  const uint32_t tDP = tmem + lane_base + C::DP_COL + 64 * w;
  const uint32_t bar_id = 1 + w;
  const int total = dq_total_items<RAG>(p);
  bool alive = true;
  // P of the current tile, bf16 pairs; over packed sequences fp32 (8 sequences of 2149 to
  // 3800 rows, 16 + 4 heads, d = 64: 811 us with dK and dV, half of them by pairs of 16 bits 828)
  Weights<64, RAG> pk;

  auto wait_all = [&](uint64_t* bar, int parity, int where) {
    alive = alive && __all_sync(0xffffffffu, mbar_wait(bar, parity, &sh.abort_flag, lim));
    if (!alive) record_timeout(p.status, &sh.abort_flag, where);
    tc_fence_after_sync();
  };
  // The next work item, agreed on by the whole warpgroup (see the main kernel).
  auto next_item = [&](int u) -> int {
    const int it = alive ? take_item(sh, u, lim) : -1;
    if (!named_barrier_and(bar_id, 128, it >= 0)) {
      if (alive) record_timeout(p.status, &sh.abort_flag, WHERE_BWD_SOFTMAX);
      alive = false;
      return total;
    }
    return it;
  };

  int u = 0, t = 0;
  int item = next_item(0);
  while (item < total) {
    const DqWork<CAUSAL, RAG> wk(item, p);
    const int row = wk.i * 128 + r;
    const bool held = !RAG || row < wk.len(p);
    // (D and L through the read-only path: the pass before this one has waited for the
    // kernel that writes them before it let this grid start.)
    const size_t srow = RAG ? static_cast<size_t>(wk.bh) * p.N + wk.row0 + row : static_cast<size_t>(wk.bh) * p.Npad + row;
    const float l2 = held ? __ldg(p.lse2 + srow) : INFINITY;  // +inf on padding rows: their P is 0
    const float dsc = held ? __ldg(p.D + srow) * sc : 0.f;
    for (int j = 0; j < wk.nkv; ++j, ++t) {
      // ---- phase A
      wait_all(&sh.s_full[t & 1], (t >> 1) & 1, WHERE_BWD_SOFTMAX);
      if (alive) {
        float pv[64];
        {
          const uint32_t tS = tS0 + 128u * uint32_t(t & 1);
          uint32_t a[32], b[32];
          tmem_ld32(tS, a);
          tmem_ld32(tS + 32, b);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            pv[c] = __uint_as_float(a[c]);
            pv[32 + c] = __uint_as_float(b[c]);
          }
        }

        // key 128j + 64w + c is seen if it is < N and (causal) <= the query row
        const int kbase = j * 128 + 64 * w;
        int c_hi = std::min(64, wk.len(p) - kbase);
        if (CAUSAL && j == wk.i) c_hi = std::min(c_hi, r - 64 * w + 1);
        const bool masked = c_hi < 64;
#pragma unroll
        for (int c4 = 0; c4 < 64; c4 += 4) {
          const float2 x01 = ffma2_bcast(pv[c4], pv[c4 + 1], c2, -l2);
          const float2 x23 = ffma2_bcast(pv[c4 + 2], pv[c4 + 3], c2, -l2);
          pv[c4] = ex2_approx(x01.x);
          pv[c4 + 1] = ex2_approx(x01.y);
          pv[c4 + 2] = ex2_approx(x23.x);
          pv[c4 + 3] = ex2_approx(x23.y);
          if (masked) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (c4 + q >= c_hi) pv[c4 + q] = 0.f;
          }
          pk.put(c4, pv[c4], pv[c4 + 1]);
          pk.put(c4 + 2, pv[c4 + 2], pv[c4 + 3]);
        }
      }
      // ---- phase B: dS into the first 32 columns of this warpgroup's half of
      // S buffer t & 1 (phase A has read them)
      wait_all(&sh.dp_full, t & 1, WHERE_BWD_SOFTMAX);
      if (alive) {
        // over packed sequences a half at a time (4 of 1197 to 7129 rows, d = 128: 1636 -> 1626 us)
        uint32_t ds[RAG ? 16 : 32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t dpv[32];
          tmem_ld32(tDP + 32 * h, dpv);
          tmem_ld_wait();
          if (h == 1) {
            tc_fence_before_sync();
            mbar_arrive(&sh.dp_free);
          }
#pragma unroll
          for (int c4 = 0; c4 < 32; c4 += 4) {
            const float2 p01 = pk.get(32 * h + c4);
            const float2 p23 = pk.get(32 * h + c4 + 2);
            const float2 g01 = ffma2_bcast(__uint_as_float(dpv[c4]), __uint_as_float(dpv[c4 + 1]), sc, -dsc);
            const float2 g23 = ffma2_bcast(__uint_as_float(dpv[c4 + 2]), __uint_as_float(dpv[c4 + 3]), sc, -dsc);
            const float2 d01 = fmul2(p01, g01);
            const float2 d23 = fmul2(p23, g23);
            ds[(RAG ? 0 : 16 * h) + c4 / 2] = pack_bf16x2(d01.x, d01.y);
            ds[(RAG ? 0 : 16 * h) + c4 / 2 + 1] = pack_bf16x2(d23.x, d23.y);
          }
          if constexpr (RAG) {
            // dP of keys behind the sequence's last may be infinite or NaN
            const int keys = wk.len(p) - j * 128 - 64 * w - 32 * h;
            if (keys < 32) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                ds[c] &= (2 * c < keys ? 0xFFFFu : 0u) | (2 * c + 1 < keys ? 0xFFFF0000u : 0u);
            }
            tmem_st16(tS0 + 128u * uint32_t(t & 1) + 16 * h, ds);
          }
        }
        if constexpr (!RAG) tmem_st32(tS0 + 128u * uint32_t(t & 1), ds);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&sh.ds_ready[t & 1]);
      }
    }
    const int item_next = next_item(u + 1);
    // ---- epilogue: dQ (fp32, TMEM) -> bf16 -> dq; rows past N are skipped
    wait_all(&sh.acc_done, u & 1, WHERE_BWD_SOFTMAX);
    if (alive) {
      const uint32_t tq = tmem + lane_base + C::DQ_COL + w * (HD / 2);
      __nv_bfloat16* dst = p.dq + w * (HD / 2);
      if constexpr (RAG)
        dst += static_cast<long long>(wk.row0 + row) * p.dq_strides[0] + wk.bh * p.dq_strides[1];
      else
        dst += (static_cast<size_t>(wk.bh) * p.N + row) * HD;
#pragma unroll
      for (int c = 0; c < HD / 2; c += 32) {
        uint32_t v[32];
        tmem_ld32(tq + c, v);
        tmem_ld_wait();
        if (c + 32 == HD / 2) {  // the next item may overwrite the accumulator
          tc_fence_before_sync();
          mbar_arrive(&sh.acc_free);
        }
        if (row < wk.len(p)) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(dst + c + 8 * q) =
                make_uint4(pack_bf16x2(__uint_as_float(v[8 * q + 0]), __uint_as_float(v[8 * q + 1])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
        }
      }
    }
    ++u;
    item = item_next;
  }
}

template <int HD, bool CAUSAL, bool RAG>
__global__ void __launch_bounds__(kernel_threads<RAG>(), 1) fa_bwd_dq_kernel(const __grid_constant__ BwdLaunch p) {
  using C = DqCfg<HD>;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ DqShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sdO = sQ + C::TILE_BYTES;
  uint8_t* sK = sdO + C::TILE_BYTES;
  uint8_t* sV = sK + C::KST * C::TILE_BYTES;
  const int warp = threadIdx.x >> 5;
  if (RAG) griddep_launch_dependents();  // the kernel that joins a split group's sums
  if (RAG && static_cast<int>(blockIdx.x) >= dq_total_items<RAG>(p)) {  // no item is left for this CTA
    if (blockIdx.x == 0 && threadIdx.x == 0) griddep_wait();
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_free, 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    // test hook: buffer 0's S or dS barrier waits for one arrival too many
    for (int b = 0; b < 2; ++b) mbar_init(&sh.s_full[b], 1 + (b == 0 ? debug_extra(p.debug_skip, WHERE_BWD_MMA) : 0u));
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.dp_free, 256);
    for (int b = 0; b < 2; ++b)
      mbar_init(&sh.ds_ready[b], 256 + (b == 0 ? debug_extra(p.debug_skip, WHERE_BWD_SOFTMAX) : 0u));
    mbar_init(&sh.dq_done, 1);
    mbar_init(&sh.acc_done, 1);
    mbar_init(&sh.acc_free, 256);
    if (RAG) tail_init(sh.tail);
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
    if (lane_id() == 0) dq_load_role<HD, CAUSAL, RAG>(p, sh, sQ, sdO, sK, sV);
  } else if (warp == kMmaWarp) {
    if (lane_id() == 0) dq_mma_role<HD, CAUSAL, RAG>(p, sh, sQ, sdO, sK, sV, tmem);
  } else if (RAG && warp == kTailWarp) {
    tail_role<C::CHUNKS, C::CHUNK_BYTES>(sh.tail, &sh.abort_flag, p.wait_limit_ns);
  } else {
    dq_softmax_role<HD, CAUSAL, RAG>(p, sh, tmem, warp >> 2);
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  // Launched to overlap the dK/dV pass (overlap_prev), this grid must not
  // complete before that pass has: work queued after it may read dK and dV. (Over
  // packed sequences one block waits and the others leave their SMs.)
  if ((!RAG || blockIdx.x == 0) && threadIdx.x == 0) griddep_wait();
}

template <int HD, bool CAUSAL, bool RAG = false>
cudaError_t launch_t(const BwdLaunch& a, cudaStream_t stream) {
  using C = DqCfg<HD>;
  auto kern = fa_bwd_dq_kernel<HD, CAUSAL, RAG>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = RAG ? allow_smem(kern, C::SMEM_BYTES, a.device, done)
                      : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  // Packed sequences: the plan, on the device, knows how many items there are.
  const long long items = static_cast<long long>(a.BH) * (RAG ? a.N : (a.N + 127) / 128);
  const long long grid = items < a.num_sms ? items : a.num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kernel_threads<RAG>());
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.overlap_prev ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_bwd_dq(const BwdLaunch& a, cudaStream_t stream) {
  if (a.plan && a.d == 64) return a.causal ? launch_t<64, true, true>(a, stream) : launch_t<64, false, true>(a, stream);
  if (a.plan && a.d == 128) return a.causal ? launch_t<128, true, true>(a, stream) : launch_t<128, false, true>(a, stream);
  switch (a.d) {
    case 64: return a.causal ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
    case 128: return a.causal ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
    case 256: return launch_bwd_dq256(a, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace fa
