// The plan of a batch of packed sequences (fa_packed_plan of fa.h): what the
// attention kernels read of it.
#pragma once

#include <cstdint>

#include "fa_kernel_common.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// Head of the plan in device memory. Behind it lie two lists of {first row of
// the sequence, its length, index in it, 0}: the sequences' 128-row tiles, and
// their pairs of neighbouring tiles. Both are ordered by the work of a query
// tile, most first: the key tiles it sees, which are index + 1 of a causal plan
// and all the sequence's else. (A causal key tile sees what is behind it, so
// the same list read with j = last - index is ordered for them too.) Sequences of
// kShortRows rows or fewer stand at the end of both lists.
struct PackedPlan {
  uint32_t magic;
  int rows;               // rows of the tensors it was made for
  int n_tiles, n_pairs;
  int n_short;            // sequences at the end of either list
  int pairs_at;           // first entry of the second list
  int max_tiles;          // tiles of the longest sequence
  int row_begin, row_end; // rows that belong to a sequence
  unsigned long long causal_products, full_products;  // (query tile, key tile) pairs per head
};
constexpr int kShortRows = 64;  // up to here a sequence is fa_packed_short.cu's
constexpr uint32_t kPackedMagic = 0x46415031u;
constexpr int kPackedHead = 256;  // bytes before the lists

__device__ __forceinline__ const int4* packed_tiles(const PackedPlan* p) {
  return reinterpret_cast<const int4*>(reinterpret_cast<const uint8_t*>(p) + kPackedHead);
}
__device__ __forceinline__ const int4* packed_pairs(const PackedPlan* p) { return packed_tiles(p) + p->pairs_at; }

// A plan that was never made, or made for other tensors, has no work.
__device__ __forceinline__ bool packed_plan_ok(const PackedPlan* p, int rows) {
  return p->magic == kPackedMagic && p->rows == rows;
}

// ---------------------------------------------------------------------------
// Backward: a thread's N weights P of a tile that dS = P (dP - D) takes stay in
// registers between the two phases of the tile. The dense kernels keep the bf16 pairs
// that the dV product reads; over packed sequences they stay in fp32, without that
// second rounding, which is as large as dS's own (with it the gradients of random
// inputs are 0.28% off in the mean, so 0.24%).
// ---------------------------------------------------------------------------
template <int N, bool RAG>
struct Weights {
  uint32_t two[RAG ? 1 : N / 2];
  float one[RAG ? N : 1];
  // columns c and c + 1 (c even, known to the compiler)
  __device__ __forceinline__ void put(int c, float a, float b) {
    if constexpr (RAG) {
      one[c] = a;
      one[c + 1] = b;
    } else {
      two[c / 2] = pack_bf16x2(a, b);
    }
  }
  __device__ __forceinline__ float2 get(int c) const {
    if constexpr (RAG) return make_float2(one[c], one[c + 1]);
    else return unpack_bf16x2(two[c / 2]);
  }
};

// ---------------------------------------------------------------------------
// A sequence's last tile ends in rows of the next one, whatever they hold. Where
// a tile's rows are the summed dimension of a product, whole steps of 16 rows
// behind the sequence are left out of it, and those in the last step taken are
// cleared (their weights are 0, but 0 * NaN): the MMA thread asks a warp of its
// own for that as soon as the tile is in, and waits for it before the product
// (most often behind a wait for the softmax). The warp sleeps in between. (The
// whole MMA warp walking the items and clearing rows itself cost 15% of the
// forward's time at 8192 keys, a clearing warp that is a consumer of every tile 3%.)
// ---------------------------------------------------------------------------
struct TailShared {
  uint64_t asked, done;
  uint32_t tile[2];  // addresses of the tiles to clear (0: none)
  int held;          // their rows that stay; 0 ends the warp
};

__device__ __forceinline__ void tail_init(TailShared& t) {
  mbar_init(&t.asked, 1);
  mbar_init(&t.done, 1);
}

// The clearing warp. A wait for the next request is no sign of a failure however
// long it takes: the MMA thread's own waits are bounded, and it ends with a last
// request or with the abort flag. The number of waits is bounded all the same.
// ALL_ROWS: 0, or the rows of a tile, all of which from the sequence's end on are cleared.
template <int CHUNKS, int CHUNK_BYTES, int ALL_ROWS = 0>
__device__ void tail_role(TailShared& t, const int* abort_flag, uint64_t lim) {
  constexpr int kMostWaits = 1 << 16;
  for (int n = 0, waits = 0; waits < kMostWaits;) {
    if (!__all_sync(0xffffffffu, mbar_wait(&t.asked, n & 1, abort_flag, drain_limit(lim)))) {
      if (__any_sync(0xffffffffu, *reinterpret_cast<const volatile int*>(abort_flag))) return;
      ++waits;
      continue;
    }
    const int held = *reinterpret_cast<volatile int*>(&t.held);
    if (held == 0) return;
    const int units = ((ALL_ROWS ? ALL_ROWS : (held + 15) & ~15) - held) * 8;  // of 16 bytes, in a chunk
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t tile = *reinterpret_cast<volatile uint32_t*>(&t.tile[k]);
      for (int i = lane_id(); tile && i < units; i += 32)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) st_shared_v4(tile + c * CHUNK_BYTES + held * 128 + i * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();  // the tensor core sees the zeros
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&t.done);
    ++n;
  }
}

// The MMA thread's side: ask, and wait until it is done. A tile whose last step
// is whole asks for nothing unless all rows are cleared.
template <bool ALL>
struct TailCalls {
  int asked = 0;
  bool open = false;
  __device__ __forceinline__ void ask(TailShared& t, int held, uint32_t tile0, uint32_t tile1 = 0) {
    if (!ALL && !(held & 15)) return;
    *reinterpret_cast<volatile uint32_t*>(&t.tile[0]) = tile0;
    *reinterpret_cast<volatile uint32_t*>(&t.tile[1]) = tile1;
    *reinterpret_cast<volatile int*>(&t.held) = held;
    mbar_arrive(&t.asked);
    ++asked;
    open = true;
  }
  __device__ __forceinline__ bool wait(TailShared& t, const int* abort_flag, uint64_t lim) {
    if (!open) return true;
    open = false;
    return mbar_wait(&t.done, (asked - 1) & 1, abort_flag, lim);
  }
  __device__ __forceinline__ void finish(TailShared& t) {
    *reinterpret_cast<volatile int*>(&t.held) = 0;
    mbar_arrive(&t.asked);
  }
};

// The MMAs of a product over N steps, of which a sequence's last tile takes only
// `steps`: the whole product stays one run of issues (a test before each of them
// cost the MMA thread 12% of the forward's time).
template <int N, bool RAG, class Issue>
__device__ __forceinline__ void issue_steps(int steps, Issue issue) {
  if (!RAG || steps == N) {
#pragma unroll
    for (int ks = 0; ks < N; ++ks) issue(ks);
  } else {
#pragma unroll 1
    for (int ks = 0; ks < steps; ++ks) issue(ks);
  }
}

}  // namespace fa
