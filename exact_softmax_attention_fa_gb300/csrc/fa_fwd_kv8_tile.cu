// Attention over the paged 8-bit cache for many query rows per K/V head: chunks
// of a prompt, on tcgen05 (fa_fwd_kv8.cu has the mathematics and the kernel for
// few rows).
//
// A CTA holds blocks of up to two tiles of 128 query rows (rows of a K/V head's
// group, position by position) and streams 128-key tiles of the cache past them,
// as the dense forward does; what differs is how the codes reach the tensor core:
//   S = Q K^T  : kind::f8f6f4. K's codes are the operand as TMA brings them. A
//       query row, moved by a power of two so that its largest |value| lies in
//       [2^7, 2^8), is the sum of two e4m3 pieces qh + ql, accumulated into the
//       same S: exact for values down to 2^-9 of the row's largest, within
//       2^-17 of it below. Two e4m3 products cost what one fp16 product would,
//       and K needs no conversion and half the shared memory.
//   O += P V   : kind::f16. A weight keeps fp16's 2^-11 and range (small weights
//       of a long row together matter, and e4m3 pieces end at 2^-17 of the
//       largest), so V's codes, exact in fp16, are converted by a warpgroup
//       of their own from a staging ring into the swizzled operand tile.
// Key and value scales enter as in fa_fwd_kv8.cu: u = c sk (q . k8) + log2 sv per
// 16-key group, P = 2^(u - m), l = sum P / sv.
//
// Roles: warpgroups 0 and 1 Q pieces, softmax, correction and epilogue of one
// slot each, warpgroup 2 converts V, warp 12 looks up pages and loads, one thread
// each of warps 13 and 14 issues the MMAs of a slot. A slot is a tile of 128 rows;
// where the rows of a K/V head fill only one (decoding a few tokens of a group),
// both slots take it with every other key tile each, and the CTA joins them
// (128 rows, B = 8, Hkv = 8, 16384 keys, d = 128: 129 us with one slot, 97 so).
// d = 256 has tensor memory for one slot.
//
// Softmax steps are 64 keys, with two buffers of S per slot: S(f + 1) is formed
// beside the softmax of step f, so a slot waits for neither product. (128-key steps
// with one buffer: the chain S, softmax, PV of a slot bound, 232 us for 1024 queries
// on 16384 keys, B = 2, 16 heads on 4, d = 128; now 208. One thread issuing for
// both slots: 369, it spends more time between MMAs than the steps leave it.)
//
// Bound: shared memory, at that size at 0.60 of the tensor rate (1160 TFLOP/s). Two
// slots take some 3600 cycles for 128 keys. The tensor core alone would take 2477
// (measured; 2049 with 128-column S, for which tensor memory has no second buffer),
// and reads operands for 59% of the time (a 64-column S: 6 KB per 48 cycles);
// loads, stores and tensor-memory reads take the same memory for 27%. A CTA's
// fixed work (the search for its run, Q pieces, the epilogue) takes 8 us of a small
// call's 21 (32 rows of 8 heads against 4096 keys).
//
// Work: every CTA takes an equal run of the flattened list of (sequence, K/V
// head, row block, key tile); a row block that CTAs share is joined by
// kv8_tile_combine_kernel. So neither ragged lengths nor few row blocks against
// long caches leave SMs idle.
#include <algorithm>
#include <cmath>
#include <utility>

#include "fa_kv8.cuh"
#include "fa_kv8_attn.cuh"

namespace fa {
namespace {

constexpr int kThreads = 480;
constexpr int kConvThreads = 128;
constexpr int kLoadWarp = 12, kMmaWarp = 13;
constexpr int kMinTiles = 2;    // a CTA's run is not cut below this, but where blocks have fewer tiles
constexpr float kSlack = 8.f;   // P <= 2^(kShift + kSlack) = 2^14, fp16
template <int D>
struct TileCfg {
  static constexpr int NT = D <= 128 ? 2 : 1;     // slots
  static constexpr int ROWS = NT * 128;
  static constexpr int Q_BYTES = 2 * 128 * D;     // two pieces of a query tile
  static constexpr int K_BYTES = 128 * D;         // codes of a key tile
  static constexpr int V_BYTES = 2 * 128 * D;     // fp16 values
  static constexpr int KST = D == 64 ? 4 : (D == 128 ? 3 : 2);
  // Barriers of the copies of K: tile i's is number i % K_BARS. Where the slots take every other
  // tile each, a slot waits for the copies of its own tiles only, and copies land in any order, so
  // the tile before it on a barrier has to be one it has waited for: an even number of tiles before.
  // (With one barrier a stage at d = 128, tile 4's wait could pass on the phase before tile 1's.)
  static constexpr int K_BARS = D == 64 ? 4 : (D == 128 ? 6 : 2);
  static_assert(K_BARS % KST == 0 && K_BARS % 2 == 0, "a slot's waits would meet the other slot's copies");
  static constexpr int VST = D == 64 ? 3 : (D == 128 ? 2 : 1);
  static constexpr int SLOTS = KST + 2;  // tiles whose scales are kept: a tile's are read before the key ring comes round
  static constexpr int SST = D == 64 ? 4 : (D == 128 ? 2 : 1);  // staged value codes
  // tensor memory: per slot two 64-key buffers of S (the weights P take the first
  // 32 columns of the S they come from), then O
  __host__ __device__ static constexpr uint32_t s_col(int t, int buf) { return uint32_t(t) * 128u + uint32_t(buf) * 64u; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + uint32_t(t) * D; }
  static constexpr int SMEM = NT * Q_BYTES + KST * K_BYTES + VST * V_BYTES + SST * K_BYTES + 1024;
};

struct TileLaunch : Kv8Call {
  CUtensorMap tmK;         // the key codes: {d, page, pages * Hkv}
  float* part;             // [2 * CTAs][ROWS][d]
  float2* part_ml;         // [2 * CTAs][ROWS]
  int4* run;               // [CTAs][2]: where each CTA's run starts (b, h, block, tile); the block's holders
  uint32_t* status;
  uint64_t wait_limit_ns;
  uint32_t debug_skip;     // test hook, see fa_kernel_common.cuh
};

// How `total` tiles are dealt: runs of per + 1 tiles to the first `more` CTAs, of
// per tiles to the others.
struct Deal {
  long long per, more;
  int used;
  Deal() = default;
  // A block's start and end cost as much as four tiles: short blocks get a CTA each
  // (60 blocks of one tile, d = 128: 18 us instead of 26).
  __device__ __forceinline__ Deal(long long total, long long blocks, int ctas) {
    const long long most = max((total + kMinTiles - 1) / kMinTiles, min(total, blocks));
    used = most < ctas ? static_cast<int>(most) : ctas;
    per = used > 0 ? total / used : 0;
    more = total - per * used;
  }
  __device__ __forceinline__ long long first(int c) const {  // tile of CTA c's run
    return c >= used ? per * used + more : c * per + min(static_cast<long long>(c), more);
  }
  __device__ __forceinline__ int holder(long long x) const {
    const long long head = more * (per + 1);
    return static_cast<int>(x < head ? x / (per + 1) : more + (x - head) / per);
  }
};

template <int D>
struct TileShared {
  static constexpr int SLOTS = TileCfg<D>::SLOTS;
  uint64_t q_full[2], q_taken[2];
  uint64_t k_full[TileCfg<D>::K_BARS], k_empty[4], st_full[4], st_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2];  // [slot][buffer of S]
  uint64_t scale_full[SLOTS];
  uint64_t mma_drain[2];
  uint64_t join_ml[4], join_o[2][4];  // two halves of the keys: per warp pair
  float2 half_ml[2][TileCfg<D>::NT == 2 ? 128 : 1];
  float4 scale[SLOTS][4][2];  // of the 8 groups of 16 keys: c sk, log2 sv, 2^-kSumBias / sv, seen (1 or 0)
  int4 start;
  float qfac[TileCfg<D>::NT][128];
  Deal deal;
  int n_tiles;
  uint32_t tmem_base;
  int abort_flag;
};

// A place in a ring of N stages and the parity of its phase.
template <int N>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Row blocks of sequence b, and the key tiles that rows < `rows` of it see.
__device__ __forceinline__ int tiles_seen(int len, int count, int rows, int g, int causal) {
  const int last = (rows - 1) / g;  // position of the last row among the new tokens
  const int keys = causal ? min(len, max(0, len - count + last + 1)) : len;
  return (keys + 127) / 128;
}

// A row block, and the part of a run that lies in it.
template <int D>
struct Walk {
  static constexpr int ROWS = TileCfg<D>::ROWS;
  int b, h, blk, s;           // s: the first key tile of the run in this block
  int len, count, blocks;     // of sequence b
  int tiles;                  // key tiles of the block
  __device__ __forceinline__ void load(const TileLaunch& p) {
    const bool in = b < p.c.B;
    len = in ? seq_len(p.c, b) : 0;
    count = in ? seq_count(p.c, b, p.Nq) : 0;
    blocks = (count * p.g + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ int tiles_of(const TileLaunch& p, int block) const {
    return tiles_seen(len, count, min(count * p.g, (block + 1) * ROWS), p.g, p.causal);
  }
  __device__ __forceinline__ void settle(const TileLaunch& p) {  // after s moved on
    while (b < p.c.B && s >= tiles) {
      s -= tiles;
      if (++blk >= blocks) {
        blk = 0;
        if (blocks == 0 || ++h >= p.c.Hkv) {
          h = 0;
          ++b;
          load(p);
        }
      }
      tiles = blk < blocks ? tiles_of(p, blk) : 0;
    }
  }
  __device__ __forceinline__ void begin(const TileLaunch& p, const int4& at) {
    b = at.x, h = at.y, blk = at.z, s = at.w;
    load(p);
    tiles = blk < blocks ? tiles_of(p, blk) : 0;
  }
  // Key tiles (relative to s) that tile t of the block sees within n tiles of the run: the last one's index.
  __device__ __forceinline__ int last_tile(const TileLaunch& p, int t, int n) const {
    const int r0 = blk * ROWS + t * 128, live = min(count * p.g - r0, 128);
    if (live <= 0) return -1;
    return min(tiles_seen(len, count, r0 + live, p.g, p.causal), s + n) - 1 - s;
  }
};

// Row `row` of the group of K/V head w.h: position and place in [B][Hq][Nq], for
// rows a fixed step apart.
struct RowPlace {
  int qi, hg, g, dq, dr, Nq;
  size_t head;
  template <class W>
  __device__ __forceinline__ RowPlace(const TileLaunch& p, const W& w, int row, int step) {
    g = p.g;
    qi = row / g;
    hg = row - qi * g;
    dq = step / g;
    dr = step - dq * g;
    Nq = p.Nq;
    head = static_cast<size_t>(w.b) * p.Hq + w.h * g;
  }
  __device__ __forceinline__ void next() {
    qi += dq;
    hg += dr;
    if (hg >= g) {
      hg -= g;
      ++qi;
    }
  }
  __device__ __forceinline__ size_t index() const { return (head + hg) * Nq + qi; }
};

// Key tiles of all blocks of sequence b for one K/V head; *blocks: how many blocks.
template <int D>
__device__ __forceinline__ long long sequence_tiles(const TileLaunch& p, int b, int* blocks) {
  constexpr int ROWS = TileCfg<D>::ROWS;
  Walk<D> w;
  w.b = b;
  w.load(p);
  *blocks = w.len > 0 ? w.blocks : 0;
  if (!p.causal) return static_cast<long long>(w.blocks) * ((w.len + 127) / 128);
  // a block sees the keys up to its last row's position, which moves by ROWS / g a block
  const int step = ROWS / p.g, part = ROWS - step * p.g;
  long long n = 0;
  int pos = (ROWS - 1) / p.g, rest = ROWS - 1 - pos * p.g;
  for (int blk = 0; blk < w.blocks; ++blk) {
    n += (min(w.len, max(0, w.len - w.count + min(pos, w.count - 1) + 1)) + 127) / 128;
    pos += step;
    rest += part;
    if (rest >= p.g) {
      rest -= p.g;
      ++pos;
    }
  }
  return n;
}

// All lanes of one warp: the block (and tile of it) that tile x of the list is;
// first: sequence_tiles of sequence `lane` (0 behind the last).
template <int D>
__device__ int4 tile_search(const TileLaunch& p, long long first, long long x) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0;; b0 += 32) {
    int unused;
    const long long one = b0 == 0 ? first : b0 + lane < p.c.B ? sequence_tiles<D>(p, b0 + lane, &unused) : 0;
    long long incl = one * p.c.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > x);
    if (!past) {
      x -= __shfl_sync(0xffffffffu, incl, 31);
      continue;
    }
    const int l = __ffs(past) - 1;
    const long long per_head = __shfl_sync(0xffffffffu, one, l);
    long long rem = x - (__shfl_sync(0xffffffffu, incl, l) - per_head * p.c.Hkv);
    Walk<D> w;
    w.b = b0 + l;
    w.load(p);
    const int h = static_cast<int>(rem / per_head);
    rem -= h * per_head;
    for (int k0 = 0;; k0 += 32) {  // the block within the head
      const int own = k0 + lane < w.blocks ? w.tiles_of(p, k0 + lane) : 0;
      int in = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, in > rem);
      if (hit) {
        const int k = __ffs(hit) - 1;
        return make_int4(w.b, h, k0 + k, static_cast<int>(rem) - __shfl_sync(0xffffffffu, in - own, k));
      }
      rem -= __shfl_sync(0xffffffffu, in, 31);
    }
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, fp32 sums; the operands lie AOFF
// and BOFF bytes behind their descriptors. (The sums are formed here: as values
// of their own the compiler keeps every product's descriptor in registers over
// the whole loop, and the issuing thread, which has few, reloads them one by one.)
template <int AOFF, int BOFF, bool ACC>
__device__ __forceinline__ void umma_ss_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                           uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "add.u32 x, %1, %6;\n\tadd.u32 y, %3, %7;\n\t"
      "mov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(AOFF >> 4), "n"(BOFF >> 4), "n"(ACC ? 1 : 0)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], fp16 operands, fp32 sums; offsets likewise.
template <int ACOL, int BOFF>
__device__ __forceinline__ void umma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
      "add.u32 x, %1, %6;\n\tadd.u32 y, %2, %7;\n\t"
      "mov.b64 b, {y, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "n"(ACOL), "n"(BOFF >> 4)
      : "memory");
}

// Instruction descriptors (fields as in make_idesc_bf16_f32): e4m3 x e4m3 and
// fp16 x fp16, whose format fields are both 0.
__host__ __device__ constexpr uint32_t make_idesc_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | ((static_cast<uint32_t>(N) >> 3) << 17) |
         ((static_cast<uint32_t>(M) >> 4) << 24);
}

// Descriptor of a K-major tile with rows of 64 bytes, 64-byte swizzle (8-row atoms of 512 bytes).
__device__ __forceinline__ uint64_t make_smem_desc_sw64(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= 1ull << 16;
  d |= static_cast<uint64_t>(512 >> 4) << 32;
  d |= 1ull << 46;
  d |= 4ull << 61;
  return d;
}

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}
// The four warps of softmax warpgroup t; they all come, also after a timeout.
__device__ __forceinline__ void warpgroup_sync(int t) { named_barrier_sync(1 + t, 128); }
// One arrival for a warp's lanes: 32 of them on one barrier are 32 passes of
// the shared-memory pipe, which the tensor core's operands need.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------------------
// Pages, scales and loads (one warp)
// ---------------------------------------------------------------------------
template <int D>
__device__ void load_role(const TileLaunch& p, TileShared<D>& sh, uint8_t* sK, uint8_t* sStage) {
  using C = TileCfg<D>;
  const int lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  constexpr int ROW_BYTES = D < 128 ? D : 128;  // a key's codes in one column chunk of the operand tile
  const int page = 1 << p.c.page_log2, pages = 128 >> p.c.page_log2;
  const int n = sh.n_tiles;
  // Lane 8 j + g looks up 16-key group g of tile 4 k + j, one batch of 4 tiles ahead.
  Walk<D> cur;
  cur.begin(p, sh.start);
  cur.s += lane >> 3;
  cur.settle(p);
  int next_id = -1;  // sequence and head
  ScaleRun scales;
  auto look_up = [&]() -> int {  // page * Hkv + head; -1: a bad page, -2: behind the sequence
    int slot = -2;
    if (cur.b < p.c.B) {
      next_id = cur.b * p.c.Hkv + cur.h;
      const int key = cur.s * 128 + (lane & 7) * 16;
      if (key < cur.len) {
        const int pid = __ldg(p.c.table + static_cast<size_t>(cur.b) * p.c.max_pages + (key >> p.c.page_log2));
        slot = pid < 0 || pid >= p.c.num_pages ? -1 : pid * p.c.Hkv + cur.h;
      }
      cur.s += 4;
      cur.settle(p);
    }
    return slot;
  };
  int next = look_up(), now = -2;
  float4 entry = make_float4(0.f, 0.f, 0.f, 0.f);
  float sk = 0.f, sv = 0.f;
  int now_id = -1;
  bool ok = true;
  int k_issued = 0, st_issued = 0;
  for (int i = 0; i < n; ++i) {
    const int j0 = (i & 3) * 8;
    if (j0 == 0) {
      now = next;
      now_id = next_id;
      if (now >= 0) sk = __ldg(p.c.scale[0] + now), sv = __ldg(p.c.scale[1] + now);
      next = look_up();
    }
    const int ks = i % C::KST;
    uint64_t* k_full = &sh.k_full[i % C::K_BARS];
    if (i >= C::KST) ok = warp_wait(&sh.k_empty[ks], ((i / C::KST) - 1) & 1, &sh.abort_flag, lim);
    if (!ok) break;
    // lane p < pages: page p of the tile
    const int slot = __shfl_sync(0xffffffffu, now, j0 + (lane * page / 16 & 7));
    const bool live = lane < pages && slot >= 0;
    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * page * D;
    uint8_t* kd = sK + ks * C::K_BYTES;
    const bool skip = debug_skip_here(p.debug_skip, WHERE_KV8_LOAD, i == 0);  // test hook
    // S of a bad page's keys has to be a number
    for (unsigned bad = __ballot_sync(0xffffffffu, lane < pages && slot == -1); bad; bad &= bad - 1) {
      const int first = (__ffs(bad) - 1) * page * ROW_BYTES;
      for (int c = 0; c < D / ROW_BYTES; ++c)
        for (int u = lane * 16; u < page * ROW_BYTES; u += 512)
          st_shared_v4(smem_u32(kd) + c * (128 * 128) + first + u, 0, 0, 0, 0);
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0 && !skip) mbar_arrive_expect_tx(k_full, bytes);
    __syncwarp();
    if (live && !skip) {
#pragma unroll
      for (int c = 0; c < D / ROW_BYTES; ++c)
        tma_load_3d(kd + c * (128 * 128) + lane * page * ROW_BYTES, &p.tmK, k_full, c * 128, 0, slot);
    }
    ++k_issued;
    if (j0 == 0) {  // the scales, while K is on its way
      entry = make_float4(0.f, 0.f, 0.f, 0.f);
      scales.take(now >= 0, sv, now_id, &entry.y, &entry.z);
      if (now >= 0) {
        entry.x = sk * p.scale_log2;
        entry.w = 1.f;
      } else if (now == -1) {
        entry.y = -INFINITY;  // its keys are not seen
        record_bad_index(p.status, WHERE_FWD_KV8);
      }
    }
    const int slot8 = i % C::SLOTS;
    if (lane >= j0 && lane < j0 + 8) {
      float* to = reinterpret_cast<float*>(sh.scale[slot8]) + lane - j0;
      to[0] = entry.x, to[8] = entry.y, to[16] = entry.z, to[24] = entry.w;
      mbar_arrive(&sh.scale_full[slot8]);
    }
    const int ss = i % C::SST;
    if (i >= C::SST) ok = warp_wait(&sh.st_empty[ss], ((i / C::SST) - 1) & 1, &sh.abort_flag, lim);
    if (!ok) break;
    if (lane == 0) mbar_arrive_expect_tx(&sh.st_full[ss], bytes);
    __syncwarp();
    if (live)
      bulk_load(sStage + ss * C::K_BYTES + lane * page * D, p.c.code[1] + (static_cast<size_t>(slot) << p.c.page_log2) * D,
                page * D, &sh.st_full[ss]);
    ++st_issued;
  }
  if (!ok && lane == 0) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_LOAD);
  __syncwarp();
  // the copies already issued land before the CTA can exit
  if (lane == 0) {
    const int first = debug_skip_here(p.debug_skip, WHERE_KV8_LOAD, true) ? 1 : 0;
    for (int i = max(first, k_issued - C::KST); i < k_issued; ++i) drain_wait(&sh.k_full[i % C::K_BARS], (i / C::K_BARS) & 1, lim);
    for (int i = max(0, st_issued - C::SST); i < st_issued; ++i)
      drain_wait(&sh.st_full[i % C::SST], (i / C::SST) & 1, lim);
  }
}

// ---------------------------------------------------------------------------
// Value codes -> fp16 operand tiles (one warpgroup)
// ---------------------------------------------------------------------------
template <int D>
__device__ void convert_role(const TileLaunch& p, TileShared<D>& sh, uint8_t* sStage, uint8_t* sV) {
  using C = TileCfg<D>;
  constexpr int UNITS = D / 8;                     // 8 codes (16 bytes of fp16) each
  constexpr int PASSES = 128 * UNITS / kConvThreads;
  constexpr int PASS_ROWS = kConvThreads / UNITS;
  const int tid = threadIdx.x & 127;
  const int unit = tid % UNITS, row0 = tid / UNITS;
  const uint64_t lim = p.wait_limit_ns;
  const int n = sh.n_tiles;
  Walk<D> w;
  w.begin(p, sh.start);
  bool ok = true;
  for (int i = 0; i < n && ok; ++i) {
    if (i > 0) {
      ++w.s;
      w.settle(p);
    }
    const int ss = i % C::SST, vs = i % C::VST, sl = i % C::SLOTS;
    ok = warp_wait(&sh.scale_full[sl], (i / C::SLOTS) & 1, &sh.abort_flag, lim) &&
         warp_wait(&sh.st_full[ss], (i / C::SST) & 1, &sh.abort_flag, lim) &&
         (i < C::VST || warp_wait(&sh.v_empty[vs], ((i / C::VST) - 1) & 1, &sh.abort_flag, lim));
    if (!ok) break;
    // Keys behind the sequence and on bad pages: 0 (what lies there may be NaN codes, and 0 * NaN is not 0).
    const int rows = w.len - w.s * 128;
    const float4 sa = sh.scale[sl][3][0], sb = sh.scale[sl][3][1];
    const uint32_t seen = (sa.x != 0.f) | (sa.y != 0.f) << 1 | (sa.z != 0.f) << 2 | (sa.w != 0.f) << 3 |
                          (sb.x != 0.f) << 4 | (sb.y != 0.f) << 5 | (sb.z != 0.f) << 6 | (sb.w != 0.f) << 7;
    const uint8_t* src = sStage + ss * C::K_BYTES + row0 * D + unit * 8;
    const uint32_t dst = smem_u32(sV + vs * C::V_BYTES) + (unit / 8) * (128 * 128);
    // rows row0 + q PASS_ROWS; the swizzle repeats every 8 rows
    constexpr int PERIOD = PASS_ROWS < 8 ? 8 / PASS_ROWS : 1;
    uint32_t at[PERIOD];
#pragma unroll
    for (int q = 0; q < PERIOD; ++q) at[q] = dst + sw128_offset(row0 + q * PASS_ROWS, unit & 7);
    auto convert = [&](int q, uint2 v) {
      st_shared_v4(at[q % PERIOD] + (q / PERIOD) * (PERIOD * PASS_ROWS * 128), e4m3x2_to_f16x2(v.x & 0xffffu),
                   e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y & 0xffffu), e4m3x2_to_f16x2(v.y >> 16));
    };
    if (rows >= 128 && seen == 0xffu) {
#pragma unroll 4  // 2 and 16: the same time; more code than the loop needs slows the softmax's fetching
      for (int q = 0; q < PASSES; ++q) convert(q, *reinterpret_cast<const uint2*>(src + q * PASS_ROWS * D));
    } else {
#pragma unroll 2
      for (int q = 0; q < PASSES; ++q) {
        const int row = row0 + q * PASS_ROWS;
        uint2 v = *reinterpret_cast<const uint2*>(src + q * PASS_ROWS * D);
        if (row >= rows || !(seen >> (row >> 4) & 1)) v = make_uint2(0, 0);
        convert(q, v);
      }
    }
    warp_arrive(&sh.st_empty[ss]);
    fence_proxy_async_smem();
    warp_arrive(&sh.v_full[vs]);
  }
  if (!ok) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_CONVERT);
}

// ---------------------------------------------------------------------------
// MMA issuer (one thread per slot)
// ---------------------------------------------------------------------------
// S of one tile: step QS multiplies 32 columns of a piece (the first D / 32
// steps: qh). A row of Q holds 128 bytes per chunk of 128 rows: both pieces
// (d = 64), or 128 columns of one; a row of K its 64, or 128 columns.
template <int D, int... QS>
__device__ __forceinline__ void issue_s_steps(std::integer_sequence<int, QS...>, uint32_t d, uint32_t q_lo, uint32_t q_hi,
                                              uint32_t k_lo, uint32_t k_hi, uint32_t idesc) {
  (umma_ss_f8<(QS >> 2) * (128 * 128) + (QS & 3) * 32,
              (QS % (D / 32) >> 2) * (128 * 128) + (QS % (D / 32) & 3) * 32, (QS > 0)>(d, q_lo, q_hi, k_lo, k_hi, idesc),
   ...);
}
// O += P V over 64 keys, 16 a step.
template <int... KS>
__device__ __forceinline__ void issue_pv_steps(std::integer_sequence<int, KS...>, uint32_t d, uint32_t p_tmem,
                                               uint32_t v_lo, uint32_t v_hi, uint32_t idesc, uint32_t accumulate) {
  (umma_ts_f16<KS * 8, KS * 2048>(d, p_tmem, v_lo, v_hi, idesc, KS > 0 ? 1u : accumulate), ...);
}

// Slot t takes its key tiles in half steps of 64 keys, f = 0, 1, ... of a part of
// the run; step f's S and P lie in buffer f % 2. S(f + 1) is there before the
// softmax of step f ends, so a slot's chain is its softmax alone: PV(f) and, into
// the buffer that it has read, S(f + 2) run beside the softmax of f + 1.
template <int D, bool HALVES>
__device__ void mma_role(const TileLaunch& p, TileShared<D>& sh, uint8_t* sQ, uint8_t* sK, uint8_t* sV, uint32_t tmem, int t) {
  using C = TileCfg<D>;
  constexpr uint32_t kIdescS = make_idesc_f32(128, 64, false);
  constexpr uint32_t kIdescPV = make_idesc_f32(128, D, true);
  const uint64_t q_desc = make_smem_desc_sw128(smem_u32(sQ + t * C::Q_BYTES), 16, 1024);
  const uint64_t k_desc = D == 64 ? make_smem_desc_sw64(smem_u32(sK)) : make_smem_desc_sw128(smem_u32(sK), 16, 1024);
  const uint64_t v_desc = make_smem_desc_sw128(smem_u32(sV), 128 * 128, 1024);
  const uint64_t lim = p.wait_limit_ns;
  const uint32_t q_lo = static_cast<uint32_t>(q_desc), q_hi = static_cast<uint32_t>(q_desc >> 32);
  const uint32_t k_hi = static_cast<uint32_t>(k_desc >> 32), v_hi = static_cast<uint32_t>(v_desc >> 32);
  constexpr uint32_t kKeyHalf = (64 * (D < 128 ? D : 128)) >> 4, kValueHalf = (64 * 128) >> 4;  // of a column chunk
  Ring<C::KST> k;       // the stages of the tiles whose S and PV come next
  Ring<C::K_BARS> kb;   // the barrier of k's copy
  Ring<C::VST> v;
  uint32_t par = 0;     // parity of the buffers' use by PV, which S is one or none ahead of
  bool used = false;    // the buffers have been used
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &sh.abort_flag, lim); };
  auto skip_k = [&]() {
    const bool ok = HALVES || wait(&sh.k_full[kb.stage], kb.phase);
    if (!HALVES && ok) mbar_arrive(&sh.k_empty[k.stage]);
    k.next();
    kb.next();
    return ok;
  };
  auto skip_v = [&]() {
    if (HALVES) return v.next(), true;
    const bool ok = wait(&sh.v_full[v.stage], v.phase);
    if (ok) mbar_arrive(&sh.v_empty[v.stage]);
    v.next();
    return ok;
  };
  auto issue_s = [&](int b, bool read, uint32_t parity) -> bool {
    if (b == 0 && !wait(&sh.k_full[kb.stage], kb.phase)) return false;
    if (read && !wait(&sh.pv_done[t][b], parity)) return false;  // the P that was there
    tc_fence_after_sync();
    issue_s_steps<D>(std::make_integer_sequence<int, 2 * (D / 32)>{}, tmem + C::s_col(t, b), q_lo, q_hi,
                     static_cast<uint32_t>(k_desc) + k.stage * (C::K_BYTES >> 4) + b * kKeyHalf, k_hi, kIdescS);
    umma_commit(&sh.s_full[t][b]);
    if (b == 1) {
      umma_commit(&sh.k_empty[k.stage]);
      k.next();
      kb.next();
    }
    return true;
  };
  auto issue_pv = [&](int b, bool first) -> bool {
    if (b == 0 && !wait(&sh.v_full[v.stage], v.phase)) return false;
    if (!wait(&sh.p_full[t][b], par)) return false;
    tc_fence_after_sync();
    issue_pv_steps(std::make_integer_sequence<int, 4>{}, tmem + C::o_col(t), tmem + C::s_col(t, b),
                   static_cast<uint32_t>(v_desc) + v.stage * (C::V_BYTES >> 4) + b * kValueHalf, v_hi, kIdescPV, first ? 0u : 1u);
    umma_commit(&sh.pv_done[t][b]);
    if (b == 1) {
      umma_commit(&sh.v_empty[v.stage]);
      v.next();
    }
    return true;
  };
  Walk<D> w;
  w.begin(p, sh.start);
  int left = sh.n_tiles;
  bool ok = true;
  for (int seg = 0; ok && left > 0; ++seg) {
    const int n = min(left, w.tiles - w.s);
    const int turns = HALVES ? (n + 1 - t) / 2 : w.last_tile(p, t, n) + 1;
    ok = wait(&sh.q_full[t], seg & 1);
    if (ok) mbar_arrive(&sh.q_taken[t]);
    left -= n;
    w.s += n;
    w.settle(p);
    tc_fence_after_sync();
    if (HALVES && t == 1) skip_k(), skip_v();
    if (ok && turns > 0) {
      ok = issue_s(0, used, par ^ 1) && issue_s(1, used, par ^ 1);
      // PV(0) overwrites O: the part before has to have read it
      if (ok && seg > 0) ok = wait(&sh.o_free[t], (seg - 1) & 1);
    }
    for (int j = 0; ok && j < turns; ++j) {
      const bool more = j + 1 < turns;
      if (HALVES && more) skip_k();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        ok = ok && issue_pv(b, j == 0 && b == 0);
        if (more) ok = ok && issue_s(b, true, par);
      }
      if (HALVES && more) skip_v();
      par ^= 1;
    }
    used = used || turns > 0;
    // tiles that only the other slot's rows see; in halves: the other slot's last
    for (int j = turns; !HALVES && ok && j < n; ++j) ok = skip_k() && skip_v();
    if (HALVES && turns > 0 && (n - 1) % 2 != t) skip_k(), skip_v();
  }
  if (!ok) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_MMA);
  drain_mmas(&sh.mma_drain[t], lim);
}

// ---------------------------------------------------------------------------
// Q pieces, softmax, correction and epilogue (warpgroup t owns query tile t)
// ---------------------------------------------------------------------------
template <int D, bool HALVES>
__device__ void softmax_role(const TileLaunch& p, TileShared<D>& sh, uint8_t* sQ, uint32_t tmem, int t) {
  using C = TileCfg<D>;
  const int r = threadIdx.x & 127, lane = r & 31;
  const uint32_t lane_base = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
  const uint32_t tS = tmem + lane_base + C::s_col(t, 0);
  const uint32_t tO = tmem + lane_base + C::o_col(t);
  const uint32_t q_dst = smem_u32(sQ + t * C::Q_BYTES);
  const uint64_t lim = p.wait_limit_ns;
  constexpr int STEP = HALVES ? 2 : 1;
  Walk<D> w;
  w.begin(p, sh.start);
  int left = sh.n_tiles, i0 = 0, cnt = 0;
  // After a timed-out wait a warp stops working but keeps arriving, so barrier counts stay matched.
  bool alive = true;
  for (int seg = 0; left > 0; ++seg) {
    const int n = min(left, w.tiles - w.s);
    const int row0 = w.blk * C::ROWS + (HALVES ? 0 : t * 128);
    const int row = row0 + r;
    // the warpgroup's key tiles of this part of the run: j0, j0 + STEP, ... <= last
    const int j0 = HALVES ? t : 0;
    const int last = HALVES ? (t < n ? n - 1 : -1) : w.last_tile(p, t, n);
    const int turns = last < 0 ? 0 : (last - j0) / STEP + 1;
    const int qi = row / p.g;
    const bool live = qi < w.count;
    const size_t at = (static_cast<size_t>(w.b) * p.Hq + w.h * p.g + row % p.g) * p.Nq + qi;
    const int limit = p.causal ? min(w.len, w.len - w.count + qi + 1) : w.len;  // keys the row sees
    // The MMA thread has taken note of the segment before (else an idle slot's
    // warpgroup could run two arrivals ahead of its parity wait).
    if (alive && seg > 0) {
      alive = warp_wait(&sh.q_taken[t], (seg - 1) & 1, &sh.abort_flag, lim);
      if (!alive) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_SOFTMAX);
    }
    // rows are in order: a warp without a live one has nothing to weigh or store
    const int live_rows = min(128, w.count * p.g - row0);
    const bool warp_live = (r & ~31) < live_rows;
    if (seg > 0) warpgroup_sync(t);  // the Q tile has served every warp's epilogue
    if (alive && last >= 0) {
      // Rows as Q pieces, 8 columns a lane (whole lines a load); S of the segment
      // before is complete, so the tile is free. The warps take turns, whatever rows
      // are live; rows up to the last live warp's 32nd are 0.
      constexpr int LPR = D / 8, RPP = 32 / LPR;  // lanes a row, rows a pass
      constexpr int BATCH = 32 / RPP < 8 ? 32 / RPP : 8;  // a batch's loads are issued together
      const int col = lane % LPR, passes = (live_rows + 31) / 32 * (32 / RPP);
      // unit numbers along the row [qh | ql]; a lane has half a unit of each
      const int uh = col >> 1, ul = uh + D / 16;
      const uint32_t hi_at = q_dst + (uh >> 3) * (128 * 128) + (col & 1) * 8;
      const uint32_t lo_at = q_dst + (ul >> 3) * (128 * 128) + (col & 1) * 8;
      RowPlace at_q(p, w, row0 + (r >> 5) * RPP + lane / LPR, 4 * RPP);
#pragma unroll 1
      for (int q0 = r >> 5; q0 < passes; q0 += 4 * BATCH) {
        uint4 raw[BATCH];
        uint32_t amax[BATCH];  // bits of the row's largest |value|
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          raw[q] = make_uint4(0, 0, 0, 0);
          if (at_q.qi < w.count) raw[q] = __ldg(reinterpret_cast<const uint4*>(p.q + at_q.index() * D) + col);
          at_q.next();
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          const uint32_t w4[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
          amax[q] = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) amax[q] = max(amax[q], max(w4[k] & 0x7fffu, (w4[k] >> 16) & 0x7fffu));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
          for (int q = 0; q < BATCH; ++q) amax[q] = max(amax[q], __shfl_xor_sync(0xffffffffu, amax[q], o));
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          if (q0 + 4 * q >= passes) break;
          const int in_tile = (q0 + 4 * q) * RPP + lane / LPR;
          const uint32_t w4[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
          // exponent of the largest value; 2^-100 and below are left as they are
          const int x = min(max(static_cast<int>(amax[q] >> 7) - 127, -100), 127);
          const float mul = query_factor(amax[q], 7 - x);
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack_bf16x2(w4[k]);
            const __half2 v = __floats2half2_rn(f.x * mul, f.y * mul);
            const uint32_t h2 = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&v));
            const uint32_t back = e4m3x2_to_f16x2(h2);
            const __half2 rest = __hsub2(v, *reinterpret_cast<const __half2*>(&back));
            hi[k >> 1] |= h2 << (16 * (k & 1));
            lo[k >> 1] |= f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest)) << (16 * (k & 1));
          }
          st_shared_v2(hi_at + sw128_offset(in_tile, uh & 7), hi[0], hi[1]);
          st_shared_v2(lo_at + sw128_offset(in_tile, ul & 7), lo[0], lo[1]);
          if (col == 0) sh.qfac[t][in_tile] = exp2i(x - 7);
        }
      }
      fence_proxy_async_smem();
    }
    warp_arrive(&sh.q_full[t]);
    warpgroup_sync(t);
    const float qfac = sh.qfac[t][r];  // the row's power of two

    float m = -INFINITY, l = 0.f;  // reference - kShift, sum of P / sv
    for (int f = 0; f < 2 * turns; ++f) {  // 64 keys
      const int j = j0 + (f >> 1) * STEP, i = i0 + j, sl = i % C::SLOTS, buf = f & 1;
      if (buf == 0) alive = alive && warp_wait(&sh.scale_full[sl], (i / C::SLOTS) & 1, &sh.abort_flag, lim);
      alive = alive && warp_wait(&sh.s_full[t][buf], (cnt + (f >> 1)) & 1, &sh.abort_flag, lim);
      if (!alive) {
        record_timeout(p.status, &sh.abort_flag, WHERE_KV8_SOFTMAX);
        break;
      }
      tc_fence_after_sync();
      if (!warp_live) {  // nobody reads what its rows of P give
        warp_arrive(&sh.p_full[t][buf]);
        continue;
      }
      const uint32_t tSb = tS + buf * 64;
      uint32_t xa[32], xb[32];
      tmem_ld32(tSb, xa);
      tmem_ld32(tSb + 32, xb);
      tmem_ld_wait();
      const int lim_col = limit - (w.s + j) * 128 - buf * 64;
      if (__any_sync(0xffffffffu, lim_col < 64)) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (k >= lim_col) xa[k] = __float_as_uint(-INFINITY);
          if (32 + k >= lim_col) xb[k] = __float_as_uint(-INFINITY);
        }
      }
      // 16-key groups: u = S fg + eg; a group's factor is positive, so its
      // largest u is that of its largest S.
      float mx = -INFINITY;
      float4 fg = sh.scale[sl][0][buf];
      const float4 eg = sh.scale[sl][1][buf];
      fg.x = fmaxf(qfac * fg.x, 1e-36f), fg.y = fmaxf(qfac * fg.y, 1e-36f);
      fg.z = fmaxf(qfac * fg.z, 1e-36f), fg.w = fmaxf(qfac * fg.w, 1e-36f);
      auto max_of = [&](const uint32_t (&x)[32], int h, float fac, float add) {
        auto f = [&](int k) { return __uint_as_float(x[16 * h + k]); };
        float ga = fmaxf(f(0), f(1)), gb = fmaxf(f(2), f(3));
#pragma unroll
        for (int k = 4; k < 16; k += 4) {
          ga = fmax3(ga, f(k), f(k + 1));
          gb = fmax3(gb, f(k + 2), f(k + 3));
        }
        mx = fmaxf(mx, fmaf(fmaxf(ga, gb), fac, add));
      };
      max_of(xa, 0, fg.x, eg.x);
      max_of(xa, 1, fg.y, eg.y);
      max_of(xb, 0, fg.z, eg.z);
      max_of(xb, 1, fg.w, eg.w);
      const bool move = __any_sync(0xffffffffu, mx > m + (kShift + kSlack));
      const float m_ref = move ? fmaxf(m, mx - kShift) : m;
      const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
      const float alpha = ex2_approx(m - m_use);  // 0 on the first step, 1 when the reference is kept
      if (move) l = scale_sum(l, m - m_use, alpha);
      // P (packed pairs) overwrites columns of S that have been read
      const float4 zg = sh.scale[sl][2][buf];
      uint32_t pk[16];
      auto weigh = [&](const uint32_t (&x)[32], int h, float a, float b, float z) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 u = ffma2_bcast(__uint_as_float(x[16 * h + 2 * k]), __uint_as_float(x[16 * h + 2 * k + 1]), a, b);
          const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
          sum = fadd2(sum, e);
          pk[8 * h + k] = pack_f16x2(e.x, e.y);
        }
        l = fmaf(sum.x + sum.y, z, l);
      };
      weigh(xa, 0, fg.x, eg.x - m_use, zg.x);
      weigh(xa, 1, fg.y, eg.y - m_use, zg.y);
      tmem_st16(tSb, pk);
      weigh(xb, 0, fg.z, eg.z - m_use, zg.z);
      weigh(xb, 1, fg.w, eg.w - m_use, zg.w);
      tmem_st16(tSb + 16, pk);
      if (f > 0 && move) {
        // O has to hold the step before
        alive = warp_wait(&sh.pv_done[t][buf ^ 1], (cnt + ((f - 1) >> 1)) & 1, &sh.abort_flag, lim);
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; alive && c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(tO + c, o);
        }
      }
      m = m_ref;
      tmem_st_wait();
      tc_fence_before_sync();
      warp_arrive(&sh.p_full[t][buf]);
    }

    const bool active = last >= 0;
    if (alive && active) {
      alive = warp_wait(&sh.pv_done[t][1], (cnt + turns - 1) & 1, &sh.abort_flag, lim);
      if (!alive) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_SOFTMAX);
    }
    tc_fence_after_sync();
    float own = 1.f;  // what this warpgroup's O is multiplied with
    // 4 KB per warp in each 16 KB of both Q tiles, whose last S is complete:
    // the warp's own rows of them
    const int quarter = r >> 5;
    const uint32_t area = smem_u32(sQ) + quarter * 4096;
    if constexpr (HALVES) {
      // The two halves of the keys: both warps of the same rows learn the other's
      // m and l; each leaves the other's half of its O's columns in the other's Q
      // tile and goes on with the sum of its own half.
      sh.half_ml[t][r] = make_float2(m, l);
      warp_arrive(&sh.join_ml[quarter]);
      alive = alive && warp_wait(&sh.join_ml[quarter], seg & 1, &sh.abort_flag, lim);
      if (alive && warp_live) {
        const float2 other = sh.half_ml[t ^ 1][r];
        const float both = fmaxf(m, other.x), ref = both == -INFINITY ? 0.f : both;
        own = ex2_approx(m - ref);
        l = add_sums(l, m - ref, own, other.y, other.x - ref, ex2_approx(other.x - ref));
        m = both;
#pragma unroll 1
        for (int c = (t ^ 1) * (D / 2); c < ((t ^ 1) + 1) * (D / 2); c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = active ? __float_as_uint(__uint_as_float(o[k]) * own) : 0u;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            st_shared_v4(area + c * 512 + sw128_offset(lane, u), o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
      warp_arrive(&sh.join_o[t][quarter]);
    }
    if (alive && warp_live) {
      const bool whole = n == w.tiles;
      const size_t slot = (static_cast<size_t>(blockIdx.x) * 2 + (seg > 0)) * C::ROWS + (HALVES ? 0 : t * 128) + r;
      // 32 columns of the warp's 32 rows at a time through its own 4 KB of the Q
      // tile: stores of 64 (bf16) or 128 bytes of a row, eight or four rows a pass.
      // Row i's pieces are XORed as in the tiles.
      const uint32_t stage = q_dst + quarter * 4096;
      const int sub = whole ? lane & 3 : lane & 7, r_in = whole ? lane >> 2 : lane >> 3, step = whole ? 8 : 4;
      uint8_t* to[8];  // where the lane stores
      RowPlace at_q(p, w, row - lane + r_in, step);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        to[q] = nullptr;
        if (q * step < 32 && at_q.qi < w.count)
          to[q] = (whole ? reinterpret_cast<uint8_t*>(p.o + at_q.index() * D)
                         : reinterpret_cast<uint8_t*>(p.part + (slot - lane + q * 4 + r_in) * D)) + sub * 16;
        at_q.next();
      }
      if constexpr (HALVES) alive = warp_wait(&sh.join_o[t ^ 1][quarter], seg & 1, &sh.abort_flag, lim);
      const RowEnd end(m, l);
#pragma unroll 1
      for (int c = HALVES ? t * (D / 2) : 0; alive && c < (HALVES ? (t + 1) * (D / 2) : D); c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_ld_wait();
        if constexpr (HALVES) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = ld_shared_v4(area + c * 512 + sw128_offset(lane, u));
            if (!active) o[4 * u] = o[4 * u + 1] = o[4 * u + 2] = o[4 * u + 3] = 0;
            o[4 * u] = __float_as_uint(fmaf(__uint_as_float(o[4 * u]), own, __uint_as_float(x.x)));
            o[4 * u + 1] = __float_as_uint(fmaf(__uint_as_float(o[4 * u + 1]), own, __uint_as_float(x.y)));
            o[4 * u + 2] = __float_as_uint(fmaf(__uint_as_float(o[4 * u + 2]), own, __uint_as_float(x.z)));
            o[4 * u + 3] = __float_as_uint(fmaf(__uint_as_float(o[4 * u + 3]), own, __uint_as_float(x.w)));
          }
        }
        __syncwarp();  // the columns before have left
        if (whole) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = pack_bf16x2(end(__uint_as_float(o[8 * u + 2 * k])), end(__uint_as_float(o[8 * u + 2 * k + 1])));
            st_shared_v4(stage + sw128_offset(lane, u), x[0], x[1], x[2], x[3]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            st_shared_v4(stage + sw128_offset(lane, u), o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q * step < 32) v[q] = ld_shared_v4(stage + sw128_offset(q * step + r_in, sub));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (!HALVES && !active) v[q] = make_uint4(0, 0, 0, 0);  // a part whose keys no row of the tile sees
          if (to[q]) *reinterpret_cast<uint4*>(to[q] + c * (whole ? 2 : 4)) = v[q];
        }
      }
      if (live && !(HALVES && t == 1)) {
        if (whole) p.lse[at] = end.lse; else p.part_ml[slot] = make_float2(m, l);
      }
    }
    if (HALVES && !alive) record_timeout(p.status, &sh.abort_flag, WHERE_KV8_SOFTMAX);
    tc_fence_before_sync();
    warp_arrive(&sh.o_free[t]);
    cnt += turns;
    i0 += n;
    left -= n;
    w.s += n;
    w.settle(p);
  }
}

// For the joining kernel: where the run starts, the CTAs that hold the block it
// starts in, and whether that is not the first block of the first of them.
template <int D>
__device__ void note_run(const TileLaunch& p, const TileShared<D>& sh) {
  const int c = blockIdx.x;
  const int4 at = sh.start;
  int4 held = make_int4(c, c, 0, 0);
  if (sh.n_tiles > 0 && at.w > 0) {
    Walk<D> w;
    w.begin(p, at);
    const Deal deal = sh.deal;
    const long long begin = deal.first(c) - at.w;  // of the block
    held.x = deal.holder(begin);
    held.y = deal.holder(begin + w.tiles - 1);
    held.z = begin > deal.first(held.x) ? 1 : 0;
    held.w = w.count;
  }
  p.run[2 * c] = at;
  p.run[2 * c + 1] = held;
}

template <int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 1) kv8_tile_kernel(const __grid_constant__ TileLaunch p) {
  using C = TileCfg<D>;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ TileShared<D> sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::NT * C::Q_BYTES;
  uint8_t* sV = sK + C::KST * C::K_BYTES;
  uint8_t* sStage = sV + C::VST * C::V_BYTES;
  const int warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.q_full[t], 4);
      mbar_init(&sh.q_taken[t], 1);
      for (int b = 0; b < 2; ++b) {
        const bool first = t == 0 && b == 0;
        mbar_init(&sh.s_full[t][b], 1 + (first ? debug_extra(p.debug_skip, WHERE_KV8_MMA) : 0u));
        mbar_init(&sh.p_full[t][b], 4 + (first ? debug_extra(p.debug_skip, WHERE_KV8_SOFTMAX) : 0u));
        mbar_init(&sh.pv_done[t][b], 1);
      }
      mbar_init(&sh.o_free[t], 4);
    }
    for (int i = 0; i < C::K_BARS; ++i) mbar_init(&sh.k_full[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.k_empty[i], HALVES ? 1 : C::NT);
      mbar_init(&sh.st_full[i], 1);
      mbar_init(&sh.st_empty[i], kConvThreads / 32);
      mbar_init(&sh.v_full[i], kConvThreads / 32 + (i == 0 ? debug_extra(p.debug_skip, WHERE_KV8_CONVERT) : 0u));
      mbar_init(&sh.v_empty[i], HALVES ? 1 : C::NT);
    }
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&sh.scale_full[i], 8);
    mbar_init(&sh.mma_drain[0], 1);
    mbar_init(&sh.mma_drain[1], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.join_ml[i], 2);
      mbar_init(&sh.join_o[0][i], 1);
      mbar_init(&sh.join_o[1][i], 1);
    }
    sh.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp) {  // the CTA's run
    if (lane_id() == 0) tma_prefetch_desc(&p.tmK);
    const int lane = threadIdx.x & 31;
    int n = 0;
    const long long first = lane < p.c.B ? sequence_tiles<D>(p, lane, &n) : 0;
    long long total = first, blocks = n;
    for (int b = lane + 32; b < p.c.B; b += 32) {
      total += sequence_tiles<D>(p, b, &n);
      blocks += n;
    }
    const Deal deal(warp_sum(total) * p.c.Hkv, warp_sum(blocks) * p.c.Hkv, gridDim.x);
    const long long x0 = deal.first(blockIdx.x), x1 = deal.first(blockIdx.x + 1);
    int4 at = make_int4(p.c.B, 0, 0, 0);
    if (x1 > x0) at = tile_search<D>(p, first, x0);
    if (lane == 0) {
      sh.start = at;
      sh.n_tiles = static_cast<int>(x1 - x0);
      sh.deal = deal;
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  if (warp < 8) {
    if (warp < 4 * C::NT) softmax_role<D, HALVES>(p, sh, sQ, tmem, warp >> 2);
  } else if (warp < 12) {
    convert_role<D>(p, sh, sStage, sV);
  } else if (warp == kLoadWarp) {
    load_role<D>(p, sh, sK, sStage);
  } else if (lane_id() == 0 && warp < kMmaWarp + C::NT) {
    if (warp == kMmaWarp) note_run<D>(p, sh);  // Q takes longer to come
    mma_role<D, HALVES>(p, sh, sQ, sK, sV, tmem, warp - kMmaWarp);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Rows that the main kernel does not write, so that this runs beside it: rows
// without a key in row blocks without one (all of a sequence without tokens, the first ones
// where queries stand before the sequence), and with `fill` those past a
// sequence's count and all of one whose length or count is out of range. A warp a
// row, the warps of the first blocks (as many as there are sequences, or those of
// blockIdx.x = 0) shared out over the sequences.
template <int D>
__device__ __forceinline__ void write_other_rows(const TileLaunch& p) {
  using C = TileCfg<D>;
  const int lane = threadIdx.x & 31;
  const int per_x = gridDim.y * 8, nx = min(static_cast<int>(gridDim.x), (p.c.B - 1) / per_x + 1);
  const int warps = nx * per_x, share = max(1, warps / p.c.B);
  auto write = [&](size_t at, float lse) {
    if (lane < D / 8) reinterpret_cast<uint4*>(p.o + at * D)[lane] = make_uint4(0, 0, 0, 0);
    if (lane == 0) p.lse[at] = lse;
  };
  for (int k = blockIdx.x * per_x + blockIdx.y * 8 + (threadIdx.x >> 5); k / share < p.c.B; k += warps) {
    const int b = k / share, part = k - b * share;
    const int len = seq_len(p.c, b), count = seq_count(p.c, b, p.Nq);
    const bool bad = len != __ldg(p.c.lens + b) || (p.c.counts && count != __ldg(p.c.counts + b));
    if (bad && part == 0 && lane == 0) record_bad_index(p.status, WHERE_FWD_KV8);
    const size_t head0 = static_cast<size_t>(b) * p.Hq;
    const int past = !p.fill ? 0 : bad ? p.Nq : p.Nq - count;  // rows a head
    for (long long x = part; x < static_cast<long long>(past) * p.Hq; x += share) {
      const long long h = x / past;
      write((head0 + h) * p.Nq + (p.Nq - past) + (x - h * past), 0.f);
    }
    if (bad || (len > 0 && !(p.causal && count > len))) continue;
    const int rows = count * p.g;
    for (int blk = 0; blk * C::ROWS < rows; ++blk) {
      const int end = min(rows, (blk + 1) * C::ROWS);
      if (tiles_seen(len, count, end, p.g, p.causal) > 0) break;
      for (int x = part; x < (end - blk * C::ROWS) * p.c.Hkv; x += share) {
        const int row = blk * C::ROWS + x / p.c.Hkv, h = x % p.c.Hkv;
        write((head0 + h * p.g + row % p.g) * p.Nq + row / p.g, -INFINITY);
      }
    }
  }
}

// Joins the row blocks that CTAs shared. blockIdx.x = c > 0: the block that the
// runs of CTAs c - 1 and c meet in, if c - 1 is the first that holds a part
// of it; blockIdx.y: 8 of its rows.
template <int D>
__global__ void __launch_bounds__(256) kv8_tile_combine_kernel(const __grid_constant__ TileLaunch p) {
  using C = TileCfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (a grid has thousands of blocks: the others compute nothing here)
  if (blockIdx.x * gridDim.y * 8 < static_cast<unsigned>(p.c.B)) write_other_rows<D>(p);
  griddep_wait();
  if (blockIdx.x == 0) return;
  const int c = blockIdx.x;
  const int4 at = p.run[2 * c], held = p.run[2 * c + 1];
  const int c0 = held.x, c1 = held.y, count = held.w;
  if (c0 != c - 1) return;  // nothing is shared at this boundary, or another one's blocks join it
  // A warp joins a row, four parts on their way at a time.
  constexpr int PER = D / 32;
  const int rb = blockIdx.y * 8 + warp, row = at.z * C::ROWS + rb, qi = row / p.g;
  if (qi >= count) return;
  float m = -INFINITY, l = 0.f, a[PER];
  float low = INFINITY;  // smallest reference of a part that saw keys
#pragma unroll
  for (int k = 0; k < PER; ++k) a[k] = 0.f;
  for (int u0 = c0; u0 <= c1; u0 += 4) {
    float2 ml[4], x[4][PER / 2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int u = min(u0 + e, c1);
      const size_t slot = (static_cast<size_t>(u) * 2 + (u == c0 ? held.z : 0)) * C::ROWS + rb;
      ml[e] = p.part_ml[slot];
#pragma unroll
      for (int k = 0; k < PER / 2; ++k) x[e][k] = *reinterpret_cast<const float2*>(p.part + slot * D + lane * PER + 2 * k);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (u0 + e > c1) break;
      const float to = fmaxf(m, ml[e].x), ref = to == -INFINITY ? 0.f : to;
      const float wa = ex2_approx(m - ref), wx = ex2_approx(ml[e].x - ref);
      l = l * wa + ml[e].y * wx;
      low = fminf(low, ml[e].y > 0.f ? ml[e].x : INFINITY);
      m = to;
#pragma unroll
      for (int k = 0; k < PER; ++k) a[k] = a[k] * wa + (k & 1 ? x[e][k / 2].y : x[e][k / 2].x) * wx;
    }
  }
  if (m - low > 100.f) {  // a part's factor may have left fp32's range, its sum is added again
    l = 0.f;
#pragma unroll 1
    for (int u = c0; u <= c1; ++u) {
      const float2 ml = p.part_ml[(static_cast<size_t>(u) * 2 + (u == c0 ? held.z : 0)) * C::ROWS + rb];
      l += scale_sum(ml.y, ml.x - m, ex2_approx(ml.x - m));
    }
  }
  const RowEnd end(m, l);
  const size_t out = (static_cast<size_t>(at.x) * p.Hq + at.y * p.g + row % p.g) * p.Nq + qi;
#pragma unroll
  for (int k = 0; k < PER; k += 2)
    *reinterpret_cast<uint32_t*>(p.o + out * D + lane * PER + k) = pack_bf16x2(end(a[k]), end(a[k + 1]));
  if (lane == 0) p.lse[out] = end.lse;
}

template <int D>
size_t tile_part_bytes(size_t* ml_off, size_t* run_off) {
  const size_t rows = static_cast<size_t>(2) * kMaxSms * TileCfg<D>::ROWS;
  *ml_off = rows * D * sizeof(float);
  *run_off = *ml_off + rows * sizeof(float2);
  return *run_off + 2 * kMaxSms * sizeof(int4);
}

template <int D, bool HALVES>
cudaError_t launch_tiles(TileLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  using C = TileCfg<D>;
  auto kern = kv8_tile_kernel<D, HALVES>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kern, C::SMEM, dev.device, allowed);
  if (e != cudaSuccess) return e;
  const int grid = std::min(dev.num_sms, kMaxSms);
  kern<<<grid, kThreads, C::SMEM, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const long long rows = std::min<long long>(C::ROWS, static_cast<long long>(a.g) * a.Nq);  // of a block
  cfg.gridDim = dim3(grid, static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_tile_combine_kernel<D>, a);
}

}  // namespace

size_t kv8_tile_workspace(int d) {
  size_t ml, run;
  return d == 64 ? tile_part_bytes<64>(&ml, &run) : d == 128 ? tile_part_bytes<128>(&ml, &run) : tile_part_bytes<256>(&ml, &run);
}

fa_status_t launch_kv8_tiles(const Kv8Call& call, int d, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
  TileLaunch a{};
  static_cast<Kv8Call&>(a) = call;
  if (!make_cache_map(&a.tmK, call.c.code[0], d, 1 << call.c.page_log2,
                      static_cast<long long>(call.c.num_pages) * call.c.Hkv))
    return FA_ERR_CUDA;
  a.status = dev.status;
  a.wait_limit_ns = dev.wait_limit_ns;
  a.debug_skip = dev.debug_skip;
  size_t ml = 0, run = 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (d == 64) tile_part_bytes<64>(&ml, &run);
  if (d == 128) tile_part_bytes<128>(&ml, &run);
  if (d == 256) tile_part_bytes<256>(&ml, &run);
  a.part = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + ml);
  a.run = reinterpret_cast<int4*>(ws + run);
  // one tile of rows: both slots take it, with every other key tile each
  const bool halves = static_cast<long long>(call.g) * call.Nq <= 128;
  if (d == 64) return from_cuda(halves ? launch_tiles<64, true>(a, dev, stream) : launch_tiles<64, false>(a, dev, stream));
  if (d == 128) return from_cuda(halves ? launch_tiles<128, true>(a, dev, stream) : launch_tiles<128, false>(a, dev, stream));
  return from_cuda(launch_tiles<256, false>(a, dev, stream));
}

}  // namespace fa
