// MLA attention (MQA mode) over listed rows of the 8-bit latent cache, and over a tree of drafted
// tokens behind a cache (8-bit or bf16), for sm_100a.
//
// For one query t with heads h and attended rows S_t,
//   z[h,s] = tau * q[t,h,:] . row[s,:]        (d_latent + d_rope dims)
//   out[t,h,:] = sum_s softmax_s(z[h,.]) * row[s, :d_latent],   lse[t,h] = ln sum_s exp z[h,s]
// S_t is the query's list of cache positions; with a tree, query i of a sequence is node i of its
// drafted tokens, and S_t also holds the drafted rows on node i's path (itself, its parent, ...).
//
// Work split. A pair of CTAs (a 2-CTA cluster) takes one query over a range of its rows, with 2-SM
// tcgen05 MMAs issued by the even CTA: the fp32 output of 128 heads x 512 dims fills one SM's tensor
// memory, so each CTA holds 64 heads. Per 64-row block,
//  * logits: M = 128 heads (64 per CTA), N = 64 rows (CTA r supplies rows 32r ..), K = all dims;
//  * output: M = 128 heads, N = 256 dims per instruction (CTA r supplies dims 256i + 128r ..),
//    K = 64 rows, A = P from shared memory.
// When there are fewer queries than pairs, a query's rows are split into ranges whose normalised
// fp32 outputs and log-sum-exps are joined by cache_attn_join_kernel. (One CTA per 256 output dims,
// which needs no cluster but computes and expands everything for the logits twice, took 1.67 ms for
// 1024 queries of 2048 rows.)
//
// What bounds it: per 64-row block the two CTAs expand 32K codes, each of them twice (both operands hold a
// row's latent dims), and every stage of the chain rows -> logits -> softmax -> output hands over through
// shared memory. 1024 queries of 2048 rows, 128 heads, take 776 us (850 in a long row of calls, under the power
// cap): 753 TFLOP/s, 0.46 of what a bf16 matrix product reaches, at 64% of the issue slots and 35% of the tensor
// pipe's cycles. Of that, 126 us are the 14 items of a pair beside their blocks. Expanding once and copying the
// outputs' operand from the logits' with bulk copies within the pair took 0.95 to 1.30 ms: a logits stage then
// waits for its copy, and the copy for the outputs two blocks back.
//
// One CTA, 24 warps:
//  * control (1 warp): how far the range's list reaches, a node's path, and the item's q, ahead of the item.
//  * producers: 8 warps bring this CTA's 32 rows of each block, all dims (the logits' operand), 8 warps
//    all 64 rows' dims that it supplies to the output; each part has a 2-stage ring of
//    128-byte-swizzled bf16 tiles. 8-bit rows are loaded into registers one block ahead and expanded
//    to bf16 on the way to shared memory (exact: see qcache.cuh). Shared memory stays below 196 KB
//    on purpose: the L1 keeps 60 KB, which is what loads in flight land in. bf16 rows (drafted rows,
//    bf16 cache) are copied with cp.async. Rows that are not attended (padding, out of range, off
//    the path) are zero rows, so nothing they hold in memory reaches a product.
//  * MMA: one warp issues the logits, one the outputs (even CTA); in the odd CTA they, and one more, pass on
//    what its own warps have ready.
//  * softmax: 4 warps; lane L has rows 32 (L / 64) .. +31 of a block of head L % 64 of this CTA.
//    Online softmax in the log2 domain; the running max is raised, and the output rescaled, only when
//    it grows by more than kRescaleSlack.
// Statistics and outputs are fp32; P is rounded to bf16 for the tensor core. The output is
// normalised by the sum of the rounded weights (so they add up to one), lse takes the unrounded.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "qcache.cuh"
#include "sparse_mla.cuh"

namespace dsa {

constexpr int kMaxDraft = 256;           // nodes of a drafted tree
// How far (log2) the running max may lag behind a block's before it is raised and the outputs so far are rescaled: a
// weight is at most 2^kRescaleSlack, so that 2048 listed and 256 drafted rows of the cache's largest magnitude,
// 448 * 2^100, sum up to 2304 * 2^7 * 448 * 2^100 < 2^127, half of what fp32 holds.
constexpr float kRescaleSlack = 7.0f;
// The longest budget of a wait, a minute: every wait has an end, and 2 clocks per ns stay far within the 63 bits
// that the waits count in.
constexpr uint64_t kMaxCacheWaitNs = 60000000000ull;

struct CacheAttnCfg {
  static constexpr int BLK = 64;                         // rows per block
  static constexpr int L_ATOM = 32 * 128;                // logits part: 32 rows x 64 dims
  static constexpr int L_BYTES = 9 * L_ATOM;             // 32 rows x 576 dims
  static constexpr int O_ATOM = BLK * 128;               // output part: 64 rows x 64 dims
  static constexpr int O_BYTES = 4 * O_ATOM;             // 64 rows x 256 dims
  static constexpr int Q_TMEM_DIMS = 320;
  static constexpr int Q_ATOM = 64 * 128;                // 64 heads x 64 dims
  static constexpr int QS_ATOMS = (kDqk - Q_TMEM_DIMS) / 64;
  static constexpr int P_BYTES = 64 * 128;               // 64 heads x 64 rows bf16
  static constexpr int S_BUFS = 3;                       // TMEM logits buffers, 32 columns each
  static constexpr int SOFTMAX_WARPS = 4;
  static constexpr int PART_WARPS = 8;                   // producer warps per part
  static constexpr int PRODUCER_WARPS = 2 * PART_WARPS;
  static constexpr int S_WARP = SOFTMAX_WARPS + PRODUCER_WARPS;   // logits MMAs (and TMEM owner)
  static constexpr int O_WARP = S_WARP + 1;                       // output MMAs
  static constexpr int CTRL_WARP = S_WARP + 2;
  static constexpr int R_WARP = S_WARP + 3;                       // odd CTA: one of its three relays
  static constexpr int THREADS = (R_WARP + 1) * 32;
  // TMEM columns
  static constexpr uint32_t COL_O = 0, COL_S = 256, COL_Q = COL_S + 32 * S_BUFS, TMEM_COLS = 512;
  // shared memory
  static constexpr int OFF_L = 0;                        // 2 stages
  static constexpr int OFF_O = OFF_L + 2 * L_BYTES;      // 2 stages
  static constexpr int OFF_QS = OFF_O + 2 * O_BYTES;
  static constexpr int OFF_P = OFF_QS + QS_ATOMS * Q_ATOM;         // 2 buffers
  static constexpr int OFF_XCHG = OFF_P + 2 * P_BYTES;             // [2][128] tagged words
  static constexpr int OFF_INFO = OFF_XCHG + 2 * 128 * 8;
  static constexpr int INFO_WORDS = 4 + kMaxDraft / 32;  // list blocks, drafted blocks, first drafted block, -, path
  static constexpr int OFF_BAR = OFF_INFO + 2 * INFO_WORDS * 4;
  static constexpr int NUM_BARS = 32;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(OFF_O % 1024 == 0 && OFF_QS % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 8 == 0, "layout");
  static_assert(COL_Q + Q_TMEM_DIMS / 2 <= TMEM_COLS, "TMEM");
  static_assert(SMEM_BYTES <= 195 * 1024, "leaves the L1 its 60 KB");
};

struct CacheAttnParams {
  uint64_t wait_budget_ns;
  const __nv_bfloat16* kv;       // bf16 cache [B, max_len, d_latent + d_rope]
  QCacheView cache;              // 8-bit cache
  const int32_t* idx;            // [T, topk], T = B * n_q
  const __nv_bfloat16* draft;    // [B, n_q, d_latent + d_rope]
  const int32_t* parents;        // [B, n_q]
  __nv_bfloat16* out;            // [T, n_heads, d_latent]
  float* lse;                    // [T, n_heads]
  float* part_out;               // [T, n_splits, n_heads, d_latent], when n_splits > 1
  float* part_lse;               // [T, n_splits, n_heads], log2 domain
  uint32_t* status;
  int32_t n_q, max_len, topk, n_heads, d_latent, d_rope;
  int32_t n_splits, split_blocks, n_items;
  float scale_log2;              // tau * log2(e), positive
};

// Arrives once on the barrier at this offset in both CTAs of the pair when every 2-SM MMA this thread
// has issued so far is done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// True in one lane of a converged warp (always the same one). The whole warp walks the MMA role's code
// and one lane, elected right at the instructions, issues them: the operands then stay in uniform
// registers, where the instructions want them. Issued from inside `if (lane == 0)` an MMA cost 90 to
// 250 clocks.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Loads that stay where they are written (volatile): the producers issue a block's loads one block
// before their use, and a load that the compiler may move is moved down to its use. Piece kPiece of
// the n that there are, kOff bytes on; zero where there are fewer.
template <int kPiece, int kOff>
__device__ __forceinline__ uint4 ld_ahead_v4(const void* src, int32_t n) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %5, %6;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4 + %7];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(src), "r"(n), "n"(kPiece), "n"(kOff));
  return v;
}
template <int kPiece, int kOff>
__device__ __forceinline__ float ld_ahead_f32(const float* src, int32_t n) {
  float v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.gt.s32 p, %2, %3;\n\tmov.b32 %0, 0f00000000;\n\t"
      "@p ld.global.nc.f32 %0, [%1 + %4];\n\t}"
      : "=&f"(v)
      : "l"(src), "r"(n), "n"(kPiece), "n"(kOff));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Bounded waits on the SM's own clock. (The wait of ptx.cuh takes its time from %globaltimer, whose
// first read, about a thousand clocks, every wait that is not over at once would pay.) Same contract:
// past the budget the error is recorded and the CTA's abort flag raised, and every later wait fails.
struct ClockWaiter {
  uint32_t* status;
  volatile int* abort;
  int64_t budget;            // clocks
  __device__ __forceinline__ bool aborted() const { return *abort != 0; }
  // One more unsuccessful try: false once the CTA has aborted or the budget is spent (looked at every 64th
  // time).
  __device__ __forceinline__ bool again(uint32_t& spins, int64_t& t0, uint32_t tag) const {
    if ((++spins & 63u) != 0) return true;
    if (*abort) return false;
    if (t0 == 0) {
      t0 = clock64();
      return true;
    }
    if (clock64() - t0 <= budget) return true;
    record_error(status, DSA_ERR_DEVICE_TIMEOUT, (4u << 16) | tag);
    *abort = 1;
    __threadfence_block();
    return false;
  }
  // kCluster: some of the barrier's arrivals come from the other CTA of the pair
  template <bool kCluster = false>
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t tag) const {
    uint32_t spins = 0;
    int64_t t0 = 0;
    while (!(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) {
      // a try may suspend the thread for longer than this kernel's waits: with a budget under 1 us (a test's
      // setting) the first unsuccessful one is the last
      if (budget < 2000) {
        spins = 63;
        t0 = 1;
      }
      if (!again(spins, t0, tag)) return false;
    }
    return true;
  }
  // The low half of the 64-bit shared word at `addr` once its high half is `number` (one aligned store
  // writes both, so the pair is seen whole).
  __device__ __forceinline__ bool wait_word(uint32_t addr, uint32_t number, uint32_t tag, uint32_t& value) const {
    uint32_t spins = 0;
    int64_t t0 = 0;
    while (true) {
      uint64_t w;
      asm volatile("ld.volatile.shared.u64 %0, [%1];" : "=l"(w) : "r"(addr) : "memory");
      value = static_cast<uint32_t>(w);
      if (static_cast<uint32_t>(w >> 32) == number) return true;
      if (!again(spins, t0, tag)) return false;
    }
  }
};

template <bool kQuant, bool kTree>
__global__ void __launch_bounds__(CacheAttnCfg::THREADS, 1) __cluster_dims__(2, 1, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap map_q, const CacheAttnParams p) {
  using C = CacheAttnCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int32_t* info_base = reinterpret_cast<volatile int32_t*>(smem + C::OFF_INFO);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto B = [&](uint32_t i) { return bar0 + 8u * i; };
  // in both CTAs
  auto info_full = [&](uint32_t i) { return B(0 + i); };     // control warp
  auto info_empty = [&](uint32_t i) { return B(2 + i); };    // everyone who reads info
  auto s_full = [&](uint32_t i) { return B(4 + i); };        // commit (3): logits of a block done, its part read
  auto o_done = [&](uint32_t j) { return B(7 + j); };        // commit (2): outputs of a block done, its part and P read
  const uint32_t o_full = B(9);                              // commit: the item's outputs are done
  const uint32_t q_empty = B(10);                            // commit: the item's logits are done
  const uint32_t q_tma = B(11);                              // this CTA's q has landed in shared memory
  auto p_local = [&](uint32_t j) { return B(12 + j); };      // odd CTA's softmax warps: P written
  auto l_local = [&](uint32_t s) { return B(28 + s); };      // odd CTA's producer warps: its logits part is in
  auto v_local = [&](uint32_t s) { return B(30 + s); };      // the same for its output part
  // in the even CTA, arrived on by both
  auto l_full = [&](uint32_t s) { return B(14 + s); };       // its producer warps, a relay: a logits part is in
  auto v_full = [&](uint32_t s) { return B(16 + s); };       // its producer warps, a relay: an output part is in
  const uint32_t q_full = B(18);                             // a relay: the odd CTA's q is in (TMEM and shared memory)
  auto p_full = [&](uint32_t j) { return B(19 + j); };       // its softmax warps, and the odd CTA's relay
  const uint32_t o_empty = B(21);                            // softmax warps: outputs read
  // in the even CTA only: a logits buffer is free, once the output warp has seen its block's P
  auto s_free = [&](uint32_t i) { return B(22 + i); };       // (3)
  // in both CTAs
  const uint32_t mma_done = B(25);                           // the MMA warps' last commits
  const uint32_t q_read = B(26);                             // producer warps: q is out of the logits ring, and in
  const uint32_t stored = B(27);                             // softmax warps: an item's outputs are out of the P buffers
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 8);   // blocks read by the softmax

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // a join behind this kernel waits for its end itself
  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(info_full(i), 1);
      // softmax and producer warps, and the MMA warps (odd CTA: the relays)
      mbar_init(info_empty(i), C::SOFTMAX_WARPS + C::PRODUCER_WARPS + (leader ? 2 : 3));
      mbar_init(o_done(i), 1);
      mbar_init(p_local(i), C::SOFTMAX_WARPS);
      mbar_init(l_full(i), C::PART_WARPS + 1);
      mbar_init(v_full(i), C::PART_WARPS + 1);
      mbar_init(l_local(i), C::PART_WARPS);
      mbar_init(v_local(i), C::PART_WARPS);
      mbar_init(p_full(i), C::SOFTMAX_WARPS + 1);
    }
    for (uint32_t i = 0; i < static_cast<uint32_t>(C::S_BUFS); ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 1);
    }
    mbar_init(o_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(q_tma, 1);
    mbar_init(q_full, 1);
    mbar_init(q_read, C::PRODUCER_WARPS);
    mbar_init(stored, C::SOFTMAX_WARPS);
    mbar_init(o_empty, 2 * C::SOFTMAX_WARPS);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    *progress = 0;
    fence_mbar_init();
    prefetch_tensormap(&map_q);
  }
  // exchange numbers start at 1
  for (uint32_t i = threadIdx.x; i < 256u; i += C::THREADS) reinterpret_cast<uint64_t*>(smem + C::OFF_XCHG)[i] = 0;
  if (warp == C::S_WARP) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();            // both CTAs' barriers and TMEM exist before any remote traffic
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const ClockWaiter wt{p.status, abort_flag, static_cast<int64_t>(p.wait_budget_ns) * 2};   // at most 2 clocks per ns
  const int32_t n_pairs = static_cast<int32_t>(nclusters_x());
  const int32_t pair = static_cast<int32_t>(cluster_id_x());
  const uint32_t lead_off = mapa(bar0, 0) - bar0;            // the even CTA's copy of a barrier
  // arrives on the even CTA's copy of a barrier: across the pair only from the odd CTA
  auto arrive_leader = [&](uint32_t bar) {
    if (leader) mbar_arrive(bar);
    else mbar_arrive_cluster(bar + lead_off);
  };
  // Every lane waits (each one's own acquire orders its accesses) and the warp goes on, or gives up, as one.
  auto warp_wait = [&](uint32_t bar, uint32_t parity, uint32_t tag) -> bool {
    return __all_sync(0xffffffffu, wt.wait(bar, parity, tag));
  };
  auto warp_wait_pair = [&](uint32_t bar, uint32_t parity, uint32_t tag) -> bool {
    return __all_sync(0xffffffffu, wt.template wait<true>(bar, parity, tag));
  };

  // the logits buffer of the next block, and the parity of that use
  auto advance = [](uint32_t& buf, uint32_t& par) {
    if (++buf == static_cast<uint32_t>(C::S_BUFS)) {
      buf = 0;
      par ^= 1u;
    }
  };

  // item -> (query, range of its rows)
  struct Item {
    int32_t qi, split;
    int32_t e0, e1;       // list entries of the range
    int32_t k0, k1;       // 64-row blocks of drafted rows of the range
  };
  auto item_of = [&](int32_t it) {
    Item m;
    m.split = it % p.n_splits;
    m.qi = it / p.n_splits;
    const int32_t list_blocks = (p.topk + C::BLK - 1) / C::BLK;
    const int32_t all_blocks = list_blocks + (kTree ? (p.n_q + C::BLK - 1) / C::BLK : 0);
    const int32_t b0 = m.split * p.split_blocks, b1 = min(b0 + p.split_blocks, all_blocks);
    m.e0 = min(b0, list_blocks) * C::BLK;
    m.e1 = min(min(b1, list_blocks) * C::BLK, p.topk);
    m.k0 = max(b0 - list_blocks, 0);
    m.k1 = max(b1 - list_blocks, 0);
    return m;
  };
  const int32_t d_qk = p.d_latent + p.d_rope;
  const int32_t k_steps = (d_qk + 15) / 16;
  uint32_t q_sent = 0;                                       // control warp: q copies, at its end

  if (warp >= static_cast<uint32_t>(C::SOFTMAX_WARPS) && warp < static_cast<uint32_t>(C::S_WARP)) {
    // ================================================================ producers
    const uint32_t pw = warp - C::SOFTMAX_WARPS;
    const bool logits_part = pw < static_cast<uint32_t>(C::PART_WARPS);
    const uint32_t gt = (pw % C::PART_WARPS) * 32u + lane;   // thread of the part, 0..255
    // Logits part: eight threads per row, thread c has the row's 16-dim pieces c, c + 8, ...: one per
    // scale group. Output part: four threads per row, thread c has piece c of each of the four atoms.
    // Eight threads in a row hold four pieces of one atom in two neighbouring rows, so that the eight
    // 16-byte chunks which they store at once fall into distinct bank groups of the swizzled tile.
    const uint32_t row = logits_part ? 4u * (gt >> 5) + 2u * (lane >> 4) + ((lane >> 2) & 1u) : gt >> 2;   // of the tile
    const uint32_t c = logits_part ? (lane & 3u) + 4u * ((lane >> 3) & 1u) : lane & 3u;
    const uint32_t row_at = (row >> 3) * 1024u + (row & 7u) * 128u;
    static_assert(2 * C::L_ATOM == C::O_ATOM, "one step from piece to piece");
    const uint32_t tile_at = row_at + (c >> 2) * C::L_ATOM;
    const uint32_t at0 = tile_at + (((2 * (c & 3u)) ^ (row & 7u)) << 4);
    const uint32_t at1 = tile_at + (((2 * (c & 3u) + 1) ^ (row & 7u)) << 4);
    const int32_t block_row = static_cast<int32_t>(row + (logits_part ? 32u * rank : 0u));   // row of the block
    // piece k of this thread: its first dim, and where it goes in the tile, from at0 and at1
    const int32_t dim0 = 16 * static_cast<int32_t>(c) + (logits_part ? 0 : 128 * static_cast<int32_t>(rank));
    const int32_t dim_step = logits_part ? 128 : 64;
    auto piece_dim = [&](int32_t k) -> int32_t { return dim0 + 256 * (k >> 1) + dim_step * (k & 1); };
    auto piece_at = [](int32_t k) -> uint32_t { return static_cast<uint32_t>(k) * C::O_ATOM; };
    uint32_t n_it = 0, n_busy = 0, nb = 0;                   // items, items with blocks, blocks so far
    uint32_t s_buf = 0, s_par = 0;                           // logits buffer of block nb - 2, and its use's parity
    for (int32_t it = pair; it < p.n_items; it += n_pairs, ++n_it) {
      const Item m = item_of(it);
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      volatile int32_t* info = info_base + slot * C::INFO_WORDS;
      const int64_t seq = m.qi / p.n_q;
      const int32_t* idx_row = p.idx + static_cast<size_t>(m.qi) * p.topk;
      // this thread's entry of list block b (read ahead of its use), and the row it stands for, or -1.
      // Entries from the extent of the range on are padding, so they need no extra check.
      auto entry = [&](int32_t b) -> int32_t {
        const int32_t j = m.e0 + b * C::BLK + block_row;
        return j < m.e1 ? __ldg(idx_row + j) : -1;
      };
      auto checked = [&](int32_t v) -> int32_t {
        if (v < p.max_len) return v;
        record_error(p.status, DSA_ERR_INDEX_RANGE, static_cast<uint32_t>(m.qi));
        return -1;
      };
      const int32_t v0 = entry(0), v1 = entry(1);
      if (!warp_wait(info_full(slot), sph, 2)) break;
      const int32_t n_list = info[0], n_tail = info[1], k0 = info[2];
      uint32_t path = 0;                                 // bit k: this thread's row of drafted block k0 + k is attended
      if constexpr (kTree) {
        for (int32_t k = 0; k < n_tail; ++k)
          path |= ((static_cast<uint32_t>(info[4 + 2 * (k0 + k) + (block_row >> 5)]) >> (block_row & 31)) & 1u) << k;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(info_empty(slot));
      if (n_list + n_tail == 0) continue;

      // ---- q: it lands in shared memory (see the control warp); its dims 0..319 go from the logits ring,
      // which is free then, into the TMEM lanes (both lane halves hold this CTA's 64 heads; every producer
      // warp a lane quarter and 80 dims). A load per lane straight from global memory touches a line each
      // and took 5K clocks.
      const uint32_t q_par = n_busy & 1u;
      ++n_busy;
      auto bring_q = [&]() -> bool {
        if (!warp_wait(q_tma, q_par, 4)) return false;
        tc_fence_after();
        constexpr uint32_t kChunks = C::Q_TMEM_DIMS / 8 / (C::PRODUCER_WARPS / 4);   // 10 of 16 bytes
        static_assert(kChunks == 10 && 5 * C::Q_ATOM <= 2 * C::L_BYTES, "column stores, staging");
        const uint32_t hl = (32u * (warp & 3u) + lane) & 63u;
        const uint32_t at = tmem + ((32u * (warp & 3u)) << 16) + C::COL_Q + 4 * kChunks * (pw >> 2);
#pragma unroll
        for (uint32_t v0 = 0; v0 < kChunks; v0 += 2) {
          uint32_t r[8];
#pragma unroll
          for (uint32_t v = 0; v < 2; ++v) {
            const uint32_t ch = kChunks * (pw >> 2) + v0 + v;
            // past the last atom that was loaded the ring holds whatever it held
            uint4 u = make_uint4(0, 0, 0, 0);
            if (static_cast<int32_t>(8 * ch) < d_qk)
              u = ld_shared_v4(sbase + C::OFF_L + (ch >> 3) * C::Q_ATOM + sw128_offset(hl, ch & 7u));
            r[4 * v + 0] = u.x;
            r[4 * v + 1] = u.y;
            r[4 * v + 2] = u.z;
            r[4 * v + 3] = u.w;
          }
          tmem_st8(at + 4 * v0, r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_read);
        __syncwarp();
        // the ring may be filled once every warp has read its part
        return !logits_part || warp_wait(q_read, q_par, 7);
      };
      // ---- the blocks
      // waits for the part's stage of block nb, and gives it
      auto acquire = [&](uint32_t& tile) -> bool {
        const uint32_t st = nb & 1u;
        if (logits_part) {                                 // last read by the logits of block nb - 2
          tile = sbase + C::OFF_L + st * C::L_BYTES;
          if (nb < 2) return true;
          const uint32_t bar = s_full(s_buf), par = s_par;
          advance(s_buf, s_par);
          return warp_wait(bar, par, 5);
        }
        tile = sbase + C::OFF_O + st * C::O_BYTES;
        return warp_wait(o_done(st), ((nb >> 1) & 1u) ^ 1u, 6);
      };
      auto announce = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
        const uint32_t st = nb & 1u;
        if (lane == 0) mbar_arrive(leader ? (logits_part ? l_full(st) : v_full(st)) : (logits_part ? l_local(st) : v_local(st)));
      };
      // one block of bf16 rows: row r of a table, zeros where r < 0
      auto copy_block = [&](const __nv_bfloat16* table, int32_t r) -> bool {
        const __nv_bfloat16* src = table + (r >= 0 ? static_cast<int64_t>(r) * d_qk : 0);
        uint32_t tile;
        if (!acquire(tile)) return false;
        const int32_t dims = logits_part ? d_qk : p.d_latent;
#pragma unroll
        for (int32_t k = 0; k < 5; ++k) {
          const int32_t d = piece_dim(k);
          if ((k == 4 && !logits_part) || d >= dims) break;
          const bool in0 = r >= 0, in1 = r >= 0 && d + 8 < d_qk;
          cp_async_16(tile + piece_at(k) + at0, src + (in0 ? d : 0), in0 ? 16u : 0u);
          cp_async_16(tile + piece_at(k) + at1, src + (in1 ? d + 8 : 0), in1 ? 16u : 0u);
        }
        cp_async_commit();
        cp_async_wait<0>();
        announce();
        return true;
      };
      bool ok = true;
      if constexpr (kQuant) {
        const int32_t groups = (p.d_latent + kScaleGroup - 1) / kScaleGroup;
        const uint8_t* codes = p.cache.codes + seq * p.max_len * static_cast<int64_t>(p.d_latent);
        const float* scales = p.cache.scales + seq * p.max_len * static_cast<int64_t>(groups);
        const __nv_bfloat16* rope = p.cache.rope + seq * p.max_len * static_cast<int64_t>(p.d_rope);
        // Pieces below d_latent are codes, from there RoPE dims. Those are at most 64, so that a thread
        // of the logits part has at most one such piece: piece rope_k, at RoPE dim rope_d.
        const int32_t rope_k = (p.d_latent / 16 - static_cast<int32_t>(c) + 7) / 8;
        const int32_t rope_d = piece_dim(rope_k) - p.d_latent;
        const bool has_rope = logits_part && rope_d < p.d_rope;
        int32_t n_codes = 0;                               // pieces of codes that this thread has
#pragma unroll
        for (int k = 0; k < 4; ++k) n_codes += piece_dim(k) < p.d_latent ? 1 : 0;
        const int32_t n_rope = has_rope ? (rope_d + 8 < p.d_rope ? 2 : 1) : 0;
        // Scales: the logits part's pieces are of one group each, the output part's pieces 2 i and 2 i + 1
        // of the same one.
        const int32_t n_odd = logits_part ? 4 : 0;
        const int32_t group0 = dim0 / kScaleGroup;
        uint4 raw[4], rp[2];
        float sc[4];
        auto load = [&](int32_t r) {
          const int32_t n = r >= 0 ? n_codes : 0, odd = min(n, n_odd), nr = r >= 0 ? n_rope : 0;
          const uint8_t* src = codes + static_cast<int64_t>(r) * p.d_latent + dim0;
          const uint8_t* src1 = src + dim_step;
          const float* s0 = scales + static_cast<int64_t>(r) * groups + group0;
          raw[0] = ld_ahead_v4<0, 0>(src, n);
          sc[0] = ld_ahead_f32<0, 0>(s0, n);
          raw[1] = ld_ahead_v4<1, 0>(src1, n);
          sc[1] = ld_ahead_f32<1, 4>(s0, odd);
          raw[2] = ld_ahead_v4<2, 256>(src, n);
          sc[2] = ld_ahead_f32<2, 8>(s0, n);
          raw[3] = ld_ahead_v4<3, 256>(src1, n);
          sc[3] = ld_ahead_f32<3, 12>(s0, odd);
          if (has_rope) {
            const __nv_bfloat16* rs = rope + static_cast<int64_t>(r) * p.d_rope + rope_d;
            rp[0] = ld_ahead_v4<0, 0>(rs, nr);
            rp[1] = ld_ahead_v4<1, 16>(rs, nr);
          }
        };
        load(checked(v0));
        int32_t v = v1;
        if (!bring_q()) break;
        for (int32_t b = 0; b < n_list; ++b) {
          // The next block's loads go out together after the announcement: a load among the uses of
          // this block's would share a scoreboard with loads still to be used, which then wait for
          // it, and the fence of the announcement waits for loads in flight.
          uint32_t tile;
          if (!acquire(tile)) { ok = false; break; }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= n_codes) break;
            uint4 lo, hi;
            expand16(raw[k], logits_part ? sc[k] : sc[k & 2], lo, hi);
            st_shared_v4(tile + piece_at(k) + at0, lo);
            st_shared_v4(tile + piece_at(k) + at1, hi);
          }
          if (has_rope) {
            st_shared_v4(tile + piece_at(rope_k) + at0, rp[0]);
            st_shared_v4(tile + piece_at(rope_k) + at1, rp[1]);
          }
          announce();
          ++nb;
          v = checked(v);
          if (b + 1 < n_list) load(v);
          v = entry(b + 2);
        }
      } else {
        const __nv_bfloat16* table = p.kv + seq * p.max_len * static_cast<int64_t>(d_qk);
        int32_t v = v0, next = v1;
        if (!bring_q()) break;
        for (int32_t b = 0; b < n_list && ok; ++b, ++nb) {
          ok = copy_block(table, checked(v));
          v = next;
          next = entry(b + 2);
        }
      }
      if constexpr (kTree) {
        const __nv_bfloat16* table = p.draft + seq * p.n_q * static_cast<int64_t>(d_qk);
        for (int32_t k = 0; k < n_tail && ok; ++k, ++nb)
          ok = copy_block(table, (path >> k) & 1u ? (k0 + k) * C::BLK + block_row : -1);
      }
      if (!ok) break;
    }
    cp_async_wait<0>();
  } else if (warp == static_cast<uint32_t>(C::CTRL_WARP)) {
    // ================================================================ control: an item's extent, path and q, ahead of it
    uint32_t n_it = 0, n_busy = 0, nb = 0;
    for (int32_t it = pair; it < p.n_items; it += n_pairs, ++n_it) {
      const Item m = item_of(it);
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      volatile int32_t* info = info_base + slot * C::INFO_WORDS;
      const int32_t node = m.qi % p.n_q;
      const int64_t seq = m.qi / p.n_q;
      const int32_t* idx_row = p.idx + static_cast<size_t>(m.qi) * p.topk;
      // ---- the extent of the list in this range (one past its last entry >= 0, found from the
      // end), and the node's path through the tree
      if (!warp_wait(info_empty(slot), sph ^ 1u, 1)) break;
      int32_t end = m.e0;
      for (int32_t hi = m.e1; hi > m.e0 && end == m.e0;) {
        const int32_t lo = max(m.e0, hi - 256);
        int32_t last = m.e0 - 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t j = lo + static_cast<int32_t>(lane) + 32 * i;
          if (j < hi && __ldg(idx_row + j) >= 0) last = j;
        }
        end = __reduce_max_sync(0xffffffffu, last) + 1;
        hi = lo;
      }
      int32_t n_list = (end - m.e0 + C::BLK - 1) / C::BLK, n_tail = 0;
      if constexpr (kTree) {
        const int32_t* par_row = p.parents + seq * p.n_q;
        int32_t par[kMaxDraft / 32];
#pragma unroll
        for (int w = 0; w < kMaxDraft / 32; ++w) {
          const int32_t j = 32 * w + static_cast<int32_t>(lane);
          par[w] = j < p.n_q ? __ldg(par_row + j) : -2;
        }
        uint32_t path = 0;                             // lane w: bits of nodes 32w .. 32w+31
        int32_t cur = node;
        bool present = true;
        while (true) {                                 // cur falls strictly: at most n_q steps
          int32_t v = par[0];
#pragma unroll
          for (int w = 1; w < kMaxDraft / 32; ++w)
            if ((cur >> 5) == w) v = par[w];
          v = __shfl_sync(0xffffffffu, v, cur & 31);
          if (static_cast<int32_t>(lane) == (cur >> 5)) path |= 1u << (cur & 31);
          if (v >= cur) {                              // not an earlier node
            if (lane == 0) record_error(p.status, DSA_ERR_INDEX_RANGE, static_cast<uint32_t>(m.qi));
            present = false;
          } else if (v < -1) {
            present = false;
          }
          if (!present || v < 0) break;
          cur = v;
        }
        n_tail = max(0, min(m.k1, node / C::BLK + 1) - m.k0);
        if (!present) n_list = n_tail = 0;             // an absent node, or one below an absent node
        if (lane < kMaxDraft / 32) info[4 + lane] = static_cast<int32_t>(path);
      }
      if (lane == 0) {
        info[0] = n_list;
        info[1] = n_tail;
        info[2] = m.k0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(info_full(slot));
      // ---- q, once the previous item's logits MMAs have read theirs: all dims by TMA, dims 320.. where they
      // stay, dims 0..319 into the logits ring. Past the query's last dim TMA fills zeros; rows past its
      // last head only reach unused lanes.
      if (n_list + n_tail == 0) continue;
      if (!warp_wait(q_empty, (n_busy & 1u) ^ 1u, 3)) break;
      ++n_busy;
      if (lane == 0) {
        const int32_t atoms = (d_qk + 63) / 64;
        fence_proxy_async_smem();                          // the ring's earlier stores before TMA's
        mbar_expect_tx(q_tma, static_cast<uint32_t>(atoms) * C::Q_ATOM);
        for (int32_t t = 0; t < atoms; ++t)
          tma_load_3d(sbase + (t < C::Q_TMEM_DIMS / 64 ? C::OFF_L + t * C::Q_ATOM
                                                       : C::OFF_QS + (t - C::Q_TMEM_DIMS / 64) * C::Q_ATOM),
                      &map_q, q_tma, 64 * t, m.qi * p.n_heads + 64 * static_cast<int32_t>(rank), 0);
      }
      __syncwarp();
      if constexpr (kQuant) {
        // ---- this CTA's rows into L2, kAhead blocks before the logits come to them (lane = row). Paced by the
        // softmax's count of blocks, which only grows: a barrier's parity would not do for a warp that
        // nothing keeps from falling behind.
        constexpr int32_t kAhead = 4;
        const int32_t groups = (p.d_latent + kScaleGroup - 1) / kScaleGroup;
        const uint32_t row0 = static_cast<uint32_t>(seq) * static_cast<uint32_t>(p.max_len);
        for (int32_t b = 2; b < n_list; ++b) {
          const int32_t j = m.e0 + b * C::BLK + static_cast<int32_t>(32u * rank + lane);
          const int32_t v = j < m.e1 ? __ldg(idx_row + j) : -1;
          uint32_t spins = 0;
          int64_t t0 = 0;
          bool ok = true;
          while (ok && static_cast<int32_t>(nb + b - kAhead - *progress) > 0) {
            __nanosleep(200);
            ok = wt.again(spins, t0, 8);
          }
          if (!__all_sync(0xffffffffu, ok)) break;
          if (v >= 0 && v < p.max_len) {
            const uint64_t r = row0 + static_cast<uint32_t>(v);
            const uint8_t* codes = p.cache.codes + r * static_cast<uint32_t>(p.d_latent);
            for (int32_t d = 0; d < p.d_latent; d += 128) prefetch_l2(codes + d);
            prefetch_l2(p.cache.scales + r * static_cast<uint32_t>(groups));
            if (p.d_rope > 0) prefetch_l2(p.cache.rope + r * static_cast<uint32_t>(p.d_rope));
          }
        }
        nb += static_cast<uint32_t>(n_list + n_tail);
      }
    }
    q_sent = n_busy;
  } else if (warp >= static_cast<uint32_t>(C::S_WARP)) {
    // ================================================================ MMA issuers (even CTA), relays (odd CTA)
    // One warp issues the logits MMAs, one the output MMAs, so that each one's waits (issue blocks
    // while the pipe is full) overlap the other's work. A commit tracks the MMAs of its own thread.
    constexpr uint32_t idesc_s = make_idesc(1, 1, 0, 0, 128, C::BLK);
    constexpr uint32_t idesc_o = make_idesc(1, 1, 0, 1, 128, 256);
    const bool logits = warp == static_cast<uint32_t>(C::S_WARP);
    const int32_t out_instr = p.d_latent > 256 ? 2 : 1;
    uint32_t n_it = 0, n_busy = 0, nb = 0;
    uint32_t buf = 0, buf_par = 0;                       // logits buffer, and the parity of its use
    bool ok = !leader || warp != static_cast<uint32_t>(C::R_WARP);      // which has nothing to do in the even CTA
    for (int32_t it = pair; it < p.n_items && ok; it += n_pairs, ++n_it) {
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      if (!warp_wait(info_full(slot), sph, 10)) break;
      const int32_t n_blocks = info_base[slot * C::INFO_WORDS] + info_base[slot * C::INFO_WORDS + 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(info_empty(slot));
      if (n_blocks == 0) continue;
      if (!leader) {
        // Relays, one each for P, the logits part and the output part (and q): the odd CTA's warps announce theirs
        // locally, and one cluster-scope arrive, which by cumulativity carries the observed stores, follows.
        // From a producer warp that arrive took 1.5K clocks of every block (a CTA-scope one 0.4K).
        const bool l_part = warp == static_cast<uint32_t>(C::O_WARP);
        const uint32_t from = logits ? p_local(0) : l_part ? l_local(0) : v_local(0);
        const uint32_t to = lead_off + (logits ? p_full(0) : l_part ? l_full(0) : v_full(0));
        if (l_part) {
          if (!warp_wait(q_read, n_busy & 1u, 18)) break;
          tc_fence_after();
          tc_fence_before();
          if (lane == 0) mbar_arrive_cluster(q_full + lead_off);
          __syncwarp();
        }
        for (int32_t b = 0; b < n_blocks; ++b, ++nb) {
          const uint32_t st = nb & 1u;
          if (!warp_wait(from + 8u * st, (nb >> 1) & 1u, 11)) { ok = false; break; }
          if (lane == 0) mbar_arrive_cluster(to + 8u * st);
          __syncwarp();
        }
      } else if (logits) {
        if (!warp_wait(q_read, n_busy & 1u, 19)) break;
        if (!warp_wait_pair(q_full, n_busy & 1u, 12)) break;
        for (int32_t b = 0; b < n_blocks; ++b, ++nb) {
          const uint32_t st = nb & 1u;
          if (!warp_wait_pair(l_full(st), (nb >> 1) & 1u, 13)) { ok = false; break; }
          if (!warp_wait(s_free(buf), buf_par ^ 1u, 14)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + C::COL_S + 32u * buf;
          const uint64_t tile = sw128_desc(sbase + C::OFF_L + st * C::L_BYTES, 1, 1024);
          const uint64_t qs = sw128_desc(sbase + C::OFF_QS, 1, 1024);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kDqk / 16; ++k) {
              if (k >= k_steps) break;
              const uint64_t bd = tile + static_cast<uint64_t>(((k >> 2) * C::L_ATOM + (k & 3) * 32) >> 4);
              constexpr int kT = C::Q_TMEM_DIMS / 16;
              if (k < kT) {
                mma2_ts(d, tmem + C::COL_Q + 8 * k, bd, idesc_s, k > 0 ? 1u : 0u);
              } else {
                mma2_ss(d, qs + static_cast<uint64_t>((((k - kT) >> 2) * C::Q_ATOM + ((k - kT) & 3) * 32) >> 4), bd,
                        idesc_s, 1u);
              }
            }
            commit_pair(s_full(buf));
          }
          __syncwarp();
          advance(buf, buf_par);
        }
        if (!ok) break;
        if (elect_one()) commit_pair(q_empty);
      } else {
        if (!warp_wait_pair(o_empty, (n_busy & 1u) ^ 1u, 15)) break;
        for (int32_t b = 0; b < n_blocks; ++b, ++nb) {
          const uint32_t st = nb & 1u;
          if (!warp_wait_pair(v_full(st), (nb >> 1) & 1u, 16)) { ok = false; break; }
          if (!warp_wait_pair(p_full(st), (nb >> 1) & 1u, 17)) { ok = false; break; }
          if (lane == 0) mbar_arrive(s_free(buf));       // the softmax is done with that logits buffer
          __syncwarp();
          advance(buf, buf_par);
          tc_fence_after();
          const uint64_t pd = sw128_desc(sbase + C::OFF_P + st * C::P_BYTES, 1, 1024);
          const uint64_t tile = sw128_desc(sbase + C::OFF_O + st * C::O_BYTES, C::O_ATOM, 1024);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i >= out_instr) break;
#pragma unroll
              for (int k = 0; k < C::BLK / 16; ++k)
                mma2_ss(tmem + C::COL_O + 128 * i, pd + static_cast<uint64_t>((32 * k) >> 4),
                        tile + static_cast<uint64_t>((2 * i * C::O_ATOM + 2048 * k) >> 4), idesc_o,
                        (b > 0 || k > 0) ? 1u : 0u);
            }
            commit_pair(o_done(st));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) commit_pair(o_full);
      }
      ++n_busy;
    }
    if (leader && warp != static_cast<uint32_t>(C::R_WARP) && elect_one()) {
      commit_pair(mma_done);
      attn_drain_wait(mma_done, 0, kDrainBudgetNs);
    }
  } else {
    // ================================================================ softmax (TMEM lane = thread)
    // Lane L: head 64 rank + L % 64; logits of block rows 32 (L / 64) ..; output dims 256 i + 128 (L / 64) ..
    // Warps w and w + 2 hold the halves of the same 32 heads' rows and exchange their maxima.
    const uint32_t L = threadIdx.x, part = L >> 6, hl = L & 63u;
    const int32_t head = static_cast<int32_t>(64u * rank + hl);
    const uint32_t lane_off = (warp * 32u) << 16;
    const float sc = p.scale_log2;
    uint32_t n_it = 0, n_busy = 0, nb = 0, nx = 0;
    uint32_t buf = 0, buf_par = 0;                       // logits buffer, and the parity of its use
    bool ok = true;
    // One float from the thread with the other half of the row. Each thread has two words and stores
    // (number, value) in one; a word is used again only after the partner has answered the next
    // exchange, so no unread value is overwritten.
    const uint32_t xchg = sbase + C::OFF_XCHG;
    auto swap_partner = [&](float mine) -> float {
      const uint32_t at = xchg + (nx & 1u) * (128u * 8u);
      ++nx;
      const uint64_t word = (static_cast<uint64_t>(nx) << 32) | __float_as_uint(mine);
      asm volatile("st.volatile.shared.u64 [%0], %1;" ::"r"(at + L * 8u), "l"(word) : "memory");
      uint32_t v = 0;
      const bool got = wt.wait_word(at + (L ^ 64u) * 8u, nx, 24, v);
      if (!__all_sync(0xffffffffu, got)) ok = false;
      return __uint_as_float(v);
    };
    for (int32_t it = pair; it < p.n_items && ok; it += n_pairs, ++n_it) {
      const Item m = item_of(it);
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      if (!warp_wait(info_full(slot), sph, 20)) break;
      volatile int32_t* info = info_base + slot * C::INFO_WORDS;
      const int32_t n_list = info[0], n_tail = info[1], k0 = info[2];
      uint32_t path[kTree ? kMaxDraft / 64 : 1];         // this half's words of the drafted blocks
      if constexpr (kTree) {
#pragma unroll
        for (int w = 0; w < kMaxDraft / 64; ++w) path[w] = static_cast<uint32_t>(info[4 + 2 * w + part]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(info_empty(slot));
      const int32_t n_blocks = n_list + n_tail;
      const size_t row = static_cast<size_t>(m.qi) * p.n_heads + head;                       // (query, head)
      const size_t prow = (static_cast<size_t>(m.qi) * p.n_splits + m.split) * p.n_heads + head;
      const bool writes = head < p.n_heads;
      if (n_blocks == 0) {
        if (writes) {
          if (p.n_splits == 1) {
            for (int32_t d = 128 * static_cast<int32_t>(part); d < p.d_latent; d += 256)
              for (int32_t u = d; u < min(d + 128, p.d_latent); u += 8)
                *reinterpret_cast<uint4*>(p.out + row * p.d_latent + u) = make_uint4(0, 0, 0, 0);
            if (part == 0) p.lse[row] = -INFINITY;
          } else if (part == 0) {
            p.part_lse[prow] = -INFINITY;
          }
        }
        continue;
      }
      // entry 32 part + lane of list block b, read one block ahead: a ballot gives the valid rows
      const int32_t* idx_row = p.idx + static_cast<size_t>(m.qi) * p.topk;
      auto entry = [&](int32_t b) -> int32_t {
        const int32_t j = m.e0 + b * C::BLK + static_cast<int32_t>(32u * part + lane);
        return j < m.e1 ? __ldg(idx_row + j) : -1;
      };
      int32_t v = entry(0);
      float m2 = -INFINITY, l_r = 0.f, l_f = 0.f;        // running max; sums of rounded and unrounded weights
      for (int32_t b = 0; b < n_blocks; ++b, ++nb) {
        const uint32_t st = nb & 1u;
        uint32_t vm = __ballot_sync(0xffffffffu, v >= 0 && v < p.max_len);
        if constexpr (kTree) {
          if (b >= n_list) {
            const int32_t k = k0 + b - n_list;
#pragma unroll
            for (int w = 0; w < kMaxDraft / 64; ++w)
              if (w == k) vm = path[w];
          }
        }
        v = entry(b + 1);
        if (!warp_wait(s_full(buf), buf_par, 21)) { ok = false; break; }
        tc_fence_after();
        uint32_t z[32];
        tmem_ld32(tmem + lane_off + C::COL_S + 32u * buf, z);
        tmem_wait_ld();
        tc_fence_before();
        advance(buf, buf_par);
        if (kQuant && threadIdx.x == 0) *progress = nb + 1;
        if (vm != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((vm >> j) & 1u)) z[j] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(z[j]));
        float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;     // sc > 0
        mb = fmaxf(mb, swap_partner(mb));
        if (!ok) break;
        const bool need = mb > m2 + kRescaleSlack;
        float alpha = 1.0f;
        if (need) {
          alpha = m2 == -INFINITY ? 0.0f : ex2_approx(m2 - mb);
          m2 = mb;
          l_r *= alpha;
          l_f *= alpha;
        }
        // while every row seen so far was masked m2 is -inf: subtract 0, so that P = 2^-inf = 0
        const float msub = m2 == -INFINITY ? 0.0f : m2;
        uint32_t pk[16];
        uint64_t sum_r = 0, sum_f = 0;                   // packed pairs of fp32
        const uint64_t sc2 = pack_f32x2(sc, sc), msub2 = pack_f32x2(-msub, -msub);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint64_t x = pack_f32x2(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1]));
          asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(sc2), "l"(msub2));
          float a0, a1;
          unpack_f32x2(x, a0, a1);
          a0 = ex2_approx(a0);
          a1 = ex2_approx(a1);
          const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);
          const float2 back = __bfloat1622float2(pr);
          asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum_r) : "l"(pack_f32x2(back.x, back.y)));
          asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum_f) : "l"(pack_f32x2(a0, a1)));
          pk[j] = *reinterpret_cast<const uint32_t*>(&pr);
        }
        float s0, s1;
        unpack_f32x2(sum_r, s0, s1);
        l_r += s0 + s1;
        unpack_f32x2(sum_f, s0, s1);
        l_f += s0 + s1;
        // ---- the P buffer is free once the outputs of block nb - 2 are done; a raised max waits for those
        // of block nb - 1, and rescales this lane's outputs
        if (b > 0 && __any_sync(0xffffffffu, need)) {
          if (!warp_wait(o_done(st ^ 1u), ((nb - 1) >> 1) & 1u, 22)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            uint32_t o[16];
            tmem_ld16(tmem + lane_off + C::COL_O + 16 * k, o);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
            tmem_st16(tmem + lane_off + C::COL_O + 16 * k, o);
          }
          tmem_wait_st();
          tc_fence_before();
        } else if (nb >= 2) {
          if (!warp_wait(o_done(st), ((nb >> 1) & 1u) ^ 1u, 23)) { ok = false; break; }
        }
        // the item before stored its outputs through the P buffers, each warp at its own pace
        if (b == 0 && n_busy > 0 && !warp_wait(stored, (n_busy - 1) & 1u, 26)) { ok = false; break; }
        // ---- P row hl, columns 32 part .. +31: four chunks of the 128-byte swizzled row
        const uint32_t prow_at = sbase + C::OFF_P + st * C::P_BYTES;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_shared_v4(prow_at + sw128_offset(hl, 4 * part + k), make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(leader ? p_full(st) : p_local(st));
      }
      if (!ok) break;
      // ---- normalise and store. A sum of zero (no row attended) gives zeros and -inf.
      l_r += swap_partner(l_r);
      l_f += swap_partner(l_f);
      if (!ok || !warp_wait(o_full, n_busy & 1u, 25)) break;
      ++n_busy;
      tc_fence_after();
      const float inv = l_r == 0.f ? 0.f : 1.0f / l_r;
      // 128 bytes of 32 heads (64 dims in bf16, 32 in fp32) at a time go through this warp's 4 KB of the P buffers
      // (free now: the outputs that read them are done), so that a store instruction writes whole 128-byte
      // pieces of rows; straight from the lanes, a row each, it took 10K clocks. The 16-byte chunks are
      // swizzled so that eight lanes at a time, writing or reading, fall into distinct bank groups.
      const uint32_t tile = sbase + C::OFF_P + warp * 4096u;
      const int32_t head0 = static_cast<int32_t>(64u * rank + (warp & 1u) * 32u);       // of lane 0
      const uint32_t ch = lane & 7u;
      // lane's row in, chunk `ch` of rows lane / 8, + 4, ... out
      auto turn = [&](const uint32_t (&w)[32]) {
        __syncwarp();                                    // the previous pass has been read
#pragma unroll
        for (int u = 0; u < 8; ++u)
          st_shared_v4(tile + lane * 128u + ((u ^ (lane & 7u)) << 4), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
        __syncwarp();
      };
      // rows 16 half + 4 i + lane / 8
      auto fetch4 = [&](int half, uint4 (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t r = 16u * half + 4u * i + (lane >> 3);
          x[i] = ld_shared_v4(tile + r * 128u + ((ch ^ (r & 7u)) << 4));
        }
      };
      // dims of column group k of `width` columns (2 instructions x 128 columns)
      auto dim_of = [&](int k, int width) {
        const int32_t col = k * width;
        return 256 * (col >> 7) + 128 * static_cast<int32_t>(part) + (col & 127);
      };
      const int32_t heads = p.n_heads - head0 - static_cast<int32_t>(lane >> 3);        // this lane's rows 4 i < heads are heads
      if (p.n_splits == 1) {
        __nv_bfloat16* base = p.out + (static_cast<size_t>(m.qi) * p.n_heads + head0 + (lane >> 3)) * p.d_latent + 8 * ch;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const int32_t dim = dim_of(k, 64);
          if (dim >= p.d_latent) break;                  // (rises with k)
          uint32_t w[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_off + C::COL_O + 64 * k + 32 * h, o);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const __nv_bfloat162 pr =
                  __floats2bfloat162_rn(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
              w[16 * h + u] = *reinterpret_cast<const uint32_t*>(&pr);
            }
          }
          turn(w);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint4 x[4];
            fetch4(half, x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * half + 4 * i < heads && dim + 8 * static_cast<int32_t>(ch) < p.d_latent)
                *reinterpret_cast<uint4*>(base + static_cast<size_t>(16 * half + 4 * i) * p.d_latent + dim) = x[i];
          }
        }
      } else {
        float* base = p.part_out + ((static_cast<size_t>(m.qi) * p.n_splits + m.split) * p.n_heads + head0 + (lane >> 3)) *
                                       p.d_latent + 4 * ch;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const int32_t dim = dim_of(k, 32);
          if (dim >= p.d_latent) break;
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + C::COL_O + 32 * k, o);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * inv);
          turn(o);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint4 x[4];
            fetch4(half, x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * half + 4 * i < heads && dim + 4 * static_cast<int32_t>(ch) < p.d_latent)
                *reinterpret_cast<uint4*>(base + static_cast<size_t>(16 * half + 4 * i) * p.d_latent + dim) = x[i];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(stored);
        arrive_leader(o_empty);
      }
      if (writes && part == 0) {
        const float l2 = l_f == 0.f ? -INFINITY : m2 + log2f(l_f);
        if (p.n_splits == 1) p.lse[row] = l2 * 0.69314718055994531f;
        else p.part_lse[prow] = l2;
      }
    }
  }
  // ---- teardown: every role reaches here (all waits are bounded)
  tc_fence_before();
  __syncthreads();
  // Without an abort the producers have seen the last q copy land. Whether there was one is known only now: they may
  // give up on that copy long after the control warp has sent it and left its loop. (1024 queries of 2048 rows take
  // 778 us this way, 810 with the control warp waiting for the copy at the end of its loop in any case.)
  if (warp == C::CTRL_WARP && lane == 0 && q_sent > 0 && wt.aborted())
    attn_drain_wait(q_tma, (q_sent - 1) & 1u, kDrainBudgetNs);
  __syncwarp();
  cluster_sync();            // no CTA leaves while its peer may still use its memory
  if (warp == C::S_WARP) {
    // The odd CTA has no MMAs of its own, but the even one's commits arrive on its barriers, and after an
    // abort nobody may have waited for them. By now the last ones have been issued and are over in the even CTA.
    if (!leader) attn_drain_wait(mma_done, 0, kDrainBudgetNs);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
  }
}

// Joins the ranges of a query: with l_s the log-sum-exp of range s (log2 domain) and o_s its
// normalised output, w_s = 2^(l_s - max l), out = sum w_s o_s / sum w_s, lse = max l + log2 sum w_s.
// One CTA per (query, head), four dims per thread; a range without a row (l_s = -inf) wrote no
// output, and what is read in its place is not used.
//
// This kernel starts while the ranges' kernel still writes what it reads. So its loads are plain ones, behind the
// wait: the read-only path (__ldg, or const pointers that nothing else may alias) is for data that does not change
// while a kernel runs, and the compiler may move such loads up past the wait. They are issued kJoinBatch ranges
// at a time, without a condition between them: one query of 2048 rows takes 18.1 us (18.9 with __ldg, 21.2 with plain
// loads each under its range's condition).
constexpr int kJoinThreads = 128;
constexpr int kJoinBatch = 8;
__global__ void __launch_bounds__(kJoinThreads) cache_attn_join_kernel(
    const float* part_out, const float* part_lse, __nv_bfloat16* out, float* lse, int32_t n_splits, int32_t n_heads,
    int32_t d_latent) {
  asm volatile("griddepcontrol.wait;" ::: "memory");    // the ranges' kernel is done and its stores are visible
  const int64_t row = blockIdx.x;                        // (query, head)
  const int64_t qi = row / n_heads, head = row - qi * n_heads;
  const float* lrow = part_lse + qi * n_splits * n_heads + head;
  const int32_t dim = 4 * static_cast<int32_t>(threadIdx.x);
  const float* orow = part_out + (qi * n_splits * n_heads + head) * d_latent + (dim < d_latent ? dim : 0);
  const int64_t step = static_cast<int64_t>(n_heads) * d_latent;
  float l[kJoinBatch];
  float4 o[kJoinBatch];
  auto fetch = [&](int32_t s0) {
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      const int32_t s = min(s0 + u, n_splits - 1);
      l[u] = lrow[static_cast<int64_t>(s) * n_heads];
      o[u] = *reinterpret_cast<const float4*>(orow + s * step);
    }
  };
  fetch(0);
  float mx = -INFINITY;
#pragma unroll 8
  for (int32_t s = 0; s < n_splits; ++s) mx = fmaxf(mx, lrow[static_cast<int64_t>(s) * n_heads]);
  const float msub = mx == -INFINITY ? 0.f : mx;
  float total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int32_t s0 = 0; s0 < n_splits; s0 += kJoinBatch) {
    if (s0 > 0) fetch(s0);
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u) {
      if (s0 + u >= n_splits || l[u] == -INFINITY) continue;
      const float w = exp2f(l[u] - msub);
      total += w;
      acc.x += w * o[u].x;
      acc.y += w * o[u].y;
      acc.z += w * o[u].z;
      acc.w += w * o[u].w;
    }
  }
  const float inv = total == 0.f ? 0.f : 1.0f / total;
  if (dim < d_latent) {
    __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(out + row * d_latent + dim) =
        make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
  if (threadIdx.x == 0) lse[row] = total == 0.f ? -INFINITY : (mx + log2f(total)) * 0.69314718055994531f;
}

}  // namespace dsa
