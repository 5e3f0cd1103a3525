// MLA attention (MQA mode) over listed rows of the 8-bit latent cache, and over a tree of drafted
// tokens behind a cache (8-bit or bf16), for sm_100a.
//
// For one query t with heads h and attended rows S_t,
//   z[h,s] = tau * q[t,h,:] . row[s,:]        (d_latent + d_rope dims)
//   out[t,h,:] = sum_s softmax_s(z[h,.]) * row[s, :d_latent],   lse[t,h] = ln sum_s exp z[h,s]
// S_t is the query's list of cache positions; with a tree, query i of a sequence is node i of its
// drafted tokens, and S_t also holds the drafted rows on node i's path (itself, its parent, ...).
//
// Work split. One CTA owns 128 heads x 256 output dims of one query over a range of its rows: the
// fp32 output (256 TMEM columns) leaves room for two 64-row logits buffers (128 columns) and 256
// dims of q (128 columns). The two halves of a query are independent CTAs that both compute the
// logits: no exchange and no cluster, every product a full-rate M = 128 one-SM tcgen05 MMA, at
// the price of reading the rows twice (from L2, half the bytes of a bf16 row each time).
// When there are fewer (query, half) pairs than SMs, a query's rows are also split into ranges
// whose normalised fp32 outputs and log-sum-exps are joined by cache_attn_join_kernel.
//
// One CTA, 13 warps:
//  * producers (8 warps): 64-row blocks into a 2-stage ring of 128-byte-swizzled bf16 tiles. 8-bit
//    rows are loaded into registers one block ahead, so the gather's latency overlaps the previous
//    block, and expanded to bf16 on the way to shared memory (exact: see qcache.cuh). bf16 rows
//    (drafted rows, bf16 cache) are copied with cp.async. Rows that are not attended (padding, out
//    of range, off the path) are zero rows, so nothing they hold in memory reaches a product.
//  * MMA (1 thread): logits of block b+1, then output of block b. Logits: M = 128 heads, N = 64
//    rows, A = q (dims 0..255 from TMEM, the rest from shared memory). Output: A = P from TMEM (it
//    overwrites the block's logits), B = the same tile's first dims, N = 256.
//  * softmax (4 warps, one thread per head): online softmax in the log2 domain. The running max is
//    raised, and the output rescaled, only when it grows by more than kLazyRescale.
// Statistics and outputs are fp32; P is rounded to bf16 for the tensor core. The output is
// normalised by the sum of the rounded weights (so they add up to one), lse takes the unrounded.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "qcache.cuh"
#include "ptx.cuh"
#include "sparse_mla.cuh"

namespace dsa {

constexpr int kMaxDraft = 256;           // nodes of a drafted tree

struct CacheAttnCfg {
  static constexpr int BLK = 64;                         // rows per block
  static constexpr int STAGES = 2;
  static constexpr int ATOM = BLK * 128;                 // 64 rows x 64 dims
  static constexpr int STAGE_BYTES = 9 * ATOM;           // 64 rows x 576 dims
  static constexpr int Q_TMEM_DIMS = 256;
  static constexpr int Q_ATOM = kHeads * 128;            // 128 heads x 64 dims
  static constexpr int QS_ATOMS = (kDqk - Q_TMEM_DIMS) / 64;
  static constexpr int SOFTMAX_WARPS = 4;
  static constexpr int PRODUCER_WARPS = 8;
  static constexpr int ROWS = BLK / PRODUCER_WARPS;      // rows of a block per producer warp
  static constexpr int MMA_WARP = SOFTMAX_WARPS + PRODUCER_WARPS;
  static constexpr int THREADS = (MMA_WARP + 1) * 32;
  static constexpr int OUT_DIMS = 256;                   // output dims per CTA
  // TMEM columns
  static constexpr uint32_t COL_O = 0, COL_S = 256, COL_Q = COL_S + 2 * BLK, TMEM_COLS = 512;
  // shared memory
  static constexpr int OFF_STAGE = 0;
  static constexpr int OFF_QS = OFF_STAGE + STAGES * STAGE_BYTES;
  static constexpr int OFF_INFO = OFF_QS + QS_ATOMS * Q_ATOM;
  static constexpr int INFO_WORDS = 4 + kMaxDraft / 32;  // list blocks, list end, tail blocks, first tail block, path
  static constexpr int OFF_BAR = OFF_INFO + 2 * INFO_WORDS * 4;
  static constexpr int NUM_BARS = 17;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(STAGE_BYTES % 1024 == 0 && OFF_QS % 1024 == 0 && OFF_BAR % 8 == 0, "layout");
  static_assert(COL_Q + Q_TMEM_DIMS / 2 <= TMEM_COLS, "TMEM");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct CacheAttnParams {
  const __nv_bfloat16* q;        // [T, n_heads, d_latent + d_rope], T = B * n_q
  const __nv_bfloat16* kv;       // bf16 cache [B, max_len, d_latent + d_rope]
  QCacheView cache;              // 8-bit cache
  const int32_t* idx;            // [T, topk]
  const __nv_bfloat16* draft;    // [B, n_q, d_latent + d_rope]
  const int32_t* parents;        // [B, n_q]
  __nv_bfloat16* out;            // [T, n_heads, d_latent]
  float* lse;                    // [T, n_heads]
  float* part_out;               // [T, n_splits, n_heads, d_latent], when n_splits > 1
  float* part_lse;               // [T, n_splits, n_heads], log2 domain
  uint32_t* status;
  int32_t n_q, max_len, topk, n_heads, d_latent, d_rope;
  int32_t n_halves, n_splits, split_blocks, n_items;
  float scale_log2;              // tau * log2(e), positive
  uint64_t wait_budget_ns;
};

// D[tmem] (+)= A[smem] * B[smem]^T, bf16 -> f32, one SM.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <bool kQuant, bool kTree>
__global__ void __launch_bounds__(CacheAttnCfg::THREADS, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap map_q, const CacheAttnParams p) {
  using C = CacheAttnCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int32_t* info_base = reinterpret_cast<volatile int32_t*>(smem + C::OFF_INFO);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto B = [&](uint32_t i) { return bar0 + 8u * i; };
  auto full = [&](uint32_t s) { return B(0 + s); };          // producer warps: a block's tile is in shared memory
  auto empty = [&](uint32_t s) { return B(2 + s); };         // commit: the block's output MMAs are done
  auto s_full = [&](uint32_t s) { return B(4 + s); };        // commit: logits ready
  auto p_full = [&](uint32_t s) { return B(6 + s); };        // softmax warps: P written
  auto info_full = [&](uint32_t i) { return B(8 + i); };     // first producer warp
  auto info_empty = [&](uint32_t i) { return B(10 + i); };   // everyone who reads info
  const uint32_t q_full = B(12);                             // producer warps + TMA
  const uint32_t q_empty = B(13);                            // commit: the item's logits MMAs are done
  const uint32_t o_full = B(14);                             // commit: the item's output MMAs are done
  const uint32_t o_empty = B(15);                            // softmax warps: output read
  const uint32_t mma_done = B(16);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const uint32_t warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(full(s), C::PRODUCER_WARPS);
      mbar_init(empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), C::SOFTMAX_WARPS);
      mbar_init(info_full(s), 1);
      mbar_init(info_empty(s), C::SOFTMAX_WARPS + (C::PRODUCER_WARPS - 1) + 1);
    }
    mbar_init(q_full, C::PRODUCER_WARPS + 1);
    mbar_init(q_empty, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, C::SOFTMAX_WARPS);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Waiter wt{p.status, abort_flag, p.wait_budget_ns, 4u};
  auto warp_wait = [&](uint32_t bar, uint32_t parity, uint32_t tag) -> bool {
    uint32_t got = 1;
    if (lane == 0) got = wt.wait(bar, parity, tag) ? 1u : 0u;
    return __shfl_sync(0xffffffffu, got, 0) != 0;
  };

  // item -> (query, range of its rows, half of the output dims); the halves of a query are
  // neighbours, so that the rows one reads are in L2 for the other
  struct Item {
    int32_t qi, split, half;
    int32_t e0, e1;       // list entries of the range
    int32_t k0, k1;       // 64-row blocks of drafted rows of the range
  };
  auto item_of = [&](int32_t it) {
    Item m;
    m.half = it % p.n_halves;
    const int32_t rest = it / p.n_halves;
    m.split = rest % p.n_splits;
    m.qi = rest / p.n_splits;
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

  if (warp >= static_cast<uint32_t>(C::SOFTMAX_WARPS) && warp < static_cast<uint32_t>(C::MMA_WARP)) {
    // ================================================================ producers
    const uint32_t pw = warp - C::SOFTMAX_WARPS;        // rows ROWS*pw .. of every block
    uint32_t n_it = 0, n_q_loads = 0, nb = 0;           // items, items with blocks, blocks so far
    bool tma_pending = false;
    for (int32_t it = blockIdx.x; it < p.n_items; it += gridDim.x, ++n_it) {
      const Item m = item_of(it);
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      volatile int32_t* info = info_base + slot * C::INFO_WORDS;
      const int32_t node = m.qi % p.n_q;
      const int64_t seq = m.qi / p.n_q;
      const int32_t* idx_row = p.idx + static_cast<size_t>(m.qi) * p.topk;
      if (pw == 0) {
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
          info[1] = end;
          info[2] = n_tail;
          info[3] = m.k0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(info_full(slot));
      } else {
        if (!warp_wait(info_full(slot), sph, 2)) break;
      }
      const int32_t n_list = info[0], end = info[1], n_tail = info[2], k0 = info[3];
      uint64_t path = 0;                                 // this warp's rows of a drafted block, by block
      if constexpr (kTree) {
        // byte k of `path`: rows ROWS*pw .. +7 of drafted block k0 + k (at most 4 blocks)
        for (int32_t k = 0; k < n_tail; ++k) {
          const uint32_t w = static_cast<uint32_t>(info[4 + 2 * (k0 + k) + (pw >> 2)]);
          path |= static_cast<uint64_t>((w >> (8 * (pw & 3u))) & 0xFFu) << (8 * k);
        }
      }
      __syncwarp();
      if (pw != 0 && lane == 0) mbar_arrive(info_empty(slot));
      if (n_list + n_tail == 0) continue;

      // ---- q: dims 0..255 into this warp's TMEM lanes, the rest by TMA, once the previous item's
      // logits MMAs have read theirs. Heads and dims past the query's own are zeros in TMEM; the TMA
      // part past the last dim is zero-filled, and rows past the last head only reach unused lanes.
      if (!warp_wait(q_empty, (n_q_loads & 1u) ^ 1u, 3)) break;
      ++n_q_loads;
      if (pw == 0 && lane == 0) {
        const int32_t atoms = (d_qk - C::Q_TMEM_DIMS + 63) / 64;
        if (atoms > 0) {
          mbar_expect_tx(q_full, static_cast<uint32_t>(atoms) * C::Q_ATOM);
          tma_pending = true;
          for (int32_t a = 0; a < atoms; ++a)
            tma_load_3d(sbase + C::OFF_QS + a * C::Q_ATOM, &map_q, q_full, C::Q_TMEM_DIMS + 64 * a,
                        m.qi * p.n_heads, 0);
        } else {
          mbar_arrive(q_full);
        }
      }
      {
        tc_fence_after();
        const int32_t head = 32 * static_cast<int32_t>(warp & 3u) + static_cast<int32_t>(lane);
        const int32_t dim0 = 128 * static_cast<int32_t>(pw >> 2);
        const __nv_bfloat16* qrow = p.q + (static_cast<size_t>(m.qi) * p.n_heads + head) * d_qk + dim0;
        uint32_t r[4][16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const bool in = head < p.n_heads && dim0 + 8 * c < d_qk;
          const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(qrow) + c) : make_uint4(0, 0, 0, 0);
          r[c >> 2][4 * (c & 3) + 0] = u.x;
          r[c >> 2][4 * (c & 3) + 1] = u.y;
          r[c >> 2][4 * (c & 3) + 2] = u.z;
          r[c >> 2][4 * (c & 3) + 3] = u.w;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_st16(tmem + ((32u * (warp & 3u)) << 16) + C::COL_Q + dim0 / 2 + 16 * c, r[c]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }

      // ---- the blocks. Row i of this warp is row ROWS*pw + i of the block; within a tile its 16-byte
      // chunk c of dims 8c.. is at atom c / 8, swizzled by i.
      const uint32_t row_off = C::OFF_STAGE + pw * 1024u;
      auto chunk_at = [&](uint32_t st, uint32_t i, uint32_t c) {
        return sbase + row_off + st * C::STAGE_BYTES + (c >> 3) * C::ATOM + i * 128u + (((c & 7u) ^ i) << 4);
      };
      const int32_t chunks = d_qk / 8, chunks_even = (chunks + 1) & ~1;   // a K step is two chunks
      auto announce = [&](uint32_t st) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(st));
      };
      // position of entry `lane` (< ROWS) of this warp in list block b, or -1
      auto entry = [&](int32_t b) -> int32_t {
        const int32_t j = m.e0 + b * C::BLK + C::ROWS * static_cast<int32_t>(pw) + static_cast<int32_t>(lane);
        if (b >= n_list || lane >= static_cast<uint32_t>(C::ROWS) || j >= end) return -1;
        const int32_t v = __ldg(idx_row + j);
        if (v >= p.max_len) {
          record_error(p.status, DSA_ERR_INDEX_RANGE, static_cast<uint32_t>(m.qi));
          return -1;
        }
        return v < 0 ? -1 : v;
      };
      // ROWS bf16 rows of a table (row r_i, or zeros where r_i < 0) into a stage by cp.async
      auto copy_rows = [&](uint32_t st, const __nv_bfloat16* table, int32_t rows) {
#pragma unroll
        for (int i = 0; i < C::ROWS; ++i) {
          const int32_t r = __shfl_sync(0xffffffffu, rows, i);
          const __nv_bfloat16* src = table + (r >= 0 ? static_cast<size_t>(r) * d_qk : 0);
          for (int32_t c = static_cast<int32_t>(lane); c < chunks_even; c += 32) {
            const bool in = r >= 0 && c < chunks;
            cp_async_16(chunk_at(st, i, c), src + (in ? 8 * c : 0), in ? 16u : 0u);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
      };
      bool ok = true;
      if constexpr (kQuant) {
        const int32_t groups = (p.d_latent + kScaleGroup - 1) / kScaleGroup;
        const uint8_t* codes = p.cache.codes + seq * p.max_len * static_cast<int64_t>(p.d_latent) + 16 * lane;
        const float* scales = p.cache.scales + seq * p.max_len * static_cast<int64_t>(groups) + (lane >> 3);
        const __nv_bfloat16* rope = p.cache.rope + seq * p.max_len * static_cast<int64_t>(p.d_rope) + 8 * (lane & 7u);
        const bool has_lat = static_cast<int32_t>(16 * lane) < p.d_latent;
        const bool has_rope = static_cast<int32_t>(8 * (lane & 7u)) < p.d_rope;
        const uint32_t lat_chunks = static_cast<uint32_t>(p.d_latent) / 8;
        const uint32_t rope_chunk = lat_chunks + (lane & 7u);
        // lanes of the two atoms that a store phase covers take their two chunks in opposite order,
        // so the phase's eight 16-byte stores fall into distinct banks
        const uint32_t swap = (lane >> 2) & 1u;
        uint4 raw[C::ROWS], rp[2];
        float sc[C::ROWS];
        auto load_row = [&](int i, int32_t rows) {
          const int32_t r = __shfl_sync(0xffffffffu, rows, i);
          const bool in = r >= 0 && has_lat;
          raw[i] = in ? __ldg(reinterpret_cast<const uint4*>(codes + static_cast<size_t>(r) * p.d_latent))
                      : make_uint4(0, 0, 0, 0);
          sc[i] = in ? __ldg(scales + static_cast<size_t>(r) * groups) : 0.f;
        };
        auto load_rope = [&](int t, int32_t rows) {
          const int32_t r = __shfl_sync(0xffffffffu, rows, 4 * t + (lane >> 3));
          rp[t] = r >= 0 && has_rope ? __ldg(reinterpret_cast<const uint4*>(rope + static_cast<size_t>(r) * p.d_rope))
                                     : make_uint4(0, 0, 0, 0);
        };
        int32_t rows = entry(0);
#pragma unroll
        for (int i = 0; i < C::ROWS; ++i) load_row(i, rows);
#pragma unroll
        for (int t = 0; t < 2; ++t) load_rope(t, rows);
        rows = entry(1);
        for (int32_t b = 0; b < n_list; ++b, ++nb) {
          const uint32_t st = nb & 1u;
          if (!warp_wait(empty(st), ((nb >> 1) & 1u) ^ 1u, 4)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < C::ROWS; ++i) {
            uint4 lo, hi;
            const Dequant expand(sc[i]);
            expand(raw[i], lo, hi);
            if (b + 1 < n_list) load_row(i, rows);
            if (has_lat) {
              st_shared_v4(chunk_at(st, i, 2 * lane + swap), swap ? hi : lo);
              st_shared_v4(chunk_at(st, i, 2 * lane + (swap ^ 1u)), swap ? lo : hi);
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (static_cast<int32_t>(rope_chunk) < chunks_even)
              st_shared_v4(chunk_at(st, 4 * t + (lane >> 3), rope_chunk), rp[t]);
            if (b + 1 < n_list) load_rope(t, rows);
          }
          rows = entry(b + 2);
          announce(st);
        }
      } else {
        const __nv_bfloat16* table = p.kv + seq * p.max_len * static_cast<int64_t>(d_qk);
        int32_t rows = entry(0);
        for (int32_t b = 0; b < n_list; ++b, ++nb) {
          const uint32_t st = nb & 1u;
          const int32_t next = entry(b + 1);
          if (!warp_wait(empty(st), ((nb >> 1) & 1u) ^ 1u, 5)) { ok = false; break; }
          copy_rows(st, table, rows);
          rows = next;
          announce(st);
        }
      }
      if constexpr (kTree) {
        const __nv_bfloat16* table = p.draft + seq * p.n_q * static_cast<int64_t>(d_qk);
        for (int32_t k = 0; k < n_tail && ok; ++k, ++nb) {
          const uint32_t st = nb & 1u;
          const uint32_t bits = static_cast<uint32_t>(path >> (8 * k)) & 0xFFu;
          const int32_t row = (k0 + k) * C::BLK + C::ROWS * static_cast<int32_t>(pw) + static_cast<int32_t>(lane);
          if (!warp_wait(empty(st), ((nb >> 1) & 1u) ^ 1u, 6)) { ok = false; break; }
          copy_rows(st, table, lane < static_cast<uint32_t>(C::ROWS) && ((bits >> lane) & 1u) ? row : -1);
          announce(st);
        }
      }
      if (!ok) break;
    }
    // after an abort: the q copy in flight lands before the CTA may leave. Its phase is the last begun
    if (tma_pending) attn_drain_wait(q_full, (n_q_loads - 1) & 1u, wt.aborted() ? kDrainBudgetNs : 0);
  } else if (warp == C::MMA_WARP) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = make_idesc(1, 1, 0, 0, 128, C::BLK);
      constexpr uint32_t idesc_o = make_idesc(1, 1, 0, 1, 128, C::OUT_DIMS);
      const int32_t k_steps = (d_qk + 15) / 16;
      uint32_t n_it = 0, n_busy = 0, nb = 0;
      bool ok = true;
      for (int32_t it = blockIdx.x; it < p.n_items && ok; it += gridDim.x, ++n_it) {
        const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
        if (!wt.wait(info_full(slot), sph, 10)) break;
        const int32_t n_blocks = info_base[slot * C::INFO_WORDS] + info_base[slot * C::INFO_WORDS + 2];
        mbar_arrive(info_empty(slot));
        if (n_blocks == 0) continue;
        const int32_t half = it % p.n_halves;
        if (!wt.wait(q_full, n_busy & 1u, 11)) break;
        // output of the item's block b - 1 after the logits of block b
        for (int32_t b = 0; b <= n_blocks; ++b) {
          if (b < n_blocks) {
            // the stage's last user was block nb - 2; a full stage means its output MMAs, which read
            // P from this logits buffer, are done
            const uint32_t st = nb & 1u;
            if (!wt.wait(full(st), (nb >> 1) & 1u, 12)) { ok = false; break; }
            tc_fence_after();
            const uint32_t tile = sbase + C::OFF_STAGE + st * C::STAGE_BYTES;
            const uint32_t d = tmem + C::COL_S + C::BLK * st;
#pragma unroll
            for (int k = 0; k < kDqk / 16; ++k) {
              if (k >= k_steps) break;
              const uint64_t bd = sw128_desc(tile + (k >> 2) * C::ATOM + (k & 3) * 32, 1, 1024);
              if (k < C::Q_TMEM_DIMS / 16) {
                mma_bf16_ts(d, tmem + C::COL_Q + 8 * k, bd, idesc_s, k > 0 ? 1u : 0u);
              } else {
                const int kq = k - C::Q_TMEM_DIMS / 16;
                mma_bf16_ss(d, sw128_desc(sbase + C::OFF_QS + (kq >> 2) * C::Q_ATOM + (kq & 3) * 32, 1, 1024), bd,
                            idesc_s, 1u);
              }
            }
            tc_commit(s_full(st));
            if (b == n_blocks - 1) tc_commit(q_empty);
          }
          if (b > 0) {
            const uint32_t pn = nb - 1, st = pn & 1u;
            if (!wt.wait(p_full(st), (pn >> 1) & 1u, 13)) { ok = false; break; }
            if (b == 1 && !wt.wait(o_empty, (n_busy & 1u) ^ 1u, 14)) { ok = false; break; }
            tc_fence_after();
            const uint32_t tile = sbase + C::OFF_STAGE + st * C::STAGE_BYTES + half * (C::OUT_DIMS / 64) * C::ATOM;
#pragma unroll
            for (int k = 0; k < C::BLK / 16; ++k)
              mma_bf16_ts(tmem + C::COL_O, tmem + C::COL_S + C::BLK * st + 8 * k,
                          sw128_desc(tile + k * 2048, C::ATOM, 1024), idesc_o, (b > 1 || k > 0) ? 1u : 0u);
            tc_commit(empty(st));
          }
          if (b < n_blocks) ++nb;
        }
        if (!ok) break;
        tc_commit(o_full);
        ++n_busy;
      }
      tc_commit(mma_done);
      attn_drain_wait(mma_done, 0, kDrainBudgetNs);
    }
  } else {
    // ================================================================ softmax (thread = head = TMEM lane)
    const int32_t head = static_cast<int32_t>(threadIdx.x);
    const uint32_t lane_off = (warp * 32u) << 16;
    const float sc = p.scale_log2;
    uint32_t n_it = 0, n_busy = 0, nb = 0;
    for (int32_t it = blockIdx.x; it < p.n_items; it += gridDim.x, ++n_it) {
      const Item m = item_of(it);
      const uint32_t slot = n_it & 1u, sph = (n_it >> 1) & 1u;
      if (!warp_wait(info_full(slot), sph, 20)) break;
      volatile int32_t* info = info_base + slot * C::INFO_WORDS;
      const int32_t n_list = info[0], end = info[1], n_tail = info[2], k0 = info[3];
      uint32_t path[kTree ? kMaxDraft / 32 : 1];
      if constexpr (kTree) {
#pragma unroll
        for (int w = 0; w < kMaxDraft / 32; ++w) path[w] = static_cast<uint32_t>(info[4 + w]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(info_empty(slot));
      const int32_t n_blocks = n_list + n_tail;
      const int32_t dim0 = C::OUT_DIMS * m.half, dims = min(C::OUT_DIMS, p.d_latent - dim0);
      const size_t row = static_cast<size_t>(m.qi) * p.n_heads + head;                       // (query, head)
      const size_t prow = (static_cast<size_t>(m.qi) * p.n_splits + m.split) * p.n_heads + head;
      const bool writes = head < p.n_heads;
      if (n_blocks == 0) {
        if (writes) {
          if (p.n_splits == 1) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + row * p.d_latent + dim0);
            for (int32_t c = 0; c < dims / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
            if (m.half == 0) p.lse[row] = -INFINITY;
          } else if (m.half == 0) {
            p.part_lse[prow] = -INFINITY;
          }
        }
        continue;
      }
      // entry `lane` / 32 + lane of list block b, read one block ahead: a ballot gives the valid rows
      const int32_t* idx_row = p.idx + static_cast<size_t>(m.qi) * p.topk;
      auto entry = [&](int32_t b, int32_t h) -> int32_t {
        const int32_t j = m.e0 + b * C::BLK + 32 * h + static_cast<int32_t>(lane);
        return b < n_list && j < end ? __ldg(idx_row + j) : -1;
      };
      int32_t v0 = entry(0, 0), v1 = entry(0, 1);
      float m2 = -INFINITY, l_r = 0.f, l_f = 0.f;        // running max; sums of rounded and unrounded weights
      bool ok = true;
      for (int32_t b = 0; b < n_blocks; ++b, ++nb) {
        const uint32_t st = nb & 1u;
        uint32_t vm0 = __ballot_sync(0xffffffffu, v0 >= 0 && v0 < p.max_len);
        uint32_t vm1 = __ballot_sync(0xffffffffu, v1 >= 0 && v1 < p.max_len);
        if constexpr (kTree) {
          if (b >= n_list) {
            const int32_t k = 2 * (k0 + b - n_list);
#pragma unroll
            for (int w = 0; w < kMaxDraft / 32; w += 2)
              if (w == k) { vm0 = path[w]; vm1 = path[w + 1]; }
          }
        }
        v0 = entry(b + 1, 0);
        v1 = entry(b + 1, 1);
        if (!warp_wait(s_full(st), (nb >> 1) & 1u, 21)) { ok = false; break; }
        tc_fence_after();
        uint32_t z[C::BLK];
        tmem_ld32(tmem + lane_off + C::COL_S + C::BLK * st, *reinterpret_cast<uint32_t(*)[32]>(&z[0]));
        tmem_ld32(tmem + lane_off + C::COL_S + C::BLK * st + 32, *reinterpret_cast<uint32_t(*)[32]>(&z[32]));
        tmem_wait_ld();
        if ((vm0 & vm1) != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < C::BLK; ++j)
            if (!(((j < 32 ? vm0 : vm1) >> (j & 31)) & 1u)) z[j] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < C::BLK; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(z[j]));
        const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;     // sc > 0
        const bool need = mb > m2 + kLazyRescale;
        float alpha = 1.0f;
        if (need) {
          alpha = m2 == -INFINITY ? 0.0f : ex2_approx(m2 - mb);
          m2 = mb;
          l_r *= alpha;
          l_f *= alpha;
        }
        // while every row seen so far was masked m2 is -inf: subtract 0, so that P = 2^-inf = 0
        const float msub = m2 == -INFINITY ? 0.0f : m2;
        uint32_t pk[C::BLK / 2];
        float fr[2] = {0.f, 0.f}, ff[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < C::BLK / 2; ++j) {
          const float a0 = ex2_approx(fmaf(__uint_as_float(z[2 * j]), sc, -msub));
          const float a1 = ex2_approx(fmaf(__uint_as_float(z[2 * j + 1]), sc, -msub));
          const __nv_bfloat162 pr = __floats2bfloat162_rn(a0, a1);
          const float2 back = __bfloat1622float2(pr);
          fr[0] += back.x;
          fr[1] += back.y;
          ff[0] += a0;
          ff[1] += a1;
          pk[j] = *reinterpret_cast<const uint32_t*>(&pr);
        }
        l_r += fr[0] + fr[1];
        l_f += ff[0] + ff[1];
        // ---- the output so far follows the raised max once the previous block's MMAs are in it
        if (b > 0 && __any_sync(0xffffffffu, need)) {
          if (!warp_wait(empty(st ^ 1u), ((nb - 1) >> 1) & 1u, 22)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < C::OUT_DIMS / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tmem + lane_off + C::COL_O + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 16; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tmem_st16(tmem + lane_off + C::COL_O + 16 * c, o);
          }
        }
        // ---- P over the logits: column j holds rows 2j and 2j+1
        tmem_st16(tmem + lane_off + C::COL_S + C::BLK * st, *reinterpret_cast<uint32_t(*)[16]>(&pk[0]));
        tmem_st16(tmem + lane_off + C::COL_S + C::BLK * st + 16, *reinterpret_cast<uint32_t(*)[16]>(&pk[16]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(st));
      }
      if (!ok) break;
      // ---- normalise and store. A sum of zero (no row attended) gives zeros and -inf.
      if (!warp_wait(o_full, n_busy & 1u, 23)) break;
      ++n_busy;
      tc_fence_after();
      const float inv = l_r == 0.f ? 0.f : 1.0f / l_r;
#pragma unroll 1
      for (int c = 0; c < C::OUT_DIMS / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_off + C::COL_O + 32 * c, o);
        tmem_wait_ld();
        if (!writes) continue;
        if (p.n_splits == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * p.d_latent + dim0 + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (32 * c + 8 * v >= dims) break;
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 pr = __floats2bfloat162_rn(__uint_as_float(o[8 * v + 2 * u]) * inv,
                                                              __uint_as_float(o[8 * v + 2 * u + 1]) * inv);
              w[u] = *reinterpret_cast<const uint32_t*>(&pr);
            }
            dst[v] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_out + prow * p.d_latent + dim0 + 32 * c);
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            if (32 * c + 4 * v >= dims) break;
            dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                 __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      if (writes && m.half == 0) {
        const float l2 = l_f == 0.f ? -INFINITY : m2 + log2f(l_f);
        if (p.n_splits == 1) p.lse[row] = l2 * 0.69314718055994531f;
        else p.part_lse[prow] = l2;
      }
    }
  }
  // ---- teardown: every role reaches here (all waits are bounded)
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the ranges of a query: with l_s the log-sum-exp of range s (log2 domain) and o_s its
// normalised output, w_s = 2^(l_s - max l), out = sum w_s o_s / sum w_s, lse = max l + log2 sum w_s.
// One CTA per (query, head), four dims per thread; a range without a row (l_s = -inf) wrote no
// output and is not read.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) cache_attn_join_kernel(
    const float* __restrict__ part_out, const float* __restrict__ part_lse, __nv_bfloat16* __restrict__ out,
    float* __restrict__ lse, int32_t n_splits, int32_t n_heads, int32_t d_latent) {
  const int64_t row = blockIdx.x;                        // (query, head)
  const int64_t qi = row / n_heads, head = row - qi * n_heads;
  const float* lrow = part_lse + qi * n_splits * n_heads + head;
  float mx = -INFINITY;
  for (int32_t s = 0; s < n_splits; ++s) mx = fmaxf(mx, __ldg(lrow + static_cast<int64_t>(s) * n_heads));
  float total = 0.f;
  const float msub = mx == -INFINITY ? 0.f : mx;
  const int32_t dim = 4 * static_cast<int32_t>(threadIdx.x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int32_t s = 0; s < n_splits; ++s) {
    const float l = __ldg(lrow + static_cast<int64_t>(s) * n_heads);
    const float w = exp2f(l - msub);
    total += w;
    if (l != -INFINITY && dim < d_latent) {
      const float4 o = __ldg(reinterpret_cast<const float4*>(
          part_out + ((qi * n_splits + s) * n_heads + head) * d_latent + dim));
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
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
