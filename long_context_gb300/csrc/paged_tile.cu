// Attention of many rows over a paged KV cache: prompt chunks, on the tensor
// cores (tcgen05, accumulators in TMEM, Q and the pages staged by TMA).
//
// A CTA has one block of rows of one KV head and one split of the keys (the
// schedule kernel's PagedWork).  The query heads that share the KV head are
// rows of one tile: a Q tile is 128 / group tokens by `group` heads (one TMA
// box), so a key tile is loaded once for all of them.  A key tile is 128 keys
// and comes as one box per page (or per 128 keys of a longer page), each lane
// of the producer warp issuing one; page numbers are read a tile ahead.
//
// The organisation is the ring-attention forward's (attn_fwd.cu):
//   warps 0-3, 4-7  softmax for Q tile 0, 1 (thread = row = TMEM lane)
//   warp  8, 11     TMA producers: Q once and K, V, through stage rings (pages
//                   of 16 tokens make eight or sixteen copies of a tile; one warp
//                   issuing both took 1,069 us for 4,864 tokens over 32,768,
//                   16 heads of 128, and two take 908, as with larger pages)
//   warp  9         MMA issuer (one thread) and TMEM owner
//   warp  10        waits for the MMA issuer, which an mbarrier wait would stall
//                   until its queued MMAs drain, and releases it through a named
//                   barrier; it also clears what the last V tile holds behind
//                   the cache's end (weight 0 times a NaN there would be NaN)
// TMEM (512 columns) at head size 128: S0 [0,128), S1 [128,256), O0 and O1 at
// 256 + t*D.  P_t (bf16, two per column) overwrites the first 64 columns of S_t,
// so S of the next key tile follows PV of this one and a Q tile's chain is
// softmax, hand-over, PV and S (about 2,900 cycles a key tile, of which the
// tensor pipe works 2,048 for two Q tiles).  Head size 64 has columns for three
// S: the products of both Q tiles take the buffers in turn, P again inside its S,
// and S of a Q tile's next key tile is there before its softmax needs it (4,864
// tokens over 32,768, 16 heads of 64: 724 us; with two S and a P of its own, S
// given back after the exponentials, 741 us, before them and so with a maximum of
// every tile, 783 us).
//
// Softmax: p = 2^(s scale log2 e - m) with a running reference m per row that
// only has to keep p below 2^16 (O and l share it, so O / l and m + ln l do not
// depend on it): the row maximum is taken while a row has no reference yet;
// later a tile is computed against the reference as it is, and again with its
// own maximum when its sum exceeds that bound or is not finite.  l sums p in
// fp32; O accumulates in fp32.  P is rounded to bf16 for its product with V, as in
// the packed forward, because the kernel is bound by its MMAs and what feeds them:
// with the rounding's remainder as a second operand (paged_rows.cu does that for up
// to 16 rows) O's error against 64 bits is 0.0017 instead of 0.0020-0.0024, for
// 1,012 instead of 746 us (2,048 tokens over 32,768, 32 / 8 heads of 128) and 1,068
// instead of 688 us (4,864 over 32,768, 16 / 4 heads of 64).  Values that are exact in
// fp16, those of a 4-bit cache's pages, take P in fp16: 2^-11 instead of 2^-8 of each
// weight for the same instructions (error 0.0017, the same times).  p is 2^7 at the
// reference: fp16 keeps its 11 bits of weights down to 2^-21 of that, is off by at most
// 2^-32 of it below and has zero for weights smaller than that, which l still sums; the
// reference moves whenever a tile's sum would pass 2^15.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr float kNegInfT = -__builtin_huge_valf();
constexpr float kLn2T = 0.69314718055994530942f;
// How P is held: bf16, or fp16 (pages of a 4-bit cache, whose values are exact in it).
template <bool HALF>
struct TileP {
  static constexpr float kMoveBy = HALF ? 0.0f : 8.0f;            // powers of two (see paged_rows.cu)
  static constexpr float kMaxSum = HALF ? 32768.0f : 65536.0f;    // bound of a tile's sum of p
  static constexpr float kLift = HALF ? 7.0f : 0.0f;  // powers of two of p at the reference
};

template <int D>
struct TileCfg {
  static constexpr int kHalves = D / 64;          // 128-byte swizzle atoms
  static constexpr int kTileBytes = 128 * D * 2;  // one 128-row bf16 tile
  static constexpr int kStages = (D == 64) ? 4 : 2;
  // Head size 64 leaves TMEM columns for a third S: product s (of tile s / nq and
  // Q tile s % nq) goes to buffer s % 3.
  static constexpr bool kRing = D == 64;
  static constexpr int kBufs = kRing ? 3 : kNQ;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kNQ * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kBarOff = kVOff + kStages * kTileBytes;
  // q_full, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full[NQ],
  // p_full[NQ], o_done[NQ], drain, staged[NQ]; s_full[kBufs] instead with a ring
  static constexpr int kNumBars = 1 + 4 * kStages + kBufs + 2 * kNQ + 1 + kNQ;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 64 + 1024;  // + align slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kOCol = kBufs * kBN;
  static_assert(kOCol + kNQ * D <= kTmemCols);
};

// Byte offset of 16-byte chunk c of row r in a tile stored as 64-column
// halves of 128-byte rows with the 128-byte swizzle (the TMA load layout).
__device__ __forceinline__ int swizzle_at(int r, int c) {
  return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Wait that ignores the CTA abort flag (used to drain copies in flight).
__device__ __forceinline__ bool drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > 200000000ull) return false;  // 0.2 s
  }
  return true;
}

}  // namespace

template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_o, const PagedParams p) {
  using C = TileCfg<D>;
  using P = TileP<HALF>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The heads of a split run together; a head's blocks walk its keys in step,
  // so most of them come from L2.  The loads are in flight together: the list has
  // room for every CTA of the grid.
  const int e = static_cast<int>(blockIdx.x) / p.num_kv_heads;
  const int h = static_cast<int>(blockIdx.x) - e * p.num_kv_heads;
  const int n_work = __ldcg(&p.hdr->n_items);
  const int err0 = __ldcg(&p.hdr->error);
  const int4* wp = reinterpret_cast<const int4*>(p.work + e);
  const int4 w0 = __ldcg(wp), w1 = __ldcg(wp + 1);
  if (e >= n_work) return;
  if (__syncthreads_or(says_timeout(err0))) return;
  const int tok0 = w0.x, q_len = w0.y, kv_len = w0.z, seq = w0.w;
  const int kv_lo = w1.y, kv_hi = w1.z, slot = w1.w;
  const int G = p.group;
  const int tile_toks = p.shape.rows / (kNQ * G);  // tokens of a Q tile
  const int tile_rows = tile_toks * G;
  // The sequence's blocks are aligned to its end, so only block 0 can be
  // short; its Q tiles start before the sequence (TMA fills rows before the
  // array with zeros), and a Q tile without rows is left out.
  const int blk_toks = kNQ * tile_toks;
  const int n_blk = (q_len + blk_toks - 1) / blk_toks;
  const int tok_hi = q_len - (n_blk - 1 - w1.x) * blk_toks;
  const int nq = tok_hi > tile_toks ? kNQ : 1;
  const int tok_lo = tok_hi - nq * tile_toks;  // first token of Q tile 0
  const int n = (kv_hi - kv_lo + kBN - 1) / kBN;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* k_empty = k_full + C::kStages;
  uint64_t* v_full = k_empty + C::kStages;
  uint64_t* v_empty = v_full + C::kStages;
  uint64_t* s_full = v_empty + C::kStages;
  uint64_t* p_full = s_full + C::kBufs;
  uint64_t* o_done = p_full + kNQ;
  uint64_t* drain = o_done + kNQ;
  uint64_t* staged = drain + 1;  // O tile t staged in shared memory (128 arrivals)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Pages: a tile's boxes are `box` keys each; lane l of the producer has box
  // l / halves, feature half l % halves.
  const int box = min(1 << p.page_shift, kBN);
  const int my_key = (lane / C::kHalves) * box;
  const int my_col = (lane % C::kHalves) * 64;
  const int* pages = p.page_table + static_cast<size_t>(seq) * p.max_pages;
  auto page_of = [&](int kv0) {  // page of this lane's box of the tile at kv0; -1: no box
    const int key = kv0 + my_key;
    if (my_key >= kBN || key >= kv_len) return -1;
    const int page = __ldg(pages + (key >> p.page_shift));
    if (page >= 0 && page < p.num_pages) return page;
    atomicCAS(&p.hdr->error, 0, kPagedBad);
    return p.num_pages;  // out of range: the copy fills zeros
  };
  auto copy_tile = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int kv0, int page,
                       uint64_t policy) {
    if (lane == 0)
      mbar_arrive_expect_tx(bar, (min(kv_len - kv0, kBN) + box - 1) / box * box * D * 2);
    __syncwarp();
    if (page >= 0)
      tma_load_4d(dst + (my_col >> 6) * 16384 + my_key * 128, map, bar, my_col, h,
                  (kv0 + my_key) & ((1 << p.page_shift) - 1), page, policy);
  };

  // The producer warp sets up the barriers and starts the copies of Q and of
  // the first K/V tile before the CTA-wide barrier, so that their latency
  // overlaps the TMEM allocation and the barrier.
  if (warp == 8) {
    if (lane == 0) {
      mbar_init(q_full, 1);
      for (int st = 0; st < C::kStages; ++st) {
        mbar_init(&k_full[st], 1);
        mbar_init(&k_empty[st], 1);
        mbar_init(&v_full[st], 1);
        mbar_init(&v_empty[st], 1);
      }
      for (int t = 0; t < kNQ; ++t) {
        mbar_init(&s_full[t], 1);
        mbar_init(&p_full[t], kBM);
        mbar_init(&o_done[t], 1);
      }
      mbar_init(drain, 1);
      for (int t = 0; t < kNQ; ++t) mbar_init(&staged[t], kBM);
      for (int b = kNQ; b < C::kBufs; ++b) mbar_init(&s_full[b], 1);
      *abort_flag = 0;
      fence_mbarrier_init();
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      const uint64_t pol_q = l2_policy_evict_first();
      mbar_arrive_expect_tx(q_full, nq * tile_rows * D * 2);
      for (int t = 0; t < nq; ++t)
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem + C::kQOff + t * C::kTileBytes + hf * 16384, &tm_q, q_full, hf * 64,
                      h * G, tok0 + tok_lo + t * tile_toks, pol_q);
    }
    __syncwarp();
    if (n > 0) {  // tile 0 goes to stage 0, which is free
      const uint64_t pol_kv = l2_policy_evict_last();
      const int page = page_of(kv_lo);
      copy_tile(&tm_k, smem + C::kKOff, &k_full[0], kv_lo, page, pol_kv);
      copy_tile(&tm_v, smem + C::kVOff, &v_full[0], kv_lo, page, pol_kv);
    }
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  static_assert(kSoftmaxRegs == 224 && kCtrlRegs == 56, "immediates below");

  if (warp >= 8) {
    regs_lower_56();
    if (warp == 8 || warp == 11) {
      // ------------------------------ TMA producers: warp 8 K, warp 11 V --
      const bool is_k = warp == 8;
      const uint64_t pol_kv = l2_policy_evict_last();
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      uint8_t* ring = smem + (is_k ? C::kKOff : C::kVOff);
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      int issued = min(n, 1);  // tiles whose copies were issued
      bool ok = true;
      int next_page = n > 1 ? page_of(kv_lo + kBN) : -1;
      for (int x = 1; x < n; ++x) {
        const int st = x % C::kStages;
        const uint32_t ph = (x / C::kStages) & 1;
        const int kv0 = kv_lo + x * kBN;
        const int page = next_page;
        if (x + 1 < n) next_page = page_of(kv0 + kBN);
        ok = __all_sync(0xffffffffu, wait_bounded(&empty[st], ph ^ 1, abort_flag));
        if (!ok) break;
        copy_tile(map, ring + st * C::kTileBytes, &full[st], kv0, page, pol_kv);
        ++issued;
      }
      if (lane == 0) {
        if (!ok) {
          atomicCAS(&p.hdr->error, 0, kPagedLate);
          *abort_flag = 1;
        }
        // Drain: every copy issued into shared memory must land before exit.
        if (is_k) drain_wait(q_full, 0);
        for (int st = 0; st < C::kStages; ++st)
          if (st < issued) {
            const int last = st + ((issued - 1 - st) / C::kStages) * C::kStages;
            drain_wait(&full[st], (last / C::kStages) & 1);
          }
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------- MMA issuer --
      // Lane 0 issues every MMA and never touches an mbarrier in the loop
      // (both warps 9 and 10 run the same number of rendezvous).
      constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, false);
      // (Bits 7 and 10 are bf16 instead of fp16.)
      constexpr uint32_t idesc_o =
          idesc_bf16_f32(kBM, D, true) & ~(HALF ? (1u << 7) | (1u << 10) : 0u);
      const uint32_t hi_kq = static_cast<uint32_t>(sdesc_sw128(0, 16, 1024) >> 32);
      const uint32_t hi_v = static_cast<uint32_t>(sdesc_sw128(0, 16384, 1024) >> 32);
      const uint32_t lo_q =
          static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024));
      const uint32_t lo_k =
          static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024));
      const uint32_t lo_v =
          static_cast<uint32_t>(sdesc_sw128(smem_u32(smem + C::kVOff), 16384, 1024));
      auto issue_s = [&](int t, int st, int buf) {
        const uint32_t d = tmem + buf * kBN;
        const uint32_t a0 = lo_q + t * (C::kTileBytes >> 4);
        const uint32_t b0 = lo_k + st * (C::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          mma_ss(d, pack_u64(a0 + off, hi_kq), pack_u64(b0 + off, hi_kq), idesc_s,
                 kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[buf]);
      };
      auto issue_pv = [&](int t, int st, int buf, bool acc) {
        const uint32_t d = tmem + C::kOCol + t * D;
        const uint32_t a = tmem + buf * kBN;
        const uint32_t b0 = lo_v + st * (C::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          mma_ts(d, a + kk * 8, pack_u64(b0 + ((kk * 2048) >> 4), hi_v), idesc_o,
                 (acc || kk > 0) ? 1u : 0u);
      };
      if constexpr (C::kRing) {
        // The first three products of Q and K, then after P_s's product with V the
        // product s + 3 into the buffer that P_s leaves (in issue order).
        const int total = n * nq;
        auto next_s = [&](int s) {
          const int x = s / nq, t = s - x * nq, st = x % C::kStages;
          issue_s(t, st, s % C::kBufs);
          if (t == nq - 1) mma_commit(&k_empty[st]);
        };
        for (int s = 0; s < min(total, C::kBufs); ++s) {
          named_bar_sync(1, 64);  // Q and its K landed
          if (lane == 0) {
            tc_fence_after();
            next_s(s);
          }
          __syncwarp();
        }
        for (int s = 0; s < total; ++s) {
          named_bar_sync(1, 64);  // P_s, its V and the K of product s + 3 are ready
          if (lane == 0) {
            tc_fence_after();
            const int x = s / nq, t = s - x * nq, st = x % C::kStages;
            issue_pv(t, st, s % C::kBufs, x > 0);
            mma_commit(&o_done[t]);
            if (t == nq - 1) mma_commit(&v_empty[st]);
            if (s + C::kBufs < total) next_s(s + C::kBufs);
          }
          __syncwarp();
        }
      } else {
        named_bar_sync(1, 64);  // Q and K(0) landed
        if (lane == 0 && n > 0) {
          tc_fence_after();
          for (int t = 0; t < nq; ++t) issue_s(t, 0, t);
          mma_commit(&k_empty[0]);
        }
        __syncwarp();
        for (int x = 0; x < n; ++x) {
          const int st = x % C::kStages;
          const bool has_next = x + 1 < n;
          const int st1 = (x + 1) % C::kStages;
          for (int t = 0; t < nq; ++t) {
            named_bar_sync(1, 64);  // P_t(x), V(x) and K(x+1) are ready
            if (lane == 0) {
              tc_fence_after();
              issue_pv(t, st, t, x > 0);
              if (!has_next) mma_commit(&o_done[t]);
              if (t == nq - 1) mma_commit(&v_empty[st]);
              if (has_next) {
                issue_s(t, st1, t);
                if (t == nq - 1) mma_commit(&k_empty[st1]);
              }
            }
            __syncwarp();
          }
        }
      }
      if (lane == 0) {
        mma_commit(drain);
        drain_wait(drain, 0);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ------------------------------------------------ waits for the MMAs --
      // After a failed (bounded) wait the remaining rendezvous still happen,
      // without waiting, so the MMA warp always runs to its end.
      bool ok = true;
      auto clear_v = [&](int x) {
        const int used = kv_len - (kv_lo + x * kBN);
        if (used < kBN) {
          // The cache ends in this tile: clear V behind it (and tell the
          // tensor core's proxy).
          ok = __shfl_sync(0xffffffffu, ok, 0);
          uint8_t* v = smem + C::kVOff + (x % C::kStages) * C::kTileBytes;
          for (int i = used * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
              *reinterpret_cast<uint4*>(v + hf * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
      };
      if constexpr (C::kRing) {
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (lane == 0 && ok) ok = wait_bounded(bar, parity, abort_flag);
        };
        auto wait_k = [&](int x) { wait(&k_full[x % C::kStages], (x / C::kStages) & 1); };
        wait(q_full, 0);
        const int total = n * nq;
        for (int s = 0; s < min(total, C::kBufs); ++s) {
          wait_k(s / nq);
          __syncwarp();
          named_bar_sync(1, 64);
        }
        for (int s = 0; s < total; ++s) {
          const int x = s / nq, t = s - x * nq;
          if (t == 0) {
            wait(&v_full[x % C::kStages], (x / C::kStages) & 1);
            clear_v(x);
          }
          if (s + C::kBufs < total) wait_k((s + C::kBufs) / nq);
          wait(&p_full[t], x & 1);
          __syncwarp();
          named_bar_sync(1, 64);
        }
      } else {
        if (lane == 0) {
          ok = wait_bounded(q_full, 0, abort_flag);
          if (ok && n > 0) ok = wait_bounded(&k_full[0], 0, abort_flag);
        }
        __syncwarp();
        named_bar_sync(1, 64);
        for (int x = 0; x < n; ++x) {
          const int st = x % C::kStages;
          const uint32_t ph = (x / C::kStages) & 1;
          const int st1 = (x + 1) % C::kStages;
          const uint32_t ph1 = ((x + 1) / C::kStages) & 1;
          for (int t = 0; t < nq; ++t) {
            if (t == 0) {
              if (lane == 0 && ok) ok = wait_bounded(&v_full[st], ph, abort_flag);
              clear_v(x);
              if (lane == 0 && ok && x + 1 < n)
                ok = wait_bounded(&k_full[st1], ph1, abort_flag);
            }
            if (lane == 0 && ok) ok = wait_bounded(&p_full[t], x & 1, abort_flag);
            __syncwarp();
            named_bar_sync(1, 64);
          }
        }
      }
      if (lane == 0 && !ok) {
        atomicCAS(&p.hdr->error, 0, kPagedLate);
        *abort_flag = 1;
      }
      __syncwarp();
    }
  } else {
    regs_raise_224();
    if (warp < 4 * nq) {
      // ---------------------------------------------------------- softmax --
      const int t = warp >> 2;
      const int r = threadIdx.x & 127;
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t o_addr = tmem + lane_base + C::kOCol + t * D;
      const int my_tok = tok_lo + t * tile_toks + r / G;
      const bool row_valid = r < tile_rows && my_tok >= 0;
      // Keys below lim are visible; a row that is not there sees none, and
      // its reference is 0 so that it never asks for a maximum.
      const int lim = !row_valid ? 0 : (p.causal ? kv_len - q_len + my_tok + 1 : kv_len);
      const float c_log2 = p.scale_log2;
      float m_run = row_valid ? kNegInfT : 0.f;  // log2 domain
      float l_run = 0.f;
      bool ok = true;

      for (int x = 0; x < n; ++x) {
        // P goes where S was.
        const int s = x * nq + t;
        const int buf = C::kRing ? s % C::kBufs : t;
        const uint32_t s_addr = tmem + lane_base + buf * kBN;
        ok = __all_sync(0xffffffffu,
                        wait_bounded(&s_full[buf], (C::kRing ? s / C::kBufs : x) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // S is still in TMEM for a second pass: P is written after it.
        bool with_max = __any_sync(0xffffffffu, m_run == kNegInfT);
        float2 acc0, acc1;
        uint32_t pk[kBN / 2];
#pragma unroll 1
        for (;;) {
          uint32_t sr[kBN];
#pragma unroll
          for (int q = 0; q < kBN / 32; ++q) tmem_ld32(s_addr + q * 32, sr + q * 32);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < kBN / 32; ++q) reg_fence32(sr + q * 32);

          // Visible keys of this row form a prefix of the tile.
          const int nvis = lim - (kv_lo + x * kBN);
          if (nvis < kBN) {
#pragma unroll
            for (int cc = 0; cc < kBN; ++cc)
              if (cc >= nvis) sr[cc] = __float_as_uint(kNegInfT);
          }
          if (with_max) {
            float mx0 = fmaxf(__uint_as_float(sr[0]), __uint_as_float(sr[1]));
            float mx1 = fmaxf(__uint_as_float(sr[2]), __uint_as_float(sr[3]));
            float mx2 = fmaxf(__uint_as_float(sr[4]), __uint_as_float(sr[5]));
            float mx3 = fmaxf(__uint_as_float(sr[6]), __uint_as_float(sr[7]));
#pragma unroll
            for (int cc = 8; cc < kBN; cc += 8) {
              mx0 = fmax3(mx0, __uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1]));
              mx1 = fmax3(mx1, __uint_as_float(sr[cc + 2]), __uint_as_float(sr[cc + 3]));
              mx2 = fmax3(mx2, __uint_as_float(sr[cc + 4]), __uint_as_float(sr[cc + 5]));
              mx3 = fmax3(mx3, __uint_as_float(sr[cc + 6]), __uint_as_float(sr[cc + 7]));
            }
            const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * c_log2;
            const float m_new = fmaxf(m_run, m_tile);
            if (__any_sync(0xffffffffu, m_new > m_run + P::kMoveBy)) {
              const float alpha = (m_run == kNegInfT) ? 0.f : ex2_approx(m_run - m_new);
              if (C::kRing && x > 0) {
                ok = __all_sync(0xffffffffu, wait_bounded(&o_done[t], (x - 1) & 1, abort_flag));
                tc_fence_after();
              }
              if (x > 0) {
                // PV of the previous tile has completed: it was waited for, or
                // came before S of this one (same issuing thread, committed in
                // order).  O_t is stable here.
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                  uint32_t orr[32];
                  tmem_ld32(o_addr + q * 32, orr);
                  tmem_wait_ld();
                  reg_fence32(orr);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                  tmem_st32(o_addr + q * 32, orr);
                }
              }
              l_run *= alpha;
              m_run = m_new;
            }
          }
          const float mref = (m_run == kNegInfT) ? 0.f : m_run;
          const float2 c2 = make_float2(c_log2, c_log2);
          const float2 nm2 = make_float2(P::kLift - mref, P::kLift - mref);
          acc0 = make_float2(0.f, 0.f);
          acc1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int k2 = 0; k2 < kBN / 2; ++k2) {
            const float2 xs = __ffma2_rn(
                make_float2(__uint_as_float(sr[2 * k2]), __uint_as_float(sr[2 * k2 + 1])), c2, nm2);
            const float2 pp = make_float2(ex2_approx(xs.x), ex2_approx(xs.y));
            if (k2 & 1) acc1 = __fadd2_rn(acc1, pp); else acc0 = __fadd2_rn(acc0, pp);
            pk[k2] = HALF ? pack_f16x2(pp.x, pp.y) : pack_bf16x2(pp.x, pp.y);
          }
          if (with_max) break;
          const float l_tile = (acc0.x + acc1.x) + (acc0.y + acc1.y);
          if (!__any_sync(0xffffffffu, !(l_tile <= P::kMaxSum))) break;
          with_max = true;
        }
        l_run += (acc0.x + acc1.x) + (acc0.y + acc1.y);
        if (C::kRing && x > 0) {  // one phase of o_done[t] at a time: its parity tells only two
          ok = __all_sync(0xffffffffu,
                          ok && wait_bounded(&o_done[t], (x - 1) & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32(s_addr, pk);
        tmem_st32(s_addr + 32, pk + 32);
        tmem_wait_st();
        tc_fence_before();
#ifdef CPATTN_FAULT_INJECT_DROP_P
        // Test-only build: CTA 0 never hands its first P tile of Q tile 0 to the
        // MMA warp, whose bounded wait then runs out (no trap, no fault).
        if (!(blockIdx.x == 0 && t == 0 && x == 0))
#endif
          mbar_arrive(&p_full[t]);
      }
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu,
                        wait_bounded(&o_done[t], C::kRing ? (n - 1) & 1 : 0, abort_flag));
        tc_fence_after();
      }
      if (ok) {
        // Epilogue: O / l and LSE = m + ln l; zeros where no key is visible.
        const bool none = l_run == 0.f;
        const float inv_l = none ? 0.f : (HALF ? p.v_unit : 1.f) / l_run;
        const float lse =
            none ? kNegInfT : ((HALF ? m_run - P::kLift : m_run) + __log2f(l_run)) * kLn2T;
        uint32_t orr[D];
        if (n > 0) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) tmem_ld32(o_addr + q * 32, orr + q * 32);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < D / 32; ++q) reg_fence32(orr + q * 32);
        } else {
#pragma unroll
          for (int e = 0; e < D; ++e) orr[e] = 0u;
        }
        if (slot >= 0) {
          // A split: normalised fp32 rows for the merge kernel.
          if (row_valid) {
            const size_t part = (static_cast<size_t>(slot) * p.num_kv_heads + h) * p.shape.rows +
                                (kNQ - nq + t) * tile_rows + r;
            float4* dst = reinterpret_cast<float4*>(p.o_part + part * D);
#pragma unroll
            for (int e = 0; e < D; e += 4)
              dst[e / 4] = make_float4(
                  __uint_as_float(orr[e]) * inv_l, __uint_as_float(orr[e + 1]) * inv_l,
                  __uint_as_float(orr[e + 2]) * inv_l, __uint_as_float(orr[e + 3]) * inv_l);
            p.lse_part[part] = lse;
          }
        } else {
          // The rows go out through Q tile t's buffer (every MMA reading it
          // completed before o_done[t]; without keys, Q landed before this
          // CTA's first rendezvous and nothing reads it).
          uint8_t* stage = smem + C::kQOff + t * C::kTileBytes;
          if (n == 0) ok = __all_sync(0xffffffffu, wait_bounded(q_full, 0, abort_flag));
          fence_proxy_async_smem();
          const float2 il2 = make_float2(inv_l, inv_l);
#pragma unroll
          for (int q = 0; q < D / 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 o2 = __fmul2_rn(make_float2(__uint_as_float(orr[q * 8 + 2 * e]),
                                                       __uint_as_float(orr[q * 8 + 2 * e + 1])),
                                           il2);
              w[e] = pack_bf16x2(o2.x, o2.y);
            }
            *reinterpret_cast<uint4*>(stage + swizzle_at(r, q)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (tok_lo + t * tile_toks >= 0) {
            // A full tile: the staged layout is the TMA layout, so one thread
            // stores it with the bulk engine once every row is staged.
            fence_proxy_async_smem();
            mbar_arrive(&staged[t]);
            if ((warp & 3) == 0 && lane == 0) {
              if (wait_bounded(&staged[t], 0, abort_flag)) {
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                  tma_store_3d(&tm_o, stage + hf * 16384, hf * 64, h * G,
                               tok0 + tok_lo + t * tile_toks);
                bulk_commit_group();
                bulk_wait_group_read0();
              } else {
                ok = false;
              }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
          } else {
            // The tile that starts a short block: its rows before the sequence
            // belong to another one, so the warp copies its own 32 rows out
            // with D / 8 lanes per row, skipping those.
            __syncwarp();
            constexpr int kLpr = D / 8;      // lanes per row: one 16-byte chunk each
            constexpr int kRpi = 32 / kLpr;  // rows per store instruction
            const int c = lane % kLpr;
#pragma unroll 4
            for (int it = 0; it < 32 / kRpi; ++it) {
              const int rr = (warp & 3) * 32 + it * kRpi + lane / kLpr;
              const uint4 val = *reinterpret_cast<const uint4*>(stage + swizzle_at(rr, c));
              const int tok = tok_lo + t * tile_toks + rr / G;
              if (rr < tile_rows && tok >= 0)
                *reinterpret_cast<uint4*>(
                    p.out + (static_cast<size_t>(tok0 + tok) * p.num_heads + h * G + rr % G) * D +
                    c * 8) = val;
            }
          }
          if (row_valid && p.lse != nullptr)
            p.lse[static_cast<size_t>(tok0 + my_tok) * p.num_heads + h * G + r % G] = lse;
        }
        tc_fence_before();
      }
      if (!ok) {
        atomicCAS(&p.hdr->error, 0, kPagedLate);
        *abort_flag = 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool HALF>
static cudaError_t launch_paged_tile_t(const CUtensorMap& tq, const CUtensorMap& tk,
                                       const CUtensorMap& tv, const CUtensorMap& to,
                                       const PagedParams& p, cudaStream_t stream) {
  auto kern = paged_tile_kernel<D, HALF>;
  // The register split inside the kernel assumes exactly kLaunchRegs per
  // thread at launch; with any other count the raise could wait forever.
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             TileCfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.max_work * p.num_kv_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = TileCfg<D>::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, to, p);
}

cudaError_t launch_paged_tile(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const PagedParams& p, int D,
                              cudaStream_t stream) {
  if (p.v_half)
    return D == 64 ? launch_paged_tile_t<64, true>(tq, tk, tv, to, p, stream)
                   : launch_paged_tile_t<128, true>(tq, tk, tv, to, p, stream);
  return D == 64 ? launch_paged_tile_t<64, false>(tq, tk, tv, to, p, stream)
                 : launch_paged_tile_t<128, false>(tq, tk, tv, to, p, stream);
}

}  // namespace cpattn
