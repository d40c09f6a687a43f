// The work list of a small decoding step, worked out by every warp for itself.
//
// Up to 32 sequences of one block of rows each, one a lane: the lengths are read,
// the share computed and the splits counted with shuffles in every warp that needs
// a split or a merge, so that no kernel has to write a list first.  (17 sequences
// of drafts 36.1 -> 32.9 us, a token or two of two short sequences 12.4 -> 10.3 us
// against a schedule kernel before the attention kernel.  With four sequences a
// lane, batches of 65 took 28.6 instead of 26.9 us.)
#pragma once

#include "kernels.h"

namespace cpattn {

constexpr int kPlanSeqs = 32;

struct PagedPlan {
  int lo, hi, kv;   // this lane's sequence: cu_seqlens and kv_lens
  int n, per;       // its splits, the units of a split
  int base;         // its first split
  int slot, item;   // its first slot (-1: whole) and its number among the split items
  int splits, merges;
  bool bad;
};

// Every lane of the warp executes it.
__device__ __forceinline__ PagedPlan make_plan(const PagedParams& p, int lane) {
  PagedPlan t;
  const bool in = lane < p.num_seqs;
  t.lo = in ? __ldg(p.cu_seqlens + lane) : 0;
  t.hi = in ? __ldg(p.cu_seqlens + lane + 1) : 0;
  t.kv = in ? __ldg(p.kv_lens + lane) : 0;
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  t.bad = __any_sync(0xffffffffu,
                     t.lo < 0 || t.hi < t.lo || t.hi > p.total_q || t.hi - t.lo > p.max_seqlen ||
                         t.kv < 0 || t.kv > p.max_kv_len || t.kv > cap ||
                         (lane == 0 && t.lo != 0));
  t.n = t.hi > t.lo ? 1 : 0;
  const int units = t.n ? (t.kv + p.shape.unit - 1) / p.shape.unit : 0;
  const int items = __popc(__ballot_sync(0xffffffffu, t.n > 0));
  long long all = units;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  int target = paged_rows_target(p.shape, all, items, p.num_kv_heads);
  if (p.shape.fit && 2 * items * p.num_kv_heads <= p.shape.round) {
    // The smallest that needs no more splits than a round has CTAs for a head: at most the
    // share above, for which a split more of every item was set aside.  (25 rows over 17
    // caches of 1 to 20,000 keys of 4-bit codes, 4 heads of 128: 61.5 -> 54.6 us; 16 rows
    // over 24 of 1,000 to 30,000, 8 heads: 170 -> 128.)
    const int slots = p.shape.round / p.num_kv_heads;
    int least = static_cast<int>(max((all + slots - 1) / slots, 1ll));
    while (least < target) {
      const int mid = (least + target) >> 1;
      const int need =
          static_cast<int>(__reduce_add_sync(0xffffffffu, (units + mid - 1) / mid + (t.n && !units)));
      if (need <= slots) target = mid;
      else least = mid + 1;
    }
  }
  t.per = units;
  if (units > target) {
    const int n = (units + target - 1) / target;
    t.per = (units + n - 1) / n;
    t.n = (units + t.per - 1) / t.per;
  }
  // First split, slot and number among the split items, in one scan (slots and
  // merges < 2^16).
  const long long v = t.n + (t.n > 1 ? (static_cast<long long>(t.n) << 32) + (1ll << 48) : 0);
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += w;
  }
  const long long before = incl - v, total = __shfl_sync(0xffffffffu, incl, 31);
  t.base = static_cast<int>(before & 0xffffffffll);
  t.slot = t.n > 1 ? static_cast<int>((before >> 32) & 0xffff) : -1;
  t.item = static_cast<int>(before >> 48);
  t.splits = t.bad ? 0 : static_cast<int>(total & 0xffffffffll);
  t.merges = t.bad ? 0 : static_cast<int>(total >> 48);
  return t;
}

// Split e (below t.splits) as the schedule kernel would list it.
__device__ __forceinline__ PagedWork plan_split(const PagedParams& p, const PagedPlan& t, int e) {
  const int b =
      __ffs(__ballot_sync(0xffffffffu, t.n > 0 && t.base <= e && e < t.base + t.n)) - 1;
  PagedWork w = {};
  w.seq = b;
  w.tok0 = __shfl_sync(0xffffffffu, t.lo, b);
  w.q_len = __shfl_sync(0xffffffffu, t.hi, b) - w.tok0;
  w.kv_len = __shfl_sync(0xffffffffu, t.kv, b);
  const int s = e - __shfl_sync(0xffffffffu, t.base, b);
  const int step = __shfl_sync(0xffffffffu, t.per, b) * p.shape.unit;
  w.kv_lo = s * step;
  w.kv_hi = min(w.kv_len, (s + 1) * step);
  w.slot0 = __shfl_sync(0xffffffffu, t.slot, b);
  w.slot = w.slot0 < 0 ? -1 : w.slot0 + s;
  w.n = __shfl_sync(0xffffffffu, t.n, b);
  w.item = __shfl_sync(0xffffffffu, t.item, b);
  return w;
}

// Split item m (below t.merges).
__device__ __forceinline__ PagedMerge plan_merge(const PagedPlan& t, int m) {
  const int b = __ffs(__ballot_sync(0xffffffffu, t.n > 1 && t.item == m)) - 1;
  PagedMerge g = {};
  g.tok0 = __shfl_sync(0xffffffffu, t.lo, b);
  g.q_len = __shfl_sync(0xffffffffu, t.hi, b) - g.tok0;
  g.slot0 = __shfl_sync(0xffffffffu, t.slot, b);
  g.n = __shfl_sync(0xffffffffu, t.n, b);
  return g;
}

}  // namespace cpattn
