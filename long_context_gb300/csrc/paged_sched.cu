// Attention over a paged KV cache: the work list, and the merge of splits.
//
// The schedule kernel reads the lengths on the device (a captured graph can be
// replayed with other lengths) and cuts the work.  W is the units of keys over
// all items of one KV head; every KV head is cut alike.
//
// Few rows (HBM bound; two CTAs a SM): an item of u units becomes
// ceil(u / target) equal splits (see paged_rows_target).
//
// Tiles (one CTA a SM, an item is up to hundreds of units): left whole, the items
// go to the SMs by decreasing size, and the last SM is done after about
//   E = max over k of (k + 1) p[k SMs],  p the sizes in decreasing order from p[0]
// (k + 1 items as large as p[k SMs] meet on some SM; sorted by counting, so p is
// the lower edge of one of 128 ranges of sizes for k > 0).  Cut, every SM has
// C = W heads / SMs units and the merge and the pieces' starts to pay, about
// `keep` = 14 units; so the items are cut when 65 / 64 E > C + 14.  (D = 128, us
// uncut and cut: C 458, E 544: 829 and 745; C 188, E 200: 359 and 341; C 1.5, E 16:
// 40 and 31; C 54, E 67: 120 and 130; C 10, E 22: 47 and 52; C 318, E 321: 545 and
// 564.  D = 64: C 31, E 50: 77 and 65; C 22, E 26: 48 and 60.)
// Then the items' units are laid end to end and cut at every multiple of
// max(min_units, C), unless the cut would fall within C / 16 of an item's end or
// the item has no more than `whole` units, and the splits are listed by decreasing
// size.
//
// Either way the split items have at most 2 ctas / heads splits in all (an item
// of n > 1 splits has more than (n - 1) target units, or n - 1 cuts), which
// bounds the partial results' memory on the host.  The host's bounds
// choose the blocks' rows (PagedShape); which items are then cut, and where,
// depends on the lengths and the number of heads alone, whichever kernel below
// lists them.  Only the order of the list differs between the kernels and, for
// equally large splits, between runs, and no result depends on it.
//
// The merge joins an item's normalised partials: LSE = ln sum exp(lse_s),
// O = sum exp(lse_s - LSE) O_s.
#include "kernels.h"
#include "paged_plan.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kPmThreads = 256;
constexpr int kBuckets = 128;  // sizes told apart in the list's order (at most NT)
constexpr int kMeet = 3;       // k up to which E is taken (beyond it is close to C)
constexpr float kNegInfP = -__builtin_huge_valf();

// Inclusive scan over the block; warp_sums[NT / 32 - 1] holds the total after it.
template <int NT>
__device__ __forceinline__ long long ps_scan(long long v, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < NT / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += n;
    }
    if (lane < NT / 32) warp_sums[lane] = w;
  }
  __syncthreads();
  return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The last index i of first[0 .. n) with first[i] <= x (first[0] <= x).
__device__ __forceinline__ int last_le(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct PagedItem {
  int tok0, q_len, kv_len, seq, blk, hi;  // keys [0, hi) are visible
};

// Item `i` of the batch: its sequence, its row block and the keys it sees.
__device__ __forceinline__ PagedItem paged_item(const PagedParams& p, const int* first, int i) {
  PagedItem t;
  t.seq = last_le(first, p.num_seqs, i);
  t.tok0 = p.cu_seqlens[t.seq];
  t.q_len = p.cu_seqlens[t.seq + 1] - t.tok0;
  t.kv_len = p.kv_lens[t.seq];
  const int n_blk = first[t.seq + 1] - first[t.seq];
  t.blk = n_blk - 1 - (i - first[t.seq]);  // costly blocks first
  const long long row_hi = static_cast<long long>(t.q_len) * p.group -
                           (n_blk - 1 - t.blk) * static_cast<long long>(p.shape.rows);
  const int last_tok = static_cast<int>((row_hi - 1) / p.group);
  t.hi = p.causal ? max(t.kv_len - t.q_len + last_tok + 1, 0) : t.kv_len;
  return t;
}

// Units of one SM's share of tiles.
__device__ __forceinline__ int paged_tiles_target(const PagedShape& s, long long all, int heads) {
  const long long share = (all * heads + s.ctas - 1) / s.ctas;
  return static_cast<int>(min(max(share, static_cast<long long>(s.min_units)), 1ll << 30));
}

// Whether tiles are cut: the estimate of the uncut time against the share.
__device__ __forceinline__ bool paged_cut(const PagedShape& s, long long all, int heads,
                                          long long uncut) {
  return uncut * 65 * s.ctas > (all * heads + static_cast<long long>(s.keep) * s.ctas) * 64;
}

// Cuts of the item that is units [at, at + units) of all laid end to end.
__device__ __forceinline__ int paged_cuts(const PagedShape& s, long long at, int units,
                                          int target) {
  const int snap = target / 16 + 1;
  if (units <= s.whole) return 0;
  const long long m0 = (at + snap) / target + 1;
  const long long m1 = (at + units - snap - 1) / target;
  return m1 >= m0 ? static_cast<int>(m1 - m0) + 1 : 0;
}

__device__ __forceinline__ int item_units(const PagedParams& p, const PagedItem& t) {
  return (t.hi + p.shape.unit - 1) / p.shape.unit;
}

// Which of kBuckets equal ranges of [0, largest] holds `units` (below 2^24, as
// units of 128 keys are), and where a range begins.
__device__ __forceinline__ int size_bucket(int units, int largest) {
  return min(kBuckets - 1, static_cast<int>(static_cast<unsigned>(units) * kBuckets /
                                            (static_cast<unsigned>(largest) + 1)));
}
__device__ __forceinline__ int bucket_edge(int bucket, int largest) {
  return static_cast<int>(static_cast<unsigned>(bucket) *
                          (static_cast<unsigned>(largest) + 1) / kBuckets);
}

}  // namespace

// Tiles, at most 32 items: every warp works the list out in its lanes, an item
// each, and the warps share the writing.  Same cuts as below.  (Three
// sequences of 90 to 193 tokens 16.6 -> 14.4 us, five of 10 to 16 16.5 -> 12.4 us.)
__global__ void __launch_bounds__(128) paged_schedule_few_kernel(const PagedParams p) {
  __shared__ int s_cost[256];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const bool in = lane < p.num_seqs;
  const int lo = in ? p.cu_seqlens[lane] : 0;
  const int hi = in ? p.cu_seqlens[lane + 1] : 0;
  const int kv = in ? p.kv_lens[lane] : 0;
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  if (__any_sync(0xffffffffu, lo < 0 || hi < lo || hi > p.total_q || hi - lo > p.max_seqlen ||
                                  kv < 0 || kv > p.max_kv_len || kv > cap ||
                                  (lane == 0 && lo != 0))) {
    if (threadIdx.x == 0) {
      p.hdr->error = kPagedBad;
      p.hdr->n_items = 0;
      p.hdr->pad[0] = 0;
    }
    return;
  }
  const int rows = p.shape.rows;
  const int n_blk = static_cast<int>(
      (static_cast<long long>(hi - lo) * p.group + rows - 1) / rows);
  int incl = n_blk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int first = incl - n_blk;
  const int items = __shfl_sync(0xffffffffu, incl, 31);
  // Item `lane`: the last sequence whose first item is at most it (one without
  // items begins where the next begins, and behind the last at `items`).
  int b = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (__shfl_sync(0xffffffffu, first, b + o) <= lane) b += o;
  const bool have = lane < items;
  PagedWork w = {};
  w.seq = b;
  w.tok0 = __shfl_sync(0xffffffffu, lo, b);
  w.q_len = __shfl_sync(0xffffffffu, hi, b) - w.tok0;
  w.kv_len = __shfl_sync(0xffffffffu, kv, b);
  const int blocks = __shfl_sync(0xffffffffu, n_blk, b);
  w.blk = blocks - 1 - (lane - __shfl_sync(0xffffffffu, first, b));  // costly blocks first
  int see = 0;  // keys [0, see) are visible
  if (have) {
    const long long row_hi = static_cast<long long>(w.q_len) * p.group -
                             (blocks - 1 - w.blk) * static_cast<long long>(rows);
    const int last_tok = static_cast<int>((row_hi - 1) / p.group);
    see = p.causal ? max(w.kv_len - w.q_len + last_tok + 1, 0) : w.kv_len;
  }
  const int units = (see + p.shape.unit - 1) / p.shape.unit;
  // Units before this item, and the splits, slots and merges before it.
  auto scan = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  const long long upto = scan(units);
  const long long at = upto - units, all = __shfl_sync(0xffffffffu, upto, 31);
  const int target = paged_tiles_target(p.shape, all, p.num_kv_heads);
  const int snap = target / 16 + 1;
  const int top = __reduce_max_sync(0xffffffffu, units);
  bool cutting = false;
  if (top > p.shape.keep) {
    int rank = 0;  // by decreasing size
#pragma unroll
    for (int o = 0; o < 32; ++o) {
      const int u = __shfl_sync(0xffffffffu, units, o);
      rank += u > units || (u == units && o < lane);
    }
    // This item's bound of the uncut time, if its rank gives one.
    int uncut = have && rank == 0 ? units : 0;
    const int edge = bucket_edge(size_bucket(units, top), top);
#pragma unroll
    for (int k = 1; k <= kMeet; ++k)
      if (have && rank == k * p.shape.ctas / p.num_kv_heads) uncut = max(uncut, (k + 1) * edge);
    uncut = __reduce_max_sync(0xffffffffu, uncut);
    cutting = paged_cut(p.shape, all, p.num_kv_heads, uncut);
  }
  const int n = have ? (cutting ? paged_cuts(p.shape, at, units, target) : 0) + 1 : 0;
  const int cut = n > 1 ? static_cast<int>(((at + snap) / target + 1) * target - at) : units;
  const long long v = n + (n > 1 ? (static_cast<long long>(n) << 32) + (1ll << 48) : 0);
  const long long after = scan(v), before = after - v;
  const long long total = __shfl_sync(0xffffffffu, after, 31);
  const int base = static_cast<int>(before & 0xffffffffll);
  const int slot = n > 1 ? static_cast<int>((before >> 32) & 0xffff) : -1;
  if (threadIdx.x < 32 && n > 1) {
    PagedMerge m = {};
    m.tok0 = w.tok0;
    m.q_len = w.q_len;
    m.blk = w.blk;
    m.slot0 = slot;
    m.n = n;
    p.merge[static_cast<int>(before >> 48)] = m;
  }
  // At most 32 and a cut a SM (152): two a thread.
  const int splits = static_cast<int>(total & 0xffffffffll);
  PagedWork mine[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * 128;
    int x = 0;  // the item of split e (items have at least one; lanes behind have none)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (__shfl_sync(0xffffffffu, base, x + o) <= e) x += o;
    x = max(min(x, items - 1), 0);
    PagedWork& t = mine[i];
    t.tok0 = __shfl_sync(0xffffffffu, w.tok0, x);
    t.q_len = __shfl_sync(0xffffffffu, w.q_len, x);
    t.kv_len = __shfl_sync(0xffffffffu, w.kv_len, x);
    t.seq = __shfl_sync(0xffffffffu, w.seq, x);
    t.blk = __shfl_sync(0xffffffffu, w.blk, x);
    const int s = e - __shfl_sync(0xffffffffu, base, x);
    const int cx = __shfl_sync(0xffffffffu, cut, x);
    t.n = __shfl_sync(0xffffffffu, n, x);
    t.kv_lo = (s == 0 ? 0 : cx + (s - 1) * target) * p.shape.unit;
    const int see_x = __shfl_sync(0xffffffffu, see, x);
    t.kv_hi = s == t.n - 1 ? see_x : (cx + s * target) * p.shape.unit;
    t.slot0 = __shfl_sync(0xffffffffu, slot, x);
    t.slot = t.slot0 < 0 ? -1 : t.slot0 + s;
    t.item = 0;
    t.pad = 0;
    s_cost[e] = t.kv_hi - t.kv_lo;
  }
  __syncthreads();
  // One round of CTAs starts together; else the list goes by decreasing size.
  const bool sorted = splits * p.num_kv_heads > p.shape.ctas;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * 128;
    if (e >= splits) continue;
    int to = e;
    if (sorted) {
      const int cost = s_cost[e];
      to = 0;
      for (int o = 0; o < splits; ++o) to += s_cost[o] > cost || (s_cost[o] == cost && o < e);
    }
    p.work[to] = mine[i];
  }
  if (threadIdx.x == 0) {
    p.hdr->error = 0;
    p.hdr->n_items = splits;
    p.hdr->pad[0] = static_cast<int>(total >> 48);
  }
}

// NT threads: few for small batches, whose barriers are then quicker.
template <int NT>
__global__ void __launch_bounds__(NT) paged_schedule_kernel(const PagedParams p) {
  constexpr int kPsThreads = NT;
  __shared__ long long warp_sums[32];
  __shared__ int s_bad;
  __shared__ int s_first[kPsThreads + 1];  // first item of each sequence (small batches)
  __shared__ int s_base[kPsThreads + 1];   // first split of each item of a round
  __shared__ int s_bucket[kBuckets];       // splits by size
  __shared__ long long s_round;
  __shared__ int s_top;
  __shared__ PagedItem s_item[kPsThreads];
  __shared__ int2 s_split[kPsThreads];     // units of the first split, first slot (-1: whole)
  __shared__ int s_number[kPsThreads];     // number among the split items
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int B = p.num_seqs;
  if (tid == 0) s_bad = s_top = 0;
  for (int i = tid; i < kBuckets; i += kPsThreads) s_bucket[i] = 0;
  __syncthreads();

  // Items of each sequence, and the checks that need device memory.
  const bool small = B <= kPsThreads;
  int* first = small ? s_first : p.first;
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  long long carry = 0;
  for (int base = 0; base < B; base += kPsThreads) {
    const int b = base + tid;
    long long n = 0;
    if (b < B) {
      const int lo = p.cu_seqlens[b], hi = p.cu_seqlens[b + 1], kv = p.kv_lens[b];
      const bool bad = lo < 0 || hi < lo || hi > p.total_q || hi - lo > p.max_seqlen || kv < 0 ||
                       kv > p.max_kv_len || kv > cap || (b == 0 && lo != 0);
      if (bad) s_bad = 1;
      else n = (static_cast<long long>(hi - lo) * p.group + p.shape.rows - 1) / p.shape.rows;
    }
    const long long incl = ps_scan<NT>(n, warp_sums);
    if (b < B) first[b] = static_cast<int>(carry + incl - n);
    carry += warp_sums[NT / 32 - 1];
    __syncthreads();
  }
  if (tid == 0) first[B] = static_cast<int>(carry);
  const int items = static_cast<int>(carry);
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      p.hdr->error = kPagedBad;
      p.hdr->n_items = 0;
      p.hdr->pad[0] = 0;
    }
    return;
  }

  // All units, and the largest split that shares them out.
  const bool tiles = p.shape.tiles;
  long long sum = 0;
  int most = 0;
  PagedItem it = {};
  for (int i = tid; i < items; i += kPsThreads) {
    it = paged_item(p, first, i);
    const int units = item_units(p, it);
    sum += units;
    most = max(most, units);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(&s_top, most);
  ps_scan<NT>(sum, warp_sums);
  const long long all = warp_sums[NT / 32 - 1];
  const int target = tiles ? paged_tiles_target(p.shape, all, p.num_kv_heads)
                           : paged_rows_target(p.shape, all, items, p.num_kv_heads);
  const int snap = target / 16 + 1;
  const int top = s_top;
  bool cutting = false;
  if (tiles && top > p.shape.keep) {
    // The items by size, and from that the estimate of the uncut time.
    for (int i = tid; i < items; i += kPsThreads) {
      if (items > kPsThreads) it = paged_item(p, first, i);
      atomicAdd(&s_bucket[kBuckets - 1 - size_bucket(item_units(p, it), top)], 1);
    }
    __syncthreads();
    // Thread b: items in the buckets up to its own, the larger sizes first.
    const int mine = tid < kBuckets ? s_bucket[tid] : 0;
    const int upto = static_cast<int>(ps_scan<NT>(mine, warp_sums));
    for (int k = 1; k <= kMeet; ++k) {
      const int rank = k * p.shape.ctas / p.num_kv_heads;
      if (upto - mine <= rank && rank < upto)
        atomicMax(&s_top, (k + 1) * bucket_edge(kBuckets - 1 - tid, top));
    }
    __syncthreads();
    cutting = paged_cut(p.shape, all, p.num_kv_heads, s_top);
  }
  // No split has more units.
  const int largest = cutting ? max(target + 2 * snap, p.shape.whole) : top;
  for (int i = tid; i < kBuckets; i += kPsThreads) s_bucket[i] = 0;
  __syncthreads();

  // Pass 0 (tiles) counts the splits of each size, pass 1 writes the list.
  const bool once = items <= kPsThreads;
  int work0 = 0, slot0 = 0, merge0 = 0;
  for (int pass = tiles ? 0 : 1; pass < 2; ++pass) {
    work0 = slot0 = merge0 = 0;
    long long unit0 = 0;
    for (int base = 0; base < items; base += kPsThreads) {
      const int in_round = min(items - base, kPsThreads);
      long long round;
      if (pass == 0 || !tiles || !once) {
        const int i = base + tid;
        int n = 0, cut = 0, units = 0;
        if (i < items) {
          if (!once) it = paged_item(p, first, i);
          units = item_units(p, it);
        }
        if (tiles) {
          // The item is [at, at + units) of the units laid end to end.
          const long long at = unit0 + ps_scan<NT>(units, warp_sums) - units;
          unit0 += warp_sums[NT / 32 - 1];
          __syncthreads();
          if (i < items) {
            n = (cutting ? paged_cuts(p.shape, at, units, target) : 0) + 1;
            cut = n > 1 ? static_cast<int>(((at + snap) / target + 1) * target - at) : units;
          }
        } else if (i < items) {
          n = units > target ? (units + target - 1) / target : 1;
          cut = (units + n - 1) / n;
          if (n > 1) n = (units + cut - 1) / cut;
        }
        const bool split = n > 1;
        // Splits, slots and merges counted in one scan (slots and merges < 2^16).
        const long long v = n + (split ? (static_cast<long long>(n) << 32) + (1ll << 48) : 0);
        const long long before = ps_scan<NT>(v, warp_sums) - v;
        round = warp_sums[NT / 32 - 1];
        const int slot = slot0 + static_cast<int>((before >> 32) & 0xffff);
        const int item = merge0 + static_cast<int>(before >> 48);
        s_base[tid] = static_cast<int>(before & 0xffffffffll);
        s_item[tid] = it;
        s_split[tid] = make_int2(cut, split ? slot : -1);
        s_number[tid] = item;
        if (pass == 1 && split && !p.shape.join) {
          PagedMerge m = {};
          m.tok0 = it.tok0;
          m.q_len = it.q_len;
          m.blk = it.blk;
          m.slot0 = slot;
          m.n = n;
          p.merge[item] = m;
        }
        if (tid == 0) s_base[kPsThreads] = static_cast<int>(round & 0xffffffffll);
        __syncthreads();
        if (tid == 0) s_round = round;
      } else {
        // One round: still there from pass 0, but for the merges.
        round = s_round;
        if (tid < in_round && s_split[tid].y >= 0 && !p.shape.join) {
          PagedMerge m = {};
          m.tok0 = it.tok0;
          m.q_len = it.q_len;
          m.blk = it.blk;
          m.slot0 = s_split[tid].y;
          m.n = (tid + 1 < in_round ? s_base[tid + 1] : s_base[kPsThreads]) - s_base[tid];
          p.merge[s_number[tid]] = m;
        }
      }
      const int splits = static_cast<int>(round & 0xffffffffll);
      for (int e = tid; e < splits; e += kPsThreads) {
        const int x = last_le(s_base, in_round, e);
        const PagedItem t = s_item[x];
        const int2 sp = s_split[x];
        const int n = (x + 1 < in_round ? s_base[x + 1] : splits) - s_base[x];
        const int s = e - s_base[x];
        const int step = tiles ? target : sp.x;
        const int units = item_units(p, t);
        const int u0 = s == 0 ? 0 : sp.x + (s - 1) * step;
        const int u1 = s == n - 1 ? units : sp.x + s * step;
        const int bucket = size_bucket(u1 - u0, largest);
        if (pass == 0) {
          atomicAdd(&s_bucket[kBuckets - 1 - bucket], 1);
          continue;
        }
        PagedWork w;
        w.tok0 = t.tok0;
        w.q_len = t.q_len;
        w.kv_len = t.kv_len;
        w.seq = t.seq;
        w.blk = t.blk;
        w.kv_lo = u0 * p.shape.unit;
        w.kv_hi = s == n - 1 ? t.hi : u1 * p.shape.unit;
        w.slot = sp.y < 0 ? -1 : sp.y + s;
        w.slot0 = sp.y;
        w.n = n;
        w.item = s_number[x];
        w.pad = 0;
        p.work[tiles ? atomicAdd(&s_bucket[kBuckets - 1 - bucket], 1) : work0 + e] = w;
      }
      work0 += splits;
      slot0 += static_cast<int>((round >> 32) & 0xffff);
      merge0 += static_cast<int>(round >> 48);
      __syncthreads();
    }
    if (pass == 0) {  // sizes in decreasing order: where each begins in the list
      const int v = tid < kBuckets ? s_bucket[tid] : 0;
      const int at = static_cast<int>(ps_scan<NT>(v, warp_sums)) - v;
      if (tid < kBuckets) s_bucket[tid] = at;
      __syncthreads();
    }
  }
  if (p.shape.join)
    for (int i = tid; i < merge0 * p.num_kv_heads; i += kPsThreads) p.arrived[i] = 0;
  if (tid == 0) {
    p.hdr->error = 0;
    p.hdr->n_items = work0;
    p.hdr->pad[0] = merge0;
  }
}

cudaError_t launch_paged_schedule(const PagedParams& p, cudaStream_t stream) {
  // At most so many items: by the rows in all, and by the blocks of each sequence.
  const long long rows = static_cast<long long>(p.max_seqlen) * p.group;
  const long long items = min(p.total_q * p.group / p.shape.rows + p.num_seqs,
                              p.num_seqs * ((rows + p.shape.rows - 1) / p.shape.rows));
  if (p.shape.tiles && items <= 32 && p.num_seqs <= 32)
    paged_schedule_few_kernel<<<1, 128, 0, stream>>>(p);
  else if (items <= 128) paged_schedule_kernel<128><<<1, 128, 0, stream>>>(p);
  else if (items <= 512) paged_schedule_kernel<512><<<1, 512, 0, stream>>>(p);
  else paged_schedule_kernel<1024><<<1, 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

// A warp joins R rows of one item and KV head at a time, S splits of each in
// flight; lane l holds the weight of row l % R and split l / R of a round of
// 32 / R splits.
template <int D, int R, int S, bool PLAN>
__global__ void __launch_bounds__(kPmThreads) paged_merge_kernel(const PagedParams p) {
  constexpr int kPer = D / 32;  // floats of a row each lane owns
  constexpr int kRound = 32 / R;
  const int lane = threadIdx.x & 31;
  PagedPlan plan;
  if (PLAN) plan = make_plan(p, lane);  // reads the lengths alone: beside the attention
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (PLAN && blockIdx.x == 0) {
    // The error word of the whole call.
    int error = 0;
    for (int i = threadIdx.x; i < plan.splits * p.num_kv_heads; i += kPmThreads)
      error |= __ldcg(p.cta_error + i);
    const bool bad = __syncthreads_or(plan.bad || (error & kPagedBad));
    const bool late = __syncthreads_or(error & kPagedLate);
    if (threadIdx.x == 0) {
      p.hdr->error = bad ? kPagedBad : (late ? kPagedLate : 0);
      p.hdr->n_items = plan.splits;
      p.hdr->pad[0] = plan.merges;
    }
  }
  const int lr = lane % R, ls = lane / R;
  const int rows = p.shape.rows, Hk = p.num_kv_heads;
  const int groups = (rows + R - 1) / R;
  const int merges = PLAN ? plan.merges : __ldcg(&p.hdr->pad[0]);
  const long long total = static_cast<long long>(merges) * Hk * groups;
  const long long step = static_cast<long long>(gridDim.x) * (kPmThreads / 32);
  const long long pitch = static_cast<long long>(Hk) * rows;  // rows from split to split
  for (long long x = static_cast<long long>(blockIdx.x) * (kPmThreads / 32) + (threadIdx.x >> 5);
       x < total; x += step) {
    const int r0 = static_cast<int>(x % groups) * R;
    const long long mh = x / groups;
    const int h = static_cast<int>(mh % Hk);
    PagedMerge item;
    if (PLAN) {
      item = plan_merge(plan, static_cast<int>(mh / Hk));
    } else {
      const int4* mp = reinterpret_cast<const int4*>(p.merge + mh / Hk);
      const int4 m0 = __ldcg(mp);
      item.n = __ldcg(mp + 1).x;
      item.tok0 = m0.x;
      item.q_len = m0.y;
      item.blk = m0.z;
      item.slot0 = m0.w;
    }
    const int n = item.n, tok0 = item.tok0, q_len = item.q_len, blk = item.blk;
    const int slot0 = item.slot0;
    const long long all_rows = static_cast<long long>(q_len) * p.group;
    const long long n_blk = (all_rows + rows - 1) / rows;
    const long long row0 = all_rows - (n_blk - blk) * rows + r0;
    const long long part = (static_cast<long long>(slot0) * Hk + h) * rows + r0;
    const bool mine = r0 + lr < rows && row0 + lr >= 0;
    float top = kNegInfP;
    bool nan = false;  // a maximum passes over NaN; the row has to show it
    for (int s = ls; s < n; s += kRound) {
      const float v = mine ? __ldcg(p.lse_part + part + lr + s * pitch) : kNegInfP;
      top = fmaxf(top, v);
      nan = nan || v != v;
    }
#pragma unroll
    for (int o = R; o < 32; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      nan = __shfl_xor_sync(0xffffffffu, nan, o) || nan;
    }
    if (nan) top = __int_as_float(0x7fffffff);
    float den = 0.f, acc[R][kPer];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[r][e] = 0.f;
    for (int s0 = 0; s0 < n; s0 += kRound) {
      float w = 0.f;
      if (mine && s0 + ls < n && top != kNegInfP)
        w = expf(__ldcg(p.lse_part + part + lr + (s0 + ls) * pitch) - top);
      den += w;
      const int m = min(kRound, n - s0);
      for (int s = 0; s < m; s += S) {
        float v[S][R][kPer];
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool in = s + u < m && r0 + r < rows && row0 + r >= 0;
            const float* src = p.o_part + (part + r + (s0 + s + u) * pitch) * D + lane * kPer;
            if (kPer == 4) {
              const float4 f = in ? __ldcg(reinterpret_cast<const float4*>(src))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
              v[u][r][0] = f.x;
              v[u][r][1] = f.y;
              v[u][r][2 % kPer] = f.z;
              v[u][r][3 % kPer] = f.w;
            } else {
              const float2 f =
                  in ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
              v[u][r][0] = f.x;
              v[u][r][1] = f.y;
            }
          }
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            // Splits beyond the last have weight 0 and were not loaded.
            const float wr = __shfl_sync(0xffffffffu, w, ((s + u) % kRound) * R + r);
            if (s + u < m) {
#pragma unroll
              for (int e = 0; e < kPer; ++e) acc[r][e] = fmaf(wr, v[u][r][e], acc[r][e]);
            }
          }
      }
    }
#pragma unroll
    for (int o = R; o < 32; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const float lse = den == 0.f ? kNegInfP : top + logf(den);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ir = __shfl_sync(0xffffffffu, inv, r);
      const float lse_r = __shfl_sync(0xffffffffu, lse, r);
      const long long row = row0 + r;
      if (r0 + r >= rows || row < 0) continue;
      const int tok = static_cast<int>(row / p.group);
      const size_t at = static_cast<size_t>(tok0 + tok) * p.num_heads + h * p.group +
                        static_cast<int>(row - static_cast<long long>(tok) * p.group);
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * kPer);
      if (kPer == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(acc[r][0] * ir, acc[r][1] * ir),
                       pack_bf16x2(acc[r][2 % kPer] * ir, acc[r][3 % kPer] * ir));
      else
        *dst = pack_bf16x2(acc[r][0] * ir, acc[r][1] * ir);
      if (lane == 0 && p.lse != nullptr) p.lse[at] = lse_r;
    }
  }
}

template <int D>
static cudaError_t launch_paged_merge_d(const PagedParams& p, const cudaLaunchConfig_t& cfg) {
  // Tiles: many rows of few splits.  Else: few rows of many splits.
  if (p.shape.tiles) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, 8, 1, false>, p);
  return p.shape.plan ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, 2, 8, true>, p)
                      : cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, 2, 4, false>, p);
}

cudaError_t launch_paged_merge(const PagedParams& p, int D, int num_sms, cudaStream_t stream) {
  // No more merges than items, nor than half the slots.
  const long long blocks =
      (static_cast<long long>(p.max_seqlen) * p.group + p.shape.rows - 1) / p.shape.rows;
  const long long items = min(min(p.total_q * p.group / p.shape.rows + p.num_seqs,
                                  p.num_seqs * blocks), p.max_slots / 2);
  const int at_once = p.shape.tiles ? 8 : 2;  // rows of a warp
  const long long warps = items * p.num_kv_heads * ((p.shape.rows + at_once - 1) / at_once);
  long long grid = (warps + kPmThreads / 32 - 1) / (kPmThreads / 32);
  grid = grid < 1 ? 1 : min(grid, num_sms * 4LL);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPmThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return D == 64 ? launch_paged_merge_d<64>(p, cfg) : launch_paged_merge_d<128>(p, cfg);
}

}  // namespace cpattn
