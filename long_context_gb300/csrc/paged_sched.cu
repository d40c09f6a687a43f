// Attention over a paged KV cache: the work list, and the merge of splits.
//
// The schedule kernel reads the lengths on the device (a captured graph can be
// replayed with other lengths) and cuts the work: with W units of keys over
// all items of a KV head, an item of u units becomes ceil(u / target) splits,
//   target = max(min_units, ceil(W * KV heads / ctas)),
// so every CTA has at most 1 / ctas of the work and a long cache with few new
// tokens still fills the GPU.  Since an item of more than one split has more
// than target units, split items have at most 2 W / target <= 2 ctas / heads
// splits in all, which bounds the partial results' memory on the host.
//
// The merge joins an item's normalised partials: LSE = ln sum exp(lse_s),
// O = sum exp(lse_s - LSE) O_s.
#include "kernels.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kPmThreads = 256;
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
  const long long row_hi =
      static_cast<long long>(t.q_len) * p.group - (n_blk - 1 - t.blk) * static_cast<long long>(p.shape.rows);
  const int last_tok = static_cast<int>((row_hi - 1) / p.group);
  t.hi = p.causal ? max(t.kv_len - t.q_len + last_tok + 1, 0) : t.kv_len;
  return t;
}

__device__ __forceinline__ int item_units(const PagedParams& p, const PagedItem& t) {
  return (t.hi + p.shape.unit - 1) / p.shape.unit;
}

}  // namespace

// NT threads; batches of up to 128 items take 128, whose barriers are quicker.
template <int NT>
__global__ void __launch_bounds__(NT) paged_schedule_kernel(const PagedParams p) {
  constexpr int kPsThreads = NT;
  __shared__ long long warp_sums[32];
  __shared__ int s_bad;
  __shared__ int s_first[kPsThreads + 1];  // first item of each sequence (small batches)
  __shared__ int s_base[kPsThreads];       // first split of each item of a round
  __shared__ PagedItem s_item[kPsThreads];
  __shared__ int2 s_split[kPsThreads];     // units of a split, first slot (-1: whole)
  __shared__ int s_number[kPsThreads];     // number among the split items
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int B = p.num_seqs;
  if (tid == 0) s_bad = 0;
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
      p.hdr->error = 1;  // CPATTN_ERR_INVALID_ARG
      p.hdr->n_items = 0;
      p.hdr->pad[0] = 0;
    }
    return;
  }

  // All units, and the largest split that shares them out.
  long long sum = 0;
  PagedItem it = {};
  for (int i = tid; i < items; i += kPsThreads) {
    it = paged_item(p, first, i);
    sum += item_units(p, it);
  }
  ps_scan<NT>(sum, warp_sums);
  const long long all = warp_sums[NT / 32 - 1];
  // With few items the splits are made to fit one round of resident CTAs
  // (sum of ceil(u / target) <= all / target + items), else to be several
  // rounds that even out.
  const long long lanes = static_cast<long long>(items) * p.num_kv_heads;
  const long long share = 2 * lanes <= p.shape.round ? p.shape.round - lanes : p.shape.ctas;
  long long target = (all * p.num_kv_heads + share - 1) / share;
  if (target < p.shape.min_units) target = p.shape.min_units;
  __syncthreads();

  int work0 = 0, slot0 = 0, merge0 = 0;
  for (int base = 0; base < items; base += kPsThreads) {
    const int i = base + tid;
    int n = 0, per = 0;
    if (i < items) {
      if (items > kPsThreads) it = paged_item(p, first, i);
      const int units = item_units(p, it);
      n = units > target ? static_cast<int>((units + target - 1) / target) : 1;
      per = (units + n - 1) / n;
      if (n > 1) n = (units + per - 1) / per;
    }
    const bool split = n > 1;
    // Splits, slots and merges counted in one scan (slots and merges < 2^16).
    const long long v = n + (split ? (static_cast<long long>(n) << 32) + (1ll << 48) : 0);
    const long long before = ps_scan<NT>(v, warp_sums) - v;
    const long long round = warp_sums[NT / 32 - 1];
    const int slot = slot0 + static_cast<int>((before >> 32) & 0xffff);
    s_base[tid] = static_cast<int>(before & 0xffffffffll);
    s_item[tid] = it;
    const int item = merge0 + static_cast<int>(before >> 48);
    s_split[tid] = make_int2(per, split ? slot : -1);
    s_number[tid] = item;
    if (split && !p.shape.join) {
      PagedMerge m = {};
      m.tok0 = it.tok0;
      m.q_len = it.q_len;
      m.blk = it.blk;
      m.slot0 = slot;
      m.n = n;
      p.merge[item] = m;
    }
    __syncthreads();
    const int in_round = min(items - base, kPsThreads);
    const int splits = static_cast<int>(round & 0xffffffffll);
    for (int e = tid; e < splits; e += kPsThreads) {
      const int x = last_le(s_base, in_round, e);
      const PagedItem t = s_item[x];
      const int2 sp = s_split[x];
      const int s = e - s_base[x];
      PagedWork w;
      w.tok0 = t.tok0;
      w.q_len = t.q_len;
      w.kv_len = t.kv_len;
      w.seq = t.seq;
      w.blk = t.blk;
      w.kv_lo = s * sp.x * p.shape.unit;
      w.kv_hi = min(t.hi, (s + 1) * sp.x * p.shape.unit);
      w.slot = sp.y < 0 ? -1 : sp.y + s;
      w.slot0 = sp.y;
      w.n = sp.y < 0 ? 1 : (item_units(p, t) + sp.x - 1) / sp.x;
      w.item = s_number[x];
      w.pad = 0;
      p.work[work0 + e] = w;
    }
    work0 += splits;
    slot0 += static_cast<int>((round >> 32) & 0xffff);
    merge0 += static_cast<int>(round >> 48);
    __syncthreads();
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
  if (p.total_q * p.group / p.shape.rows + p.num_seqs <= 128)
    paged_schedule_kernel<128><<<1, 128, 0, stream>>>(p);
  else
    paged_schedule_kernel<1024><<<1, 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

// A warp joins R rows of one item and KV head at a time, S splits of each in
// flight; lane l holds the weight of row l % R and split l / R of a round of
// 32 / R splits.
template <int D, int R, int S>
__global__ void __launch_bounds__(kPmThreads) paged_merge_kernel(const PagedParams p) {
  constexpr int kPer = D / 32;  // floats of a row each lane owns
  constexpr int kRound = 32 / R;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int lr = lane % R, ls = lane / R;
  const int rows = p.shape.rows, Hk = p.num_kv_heads;
  const int groups = (rows + R - 1) / R;
  const long long total = static_cast<long long>(__ldcg(&p.hdr->pad[0])) * Hk * groups;
  const long long step = static_cast<long long>(gridDim.x) * (kPmThreads / 32);
  const long long pitch = static_cast<long long>(Hk) * rows;  // rows from split to split
  for (long long x = static_cast<long long>(blockIdx.x) * (kPmThreads / 32) + (threadIdx.x >> 5);
       x < total; x += step) {
    const int r0 = static_cast<int>(x % groups) * R;
    const long long mh = x / groups;
    const int h = static_cast<int>(mh % Hk);
    const int4* mp = reinterpret_cast<const int4*>(p.merge + mh / Hk);
    const int4 m0 = __ldcg(mp);
    const int n = __ldcg(mp + 1).x;
    const int tok0 = m0.x, q_len = m0.y, blk = m0.z, slot0 = m0.w;
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

cudaError_t launch_paged_merge(const PagedParams& p, int D, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms * 4));
  cfg.blockDim = dim3(kPmThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Tiles: many rows of few splits.  32 rows: many splits.
  if (p.shape.tiles)
    return D == 64 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<64, 8, 1>, p)
                   : cudaLaunchKernelEx(&cfg, paged_merge_kernel<128, 8, 1>, p);
  return D == 64 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<64, 2, 4>, p)
                 : cudaLaunchKernelEx(&cfg, paged_merge_kernel<128, 2, 4>, p);
}

}  // namespace cpattn
