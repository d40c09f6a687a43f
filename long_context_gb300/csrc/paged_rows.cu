// Attention of few rows over a paged KV cache: one token a sequence, or a few,
// for every query head that shares a KV head.
//
// A CTA (4 warps) has one block of up to 16 or 32 rows of one KV head and one
// split of the keys.  Its work is HBM bound: a key and its value (4 D bytes)
// are read once and meet at most 32 rows.  Each warp takes every fourth group
// of 16 keys on its own: it copies the group's K and V rows into its ring of
// stages with cp.async (a group never straddles a page, so it needs one page
// number, read a group ahead), multiplies with 16 x 8 x 16 matrix
// instructions (the 16 rows of Q in registers are the left operand) and keeps
// its own softmax state, so the warps never wait for one another until they
// join their states at the end.  tcgen05 has nothing to give here: its tiles
// have 64 or 128 rows, of which 16 would be used, and the matrix instructions
// that 16 rows need take a small part of the time that the bytes take.
//
// Softmax: p = 2^(s scale log2 e - m), one pass with a running maximum m that
// moves only when a group's maximum exceeds it by 8 powers of two (O and l
// share the reference, so O / l and m + ln l do not depend on it); l sums p in
// fp32, O accumulates in fp32.  The matrix instructions take P in bf16.  Blocks of
// up to 16 rows (the decoding step) keep what that rounding leaves: the remainder
// p - bf16(p) is a second bf16 operand, so P is off by 2^-16 and O has its own
// rounding's error alone (relative to 64 bits 0.0017 instead of 0.0020).  Up to 8
// rows leave the other half of the 16-row operand free, which takes the remainder
// without another instruction (a token each of 64 caches, 32 / 8 heads of 128: 655
// instead of 645 us; 65 caches of 327 to 655 keys, 4 KV heads: 22.6, before 22.9);
// 9 to 16 rows cost a second product (the same rows in such a block: 658 and 23.7
// us).  Blocks of 32 rows round P to bf16 as the tile kernel and the packed forward
// do: their products take most of the time, and a second one costs an eighth of it
// (drafts 33.2 and 37.4 us; 4 tokens of 8 heads each over 17 caches 82 and 92 us).
#include <cuda_bf16.h>

#include "kernels.h"
#include "paged_plan.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kPrThreads = 128;
constexpr int kPrWarps = kPrThreads / 32;
constexpr int kGroupKeys = 16;
constexpr float kNegInfR = -__builtin_huge_valf();
constexpr float kLn2R = 0.69314718055994530942f;
constexpr float kLog2eR = 1.44269504088896340736f;
constexpr float kMoveBy = 8.0f;  // powers of two

template <int D>
struct RowsCfg {
  static constexpr int kHalf = kGroupKeys * D * 2;  // K (or V) of one group
  static constexpr int kGroups = D == 128 ? 1 : 2;  // groups of a step
  static constexpr int kStage = kGroups * 2 * kHalf;
  static constexpr int kStages = 3;
  static constexpr int kSmem = kPrWarps * kStages * kStage;  // 96 KB: two CTAs a SM
};

// Byte offset of 16-byte chunk c of row r; the low chunk bits are exchanged
// with the row's so that ldmatrix reads eight rows without a bank conflict.
template <int D>
__device__ __forceinline__ int at(int r, int c) {
  return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

}  // namespace

template <int D, int MT, bool HALF, bool PLAN>
__global__ void __launch_bounds__(kPrThreads, 2) paged_rows_kernel(const PagedParams p) {
  using C = RowsCfg<D>;
  // HALF: at most 8 rows, which lie in the second half of the block (its rows end
  // with the sequence's); the first half of P holds the remainders.
  static_assert(!HALF || MT == 1);
  constexpr int kRows = 16 * MT;
  constexpr int kH0 = HALF ? 1 : 0;
  constexpr bool kSecond = MT == 1 && !HALF;  // the remainders are an operand of their own
  constexpr int kCh = D / 8;         // 16-byte chunks of a row
  constexpr int kRpi = 32 / kCh;     // rows one warp copy covers
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kPrWarps][kRows], s_l[kPrWarps][kRows];
  __shared__ int s_last;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int Hk = p.num_kv_heads, G = p.group;
  const int e = static_cast<int>(blockIdx.x) / Hk;
  const int h = static_cast<int>(blockIdx.x) - e * Hk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PagedWork w;
  if (PLAN) {
    const PagedPlan plan = make_plan(p, lane);
    if (e >= plan.splits) return;
    w = plan_split(p, plan, e);
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // In flight together: the list has room for every CTA of the grid.
    const int n_work = __ldcg(&p.hdr->n_items);
    const int4* wp = reinterpret_cast<const int4*>(p.work + e);
    const int4 w0 = __ldcg(wp), w1 = __ldcg(wp + 1), w2 = __ldcg(wp + 2);
    if (e >= n_work) return;
    w.tok0 = w0.x;
    w.q_len = w0.y;
    w.kv_len = w0.z;
    w.seq = w0.w;
    w.blk = w1.x;
    w.kv_lo = w1.y;
    w.kv_hi = w1.z;
    w.slot = w1.w;
    w.slot0 = w2.x;
    w.n = w2.y;
    w.item = w2.z;
  }
  const int tok0 = w.tok0, q_len = w.q_len, kv_len = w.kv_len, seq = w.seq;
  const int blk = w.blk, kv_lo = w.kv_lo, kv_hi = w.kv_hi, slot = w.slot;
  // Rows of this block: [row0, row0 + kRows), those below 0 are not there.
  const int all_rows = q_len * G;
  const int n_blk = (all_rows + kRows - 1) / kRows;
  const int row0 = all_rows - (n_blk - blk) * kRows;

  bool bad_page = false;
  const int* pages = p.page_table + static_cast<size_t>(seq) * p.max_pages;
  const int page_mask = (1 << p.page_shift) - 1;
  const size_t row_pitch = static_cast<size_t>(Hk) * D;
  const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);

  // Groups of this warp: kv_lo / 16 + warp, + 4, ...; kGroups of them a step.
  constexpr int NG = C::kGroups;
  const int n_groups = (kv_hi - kv_lo + kGroupKeys - 1) / kGroupKeys;
  const int n = n_groups > warp ? (n_groups - warp + kPrWarps - 1) / kPrWarps : 0;
  const int steps = (n + NG - 1) / NG;
  auto group_key = [&](int j) { return kv_lo + (warp + j * kPrWarps) * kGroupKeys; };
  int next_page[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    next_page[g] = g < n ? __ldg(pages + (group_key(g) >> p.page_shift)) : 0;
  auto copy = [&](int step) {
    if (step < steps) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int j = step * NG + g;
        const int key0 = group_key(j);
        int page = next_page[g];
        if (j + NG < n) next_page[g] = __ldg(pages + (group_key(j + NG) >> p.page_shift));
        int last = j < n ? kv_len : 0;  // keys at or beyond it are filled with zeros
        if (page < 0 || page >= p.num_pages) {
          bad_page = bad_page || j < n;
          page = 0;
          last = 0;
        }
        const int r0 = lane / kCh, c = lane % kCh;
        const size_t off = static_cast<size_t>(page) * p.page_stride +
                           static_cast<size_t>((key0 & page_mask) + r0) * row_pitch +
                           static_cast<size_t>(h) * D + c * 8;
        const __nv_bfloat16* ks = p.k_cache + off;
        const __nv_bfloat16* vs = p.v_cache + off;
        const uint32_t dst = ring + (step % C::kStages) * C::kStage + g * 2 * C::kHalf;
#pragma unroll
        for (int it = 0; it < kGroupKeys / kRpi; ++it) {
          const int r = r0 + it * kRpi;
          const bool in = key0 + r < last;
          const size_t skip = in ? it * kRpi * row_pitch : 0;
          const __nv_bfloat16* kr = in ? ks + skip : p.k_cache;
          const __nv_bfloat16* vr = in ? vs + skip : p.v_cache;
          cp_async16(dst + at<D>(r, c), kr, in ? 16 : 0);
          cp_async16(dst + C::kHalf + at<D>(r, c), vr, in ? 16 : 0);
        }
      }
    }
    cp_async_commit();
  };
  // Q (in flight with the first page numbers) as left operands: lane l holds rows l / 4 and l / 4 + 8, columns
  // 2 (l % 4) + {0, 1} and + 8 of each 16 x 16 block.
  uint32_t qa[MT][D / 16][4];
  int lim[MT][2];  // keys below it are visible
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int row = row0 + mt * 16 + hf * 8 + (lane >> 2);
      const bool in = row >= 0;
      const int tok = in ? row / G : 0;
      lim[mt][hf] = in ? (p.causal ? kv_len - q_len + tok + 1 : kv_len) : 0;
      const __nv_bfloat16* src =
          p.q + (static_cast<size_t>(tok0 + tok) * p.num_heads + h * G + (in ? row - tok * G : 0)) * D +
          2 * (lane & 3);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qa[mt][kk][hf] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16)) : 0u;
        qa[mt][kk][hf + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8)) : 0u;
      }
    }
#pragma unroll
  for (int j = 0; j < C::kStages - 1; ++j) copy(j);

  // Groups ending at or below this key need no mask (rows are in order, so
  // the block's first row sees the fewest keys).
  const int first_tok = max(row0, 0) / G;
  const int free_end = row0 < 0 ? 0 : (p.causal ? kv_len - q_len + first_tok + 1 : kv_len);

  float o[MT][D / 8][4];
  float m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt][0] = m[mt][1] = kNegInfR;
    l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
    for (int f = 0; f < D / 8; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[mt][f][i] = 0.f;
  }

#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    copy(step + C::kStages - 1);
    const uint32_t kb = ring + (step % C::kStages) * C::kStage;
    const uint32_t vb = kb + C::kHalf;
    float s[NG][MT][2][4];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[g][mt][i >> 2][i & 3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t b[4];
        ldmatrix4(kb + g * 2 * C::kHalf +
                      at<D>((lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)),
                  b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_16816(s[g][mt][0], qa[mt][kk], b[0], b[1]);
          mma_16816(s[g][mt][1], qa[mt][kk], b[2], b[3]);
        }
      }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // A step's groups beyond the last hold zeros and lie beyond every limit
      // (or beyond kv_hi, which a following split starts with: masked too).
      const int j = step * NG + g;
      const int key0 = group_key(j);
      if (key0 + kGroupKeys > free_end || j >= n) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (HALF && !(i & 2)) continue;
            const int key = key0 + (i >> 2) * 8 + 2 * (lane & 3) + (i & 1);
            if (key >= lim[mt][(i >> 1) & 1] || j >= n) s[g][mt][i >> 2][i & 3] = kNegInfR;
          }
      }
    }
    bool move = false;
    float top[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = kH0; hf < 2; ++hf) {
        float t = kNegInfR;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          t = fmaxf(t, fmaxf(fmaxf(s[g][mt][0][2 * hf], s[g][mt][0][2 * hf + 1]),
                             fmaxf(s[g][mt][1][2 * hf], s[g][mt][1][2 * hf + 1])));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        top[mt][hf] = t * p.scale_log2;
        move = move || top[mt][hf] > m[mt][hf] + kMoveBy;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = kH0; hf < 2; ++hf) {
          const float mn = fmaxf(m[mt][hf], top[mt][hf]);
          const float alpha = m[mt][hf] == kNegInfR ? 0.f : ex2_approx(m[mt][hf] - mn);
          m[mt][hf] = mn;
          l[mt][hf] *= alpha;
#pragma unroll
          for (int f = 0; f < D / 8; ++f) {
            o[mt][f][2 * hf] *= alpha;
            o[mt][f][2 * hf + 1] *= alpha;
            if (HALF) {
              o[mt][f][0] *= alpha;
              o[mt][f][1] *= alpha;
            }
          }
        }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t pa[MT][4], pb[4];  // P and, of up to 16 rows, what its rounding left
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = kH0; hf < 2; ++hf) {
          const float ref = m[mt][hf] == kNegInfR ? 0.f : m[mt][hf];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float p0 = ex2_approx(fmaf(s[g][mt][t][2 * hf], p.scale_log2, -ref));
            const float p1 = ex2_approx(fmaf(s[g][mt][t][2 * hf + 1], p.scale_log2, -ref));
            l[mt][hf] += p0 + p1;
            const uint32_t up = pack_bf16x2(p0, p1);
            pa[mt][2 * t + hf] = up;
            if (MT == 1)
              (HALF ? pa[mt][2 * t] : pb[2 * t + hf]) = pack_bf16x2(
                  p0 - __uint_as_float(up << 16), p1 - __uint_as_float(up & 0xffff0000u));
          }
        }
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        uint32_t b[4];
        ldmatrix4_trans(vb + g * 2 * C::kHalf +
                            at<D>((lane & 7) + (((lane >> 3) & 1) << 3), f * 2 + (lane >> 4)),
                        b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_16816(o[mt][2 * f], pa[mt], b[0], b[1]);
          mma_16816(o[mt][2 * f + 1], pa[mt], b[2], b[3]);
          if (kSecond) {
            mma_16816(o[mt][2 * f], pb, b[0], b[1]);
            mma_16816(o[mt][2 * f + 1], pb, b[2], b[3]);
          }
        }
      }
    }
  }

  // Join the warps' states (their rings are done with) and write the rows.
  cp_async_wait<0>();
  const bool any_bad = __syncthreads_or(bad_page);
  if (threadIdx.x == 0) {
    if (PLAN) p.cta_error[blockIdx.x] = any_bad ? kPagedBad : 0;
    else if (any_bad) atomicCAS(&p.hdr->error, 0, kPagedBad);
  }
  float* so = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = kH0; hf < 2; ++hf) {
      const int r = mt * 16 + hf * 8 + (lane >> 2);
      float sum = l[mt][hf];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if ((lane & 3) == 0) {
        s_m[warp][r] = m[mt][hf];
        s_l[warp][r] = sum;
      }
#pragma unroll
      for (int f = 0; f < D / 8; ++f)
        *reinterpret_cast<float2*>(so + r * D + f * 8 + 2 * (lane & 3)) =
            HALF ? make_float2(o[mt][f][2] + o[mt][f][0], o[mt][f][3] + o[mt][f][1])
                 : make_float2(o[mt][f][2 * hf], o[mt][f][2 * hf + 1]);
    }
  __syncthreads();
  // Joins the warps' states: to the partial results of `to` (a slot), or to
  // the output (to < 0).
  auto join = [&](int to) {
    const float* all = reinterpret_cast<const float*>(smem);
    for (int x = threadIdx.x; x < kRows * (D / 4); x += kPrThreads) {
      const int r = x / (D / 4), c = (x % (D / 4)) * 4;
      const int row = row0 + r;
      if (row < 0) continue;
      float top = kNegInfR;
#pragma unroll
      for (int w = 0; w < kPrWarps; ++w) top = fmaxf(top, s_m[w][r]);
      float den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kPrWarps; ++w) {
        // A warp without a visible key has l = 0 and O = 0 (or NaN in both,
        // which the row then shows).
        const float f = s_m[w][r] == kNegInfR ? 1.f : ex2_approx(s_m[w][r] - top);
        den = fmaf(f, s_l[w][r], den);
        const float4 v = *reinterpret_cast<const float4*>(all + (w * kRows + r) * D + c);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      const float inv = den == 0.f ? 0.f : 1.f / den;
      const float ref = top == kNegInfR ? 0.f : top;
      const float lse = den == 0.f ? kNegInfR : (ref + __log2f(den)) * kLn2R;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (to >= 0) {
        const size_t part = (static_cast<size_t>(to) * Hk + h) * kRows + r;
        *reinterpret_cast<float4*>(p.o_part + part * D + c) = acc;
        if (c == 0) p.lse_part[part] = lse;
      } else {
        const int tok = row / G;
        const size_t at_row =
            static_cast<size_t>(tok0 + tok) * p.num_heads + h * G + (row - tok * G);
        *reinterpret_cast<uint2*>(p.out + at_row * D + c) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (c == 0 && p.lse != nullptr) p.lse[at_row] = lse;
      }
    }
  };
  join(slot);
  if (slot < 0 || PLAN || MT > 1) return;  // else paged_merge_kernel joins them

  // The last of an item's splits to be done joins them all, in their order:
  // each warp takes every fourth split, with its own running maximum.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(p.arrived + static_cast<size_t>(w.item) * Hk + h, 1) == w.n - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  const int splits = w.n;
  const size_t part0 = (static_cast<size_t>(w.slot0) * Hk + h) * kRows;
  const size_t pitch = static_cast<size_t>(Hk) * kRows;  // rows from split to split
  constexpr int kPer = D / 32;                          // floats of a row each lane owns
  constexpr int kAhead = 4;                             // splits in flight of each of
  constexpr int kAbreast = 4;                           // so many rows
  for (int r0 = max(0, -row0); r0 < kRows; r0 += kAbreast) {
    float mx[kAbreast], sum[kAbreast], acc[kAbreast][kPer];
#pragma unroll
    for (int i = 0; i < kAbreast; ++i) {
      mx[i] = kNegInfR;
      sum[i] = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) acc[i][q] = 0.f;
    }
    for (int s0 = warp; s0 < splits; s0 += kAhead * kPrWarps) {
      float x[kAbreast][kAhead], v[kAbreast][kAhead][kPer];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int s = s0 + u * kPrWarps;
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) {
          x[i][u] = kNegInfR;
#pragma unroll
          for (int q = 0; q < kPer; ++q) v[i][u][q] = 0.f;
          if (s < splits && r0 + i < kRows) {
            const size_t part = part0 + s * pitch + r0 + i;
            x[i][u] = __ldcg(p.lse_part + part) * kLog2eR;
            const float* src = p.o_part + part * D + lane * kPer;
            if (kPer == 4) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
              v[i][u][0] = f.x;
              v[i][u][1] = f.y;
              v[i][u][2 % kPer] = f.z;
              v[i][u][3 % kPer] = f.w;
            } else {
              const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
              v[i][u][0] = f.x;
              v[i][u][1] = f.y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAbreast; ++i) {
        float mn = mx[i];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) mn = fmaxf(mn, x[i][u]);
        const float alpha = mx[i] == kNegInfR ? 0.f : ex2_approx(mx[i] - mn);
        mx[i] = mn;
        sum[i] *= alpha;
#pragma unroll
        for (int q = 0; q < kPer; ++q) acc[i][q] *= alpha;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float f = x[i][u] == kNegInfR ? 0.f : ex2_approx(x[i][u] - mn);
          sum[i] += f;
#pragma unroll
          for (int q = 0; q < kPer; ++q) acc[i][q] = fmaf(f, v[i][u][q], acc[i][q]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAbreast; ++i) {
      const int r = r0 + i;
      if (r >= kRows) break;
      if (lane == 0) {
        s_m[warp][r] = mx[i];
        s_l[warp][r] = sum[i];
      }
#pragma unroll
      for (int q = 0; q < kPer; q += 2)
        *reinterpret_cast<float2*>(so + r * D + lane * kPer + q) =
            make_float2(acc[i][q], acc[i][q + 1]);
    }
  }
  __syncthreads();
  join(-1);
}

template <int D, int MT, bool HALF, bool PLAN>
static cudaError_t launch_paged_rows_t(const PagedParams& p, cudaStream_t stream) {
  auto kern = paged_rows_kernel<D, MT, HALF, PLAN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             RowsCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.max_work * p.num_kv_heads));
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = RowsCfg<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PLAN ? 0 : 1;  // after the schedule kernel
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, int MT, bool HALF>
static cudaError_t launch_paged_rows_p(const PagedParams& p, cudaStream_t stream) {
  return p.shape.plan ? launch_paged_rows_t<D, MT, HALF, true>(p, stream)
                      : launch_paged_rows_t<D, MT, HALF, false>(p, stream);
}

template <int D>
static cudaError_t launch_paged_rows_d(const PagedParams& p, cudaStream_t stream) {
  if (p.shape.rows != 16) return launch_paged_rows_p<D, 2, false>(p, stream);
  return p.max_seqlen * p.group <= 8 ? launch_paged_rows_p<D, 1, true>(p, stream)
                                     : launch_paged_rows_p<D, 1, false>(p, stream);
}

cudaError_t launch_paged_rows(const PagedParams& p, int D, cudaStream_t stream) {
  return D == 64 ? launch_paged_rows_d<64>(p, stream) : launch_paged_rows_d<128>(p, stream);
}

}  // namespace cpattn
