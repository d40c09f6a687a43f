// RMS norm of every query and key head with the rotary position embedding in
// the same pass, its gradients, and the same pass writing keys and values into
// a paged KV cache.
//
// For a head row x [D] at position p, weight w [D]:
//   r = 1 / sqrt(mean(x^2) + eps),   n = x r w        (n = x without weights)
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin for the pairs (a, b) of
//   the first R features at angle j of position p; the other features are n.
// Pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved; the table row of
// position p holds cos of the R/2 angles, then sin.  Gradients, with
// hat = x r: g is dy rotated back (sin negated), and
//   dw = sum over rows of g hat,  u = g w,  dx = r (u - hat mean(u hat)).
//
// HBM bound: a row is read once and written once (the backward reads two rows
// and writes one).  D / 8 lanes own a row, 16 bytes each, so the mean is a few
// shuffles inside the row's lanes and a half-split pair is one shuffle away;
// everything between the load and the store is fp32 in registers, rounded to
// bf16 once.  A lane group takes kUnit heads of one token at a time: their
// loads are in flight together and share the position's cos and sin, which
// are the only loads that depend on another load.
#include <cuda_bf16.h>

#include "kernels.h"

namespace cpattn {

namespace {

constexpr int kNrThreads = 256;
constexpr int kUnit = 4;     // heads of one token a lane group has in flight
constexpr int kBwdUnit = 2;  // backward: two rows (x, dy) per head
constexpr int kErrArg = 1;   // CPATTN_ERR_INVALID_ARG

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = __bfloat1622float2(h[e]);
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  return u;
}

// Sum over the lanes of a row (groups of LG lanes never straddle a warp).
template <int LG>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rotation's coefficients for the 8 features of lane chunk c:
// y_e = n_e cs[e] + partner_e sn[e], the sign of the sine folded into sn.
// `partner_lane` is the lane (of the warp) that holds the partner features
// (half split); chunks at or beyond R take no part.
struct Turn {
  float cs[8], sn[8];
  int partner_lane;
  bool on;
};

template <bool INTERLEAVED>
__device__ __forceinline__ void load_turn(Turn& t, const float* row, int rot, int c, int lane,
                                          bool valid) {
  const int f0 = c * 8, half = rot >> 1;
  t.on = f0 < rot;
  t.partner_lane = lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t.cs[e] = 1.f;
    t.sn[e] = 0.f;
  }
  if (!t.on) return;
  if (INTERLEAVED) {
    if (valid) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + (f0 >> 1)));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + (f0 >> 1)));
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w};
      const float ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t.cs[2 * e] = t.cs[2 * e + 1] = cc[e];
        t.sn[2 * e] = -ss[e];
        t.sn[2 * e + 1] = ss[e];
      }
    }
  } else {
    const bool first = f0 < half;
    const int j0 = first ? f0 : f0 - half;
    t.partner_lane = first ? lane + (half >> 3) : lane - (half >> 3);
    if (valid) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row + j0) + q);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + j0) + q);
        t.cs[4 * q] = cv.x;
        t.cs[4 * q + 1] = cv.y;
        t.cs[4 * q + 2] = cv.z;
        t.cs[4 * q + 3] = cv.w;
        t.sn[4 * q] = first ? -sv.x : sv.x;
        t.sn[4 * q + 1] = first ? -sv.y : sv.y;
        t.sn[4 * q + 2] = first ? -sv.z : sv.z;
        t.sn[4 * q + 3] = first ? -sv.w : sv.w;
      }
    }
  }
}

// n -> y in place; `sgn` is 1 for the rotation and -1 for its inverse.  Every
// lane of the warp executes it (the partner exchange is a shuffle).
template <bool INTERLEAVED>
__device__ __forceinline__ void apply_turn(const Turn& t, float* n, float sgn) {
  float pn[8];
  if (INTERLEAVED) {
#pragma unroll
    for (int e = 0; e < 8; ++e) pn[e] = n[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) pn[e] = __shfl_sync(0xffffffffu, n[e], t.partner_lane);
  }
  if (t.on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = n[e] * t.cs[e] + pn[e] * (sgn * t.sn[e]);
  }
}

// Sequence of token t: the last b with cu[b] <= t, found LG candidates at a
// time by the lanes of one row (B >= 1).  Every lane of the warp executes it.
template <int LG>
__device__ __forceinline__ int find_seq(const int* cu, int B, int t, int c, int lane) {
  const int shift = (lane / LG) * LG;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + LG - 1) / LG;
    const int i = lo + c * step;
    const bool le = c * step < n && (c == 0 || __ldg(cu + i) <= t);
    const unsigned hit =
        (__ballot_sync(0xffffffffu, le) >> shift) & ((LG == 32) ? 0xffffffffu : ((1u << LG) - 1));
    // Lengths are not negative in a valid batch, so the hits are a prefix; in
    // an invalid one the caller's check of the result rejects it.
    const int k = 31 - __clz(hit);
    const int off = k * step;
    n = min(step, n - off);
    lo += off;
  }
  return lo;
}

}  // namespace

template <int D, bool INTERLEAVED, bool PAGED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LG = D / 8;
  constexpr int kGroups = kNrThreads / LG;
  const int lane = threadIdx.x & 31;
  const int c = lane % LG;
  const int uq = (p.q_heads + kUnit - 1) / kUnit;
  const int uk = (p.kv_heads + kUnit - 1) / kUnit;
  const int upt = uq + (PAGED ? 2 : 1) * uk;  // units of a token
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LG;
  const bool live = unit < p.total_tokens * upt;
  const int token = live ? static_cast<int>(static_cast<unsigned>(unit) / upt) : 0;
  int hu = live ? static_cast<int>(static_cast<unsigned>(unit) - token * upt) : 0;
  // Which of q (0), k (1), v (2) this unit belongs to.
  const int which = hu < uq ? 0 : (hu < uq + uk ? 1 : 2);
  hu -= which == 0 ? 0 : (which == 1 ? uq : uq + uk);
  const int h0 = hu * kUnit;
  const int heads = which == 0 ? p.q_heads : p.kv_heads;
  const __nv_bfloat16* in =
      (which == 0 ? p.q : which == 1 ? p.k : p.v) +
      static_cast<size_t>(token) *
          (which == 0 ? p.q_stride : which == 1 ? p.k_stride : p.v_stride);
  uint4 x[kUnit];
#pragma unroll
  for (int u = 0; u < kUnit; ++u) {
    x[u] = make_uint4(0, 0, 0, 0);
    if (live && h0 + u < heads)
      x[u] = __ldcs(reinterpret_cast<const uint4*>(in + static_cast<size_t>(h0 + u) * D) + c);
  }

  bool ok = live;
  int pos = 0;
  __nv_bfloat16* out;
  if (PAGED) {
    const int b = find_seq<LG>(p.cu_seqlens, p.num_seqs, token, c, lane);
    const int lo = __ldg(p.cu_seqlens + b), hi = __ldg(p.cu_seqlens + b + 1);
    const int kv = __ldg(p.kv_lens + b);
    // A token behind the last sequence belongs to none and is left alone.
    const bool behind = token >= __ldg(p.cu_seqlens + p.num_seqs);
    const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
    bool good = lo >= 0 && token >= lo && token < hi && kv >= 0 && kv <= cap;
    if (good) pos = kv - (hi - token);
    good = good && pos >= 0;
    int page = -1;
    if (good && ok) {
      page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages + (pos >> p.page_shift));
      good = page >= 0 && page < p.num_pages;
    }
    if (p.table != nullptr) good = good && pos < p.max_pos;
    if (ok && !good && !behind && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArg);
    ok = ok && good && !behind;
    if (which == 0) {
      out = p.q_out + static_cast<size_t>(token) * p.q_out_stride;
    } else {
      const size_t slot = pos & ((1 << p.page_shift) - 1);
      out = (which == 1 ? p.k_out : p.v_out) + static_cast<size_t>(ok ? page : 0) * p.page_stride +
            (ok ? slot : 0) * p.kv_heads * D;
    }
  } else {
    if (p.table != nullptr) {
      pos = live ? __ldg(p.positions + token) : 0;
      const bool good = pos >= 0 && pos < p.max_pos;
      if (live && !good && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArg);
      ok = ok && good;
    }
    out = (which == 0 ? p.q_out : p.k_out) +
          static_cast<size_t>(token) * (which == 0 ? p.q_out_stride : p.k_out_stride);
  }

  if (PAGED && __all_sync(0xffffffffu, which == 2 || !ok)) {
    // A warp of values alone: copied as they are.
#pragma unroll
    for (int u = 0; u < kUnit; ++u)
      if (ok && h0 + u < heads)
        *(reinterpret_cast<uint4*>(out + static_cast<size_t>(h0 + u) * D) + c) = x[u];
    return;
  }

  Turn t;
  const bool turning = p.table != nullptr;
  if (turning)
    load_turn<INTERLEAVED>(t, p.table + static_cast<size_t>(ok ? pos : 0) * p.rot, p.rot, c, lane,
                           ok);
  const __nv_bfloat16* wp = which == 0 ? p.q_weight : p.k_weight;
  float w[8];
  if (wp != nullptr) unpack8(__ldg(reinterpret_cast<const uint4*>(wp) + c), w);
#pragma unroll
  for (int u = 0; u < kUnit; ++u) {
    float n[8];
    unpack8(x[u], n);
    if (wp != nullptr) {  // the same for every lane: both weights or no queries
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(n[e], n[e], ss);
      const float r = rsqrtf(row_sum<LG>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = n[e] * r * w[e];
    }
    if (turning) apply_turn<INTERLEAVED>(t, n, 1.f);
    if (ok && h0 + u < heads)
      *(reinterpret_cast<uint4*>(out + static_cast<size_t>(h0 + u) * D) + c) =
          (PAGED && which == 2) ? x[u] : pack8(n);
  }
}

// Gradients.  A fixed number of CTAs walk the units (kBwdUnit heads of one
// token): the first q_ctas take the query heads, the others the key heads, so
// a lane holds one weight's 8 features and their sums of g hat in registers.
// The CTA adds its lane groups in shared memory and norm_rope_dw_kernel adds
// the CTAs' rows: the same order in every run, no atomics.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kNrThreads, 3) norm_rope_bwd_kernel(const NormRopeBwdParams p) {
  constexpr int LG = D / 8;
  constexpr int kGroups = kNrThreads / LG;
  __shared__ float red[kGroups][D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int c = lane % LG;
  const int group = threadIdx.x / LG;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.q_ctas;
  const int cta = static_cast<int>(blockIdx.x) - (is_k ? p.q_ctas : 0);
  const int ctas = is_k ? static_cast<int>(gridDim.x) - p.q_ctas : p.q_ctas;
  const int heads = is_k ? p.kv_heads : p.q_heads;
  const int upt = (heads + kBwdUnit - 1) / kBwdUnit;
  const long long units = p.total_tokens * upt;
  const __nv_bfloat16* xin = is_k ? p.k : p.q;
  const __nv_bfloat16* gin = is_k ? p.dk_out : p.dq_out;
  __nv_bfloat16* out = is_k ? p.dk : p.dq;
  const long long x_stride = is_k ? p.k_stride : p.q_stride;
  const long long g_stride = is_k ? p.dk_out_stride : p.dq_out_stride;
  const long long o_stride = is_k ? p.dk_stride : p.dq_stride;
  const bool normed = p.q_weight != nullptr;
  const bool turning = p.table != nullptr;
  float w[8], dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;
  if (normed) unpack8(__ldg(reinterpret_cast<const uint4*>(is_k ? p.k_weight : p.q_weight) + c), w);
  const long long stride = static_cast<long long>(ctas) * kGroups;
  // Whole warps stay in the loop together (the shuffles are warp-wide).
  for (long long base = static_cast<long long>(cta) * kGroups; base < units; base += stride) {
    const long long unit = base + group;
    const bool live = unit < units;
    const int token = live ? static_cast<int>(static_cast<unsigned>(unit) / upt) : 0;
    const int h0 =
        live ? static_cast<int>(static_cast<unsigned>(unit) - token * upt) * kBwdUnit : 0;
    const __nv_bfloat16* xt = xin + token * x_stride;
    const __nv_bfloat16* gt = gin + token * g_stride;
    uint4 xr[kBwdUnit], gr[kBwdUnit];
#pragma unroll
    for (int u = 0; u < kBwdUnit; ++u) {
      xr[u] = gr[u] = make_uint4(0, 0, 0, 0);
      if (live && h0 + u < heads) {
        gr[u] = __ldcs(reinterpret_cast<const uint4*>(gt + static_cast<size_t>(h0 + u) * D) + c);
        if (normed)
          xr[u] = __ldcs(reinterpret_cast<const uint4*>(xt + static_cast<size_t>(h0 + u) * D) + c);
      }
    }
    bool ok = live;
    Turn t;
    if (turning) {
      const int pos = live ? __ldg(p.positions + token) : 0;
      const bool good = pos >= 0 && pos < p.max_pos;
      if (live && !good && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArg);
      ok = ok && good;
      load_turn<INTERLEAVED>(t, p.table + static_cast<size_t>(ok ? pos : 0) * p.rot, p.rot, c,
                             lane, ok);
    }
#pragma unroll
    for (int u = 0; u < kBwdUnit; ++u) {
      const bool count = ok && h0 + u < heads;
      float g[8];
      unpack8(gr[u], g);
      if (turning) apply_turn<INTERLEAVED>(t, g, -1.f);
      if (normed) {
        float x[8];
        unpack8(xr[u], x);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[e], x[e], ss);
          dot = fmaf(g[e] * w[e], x[e], dot);
        }
        ss = row_sum<LG>(ss);
        dot = row_sum<LG>(dot);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = dot * r * (1.f / D);  // mean(u hat)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float hat = x[e] * r;
          if (count) dw[e] = fmaf(g[e], hat, dw[e]);
          g[e] = r * (g[e] * w[e] - hat * m);
        }
      }
      if (count)
        *(reinterpret_cast<uint4*>(out + token * o_stride + static_cast<size_t>(h0 + u) * D) + c) =
            pack8(g);
    }
  }
  if (!normed) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[group][c * 8 + e] = dw[e];
  __syncthreads();
  for (int f = threadIdx.x; f < D; f += kNrThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) s += red[g][f];
    p.partial[static_cast<size_t>(blockIdx.x) * D + f] = s;
  }
}

// Adds the CTAs' partial weight gradients: 8 warps share 32 features of one
// weight, each taking every eighth row, and are added in a fixed order.
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float* partial, int q_rows, int rows, int D, float* dqw, float* dkw) {
  __shared__ float red[8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = D / 32;
  const bool is_k = static_cast<int>(blockIdx.x) >= per;
  const int col = (static_cast<int>(blockIdx.x) - (is_k ? per : 0)) * 32 + lane;
  const int r1 = is_k ? rows : q_rows;
  float s = 0.f;
#pragma unroll 8
  for (int r = (is_k ? q_rows : 0) + warp; r < r1; r += 8)
    s += __ldcg(partial + static_cast<size_t>(r) * D + col);
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += red[w][lane];
    (is_k ? dkw : dqw)[col] = t;
  }
}

template <int D>
static cudaError_t launch_norm_rope_d(const NormRopeParams& p, bool interleaved,
                                      cudaStream_t stream) {
  const bool paged = p.page_table != nullptr;
  const long long uq = (p.q_heads + kUnit - 1) / kUnit, uk = (p.kv_heads + kUnit - 1) / kUnit;
  const long long units = p.total_tokens * (uq + (paged ? 2 : 1) * uk);
  const int groups = kNrThreads / (D / 8);
  const unsigned grid = static_cast<unsigned>((units + groups - 1) / groups);
  if (grid == 0) return cudaSuccess;
  if (paged) {
    if (interleaved) norm_rope_kernel<D, true, true><<<grid, kNrThreads, 0, stream>>>(p);
    else norm_rope_kernel<D, false, true><<<grid, kNrThreads, 0, stream>>>(p);
  } else {
    if (interleaved) norm_rope_kernel<D, true, false><<<grid, kNrThreads, 0, stream>>>(p);
    else norm_rope_kernel<D, false, false><<<grid, kNrThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const NormRopeParams& p, int D, bool interleaved,
                             cudaStream_t stream) {
  return D == 64 ? launch_norm_rope_d<64>(p, interleaved, stream)
                 : launch_norm_rope_d<128>(p, interleaved, stream);
}

cudaError_t launch_norm_rope_bwd(NormRopeBwdParams p, int D, bool interleaved, float* dqw,
                                 float* dkw, int num_sms, cudaStream_t stream) {
  const long long uq = (p.q_heads + kBwdUnit - 1) / kBwdUnit;
  const long long uk = (p.kv_heads + kBwdUnit - 1) / kBwdUnit;
  const int groups = kNrThreads / (D / 8);
  const long long needed = (p.total_tokens * (uq + uk) + groups - 1) / groups;
  // Three CTAs a SM, shared out by the number of heads; at least one for each.
  long long grid = num_sms * 3LL < kNormRopeBwdCtas ? num_sms * 3LL : kNormRopeBwdCtas;
  if (needed < grid) grid = needed;
  if (grid < 2) grid = 2;
  long long gq = (grid * uq + (uq + uk) / 2) / (uq + uk);
  gq = gq < 1 ? 1 : (gq > grid - 1 ? grid - 1 : gq);
  p.q_ctas = static_cast<int>(gq);
  const unsigned g = static_cast<unsigned>(grid);
  if (p.total_tokens > 0) {
    if (D == 64) {
      if (interleaved) norm_rope_bwd_kernel<64, true><<<g, kNrThreads, 0, stream>>>(p);
      else norm_rope_bwd_kernel<64, false><<<g, kNrThreads, 0, stream>>>(p);
    } else {
      if (interleaved) norm_rope_bwd_kernel<128, true><<<g, kNrThreads, 0, stream>>>(p);
      else norm_rope_bwd_kernel<128, false><<<g, kNrThreads, 0, stream>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.q_weight == nullptr) return cudaSuccess;
  // No tokens: both sums are empty (zero rows of partials) and come out zero.
  const bool any = p.total_tokens > 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * D / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = any ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(p.partial),
                            any ? p.q_ctas : 0, any ? static_cast<int>(g) : 0, D, dqw, dkw);
}

}  // namespace cpattn
