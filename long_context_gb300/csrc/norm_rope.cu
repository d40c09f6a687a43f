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
// Without weights dx is g: the forward kernel with its sine negated.
//
// HBM bound: a row is read once and written once (the backward reads two rows
// and writes one).  D / 8 lanes own a row.  The rows reach shared memory by
// 16-byte asynchronous copies, so that many are in flight without registers;
// from there a lane takes both members of its pairs, four features at its two
// places (4 c and R/2 + 4 c for lane c of a half-split rotation, else 8 c and
// 8 c + 4), so no value passes between lanes but the mean's partial sums.
// Everything between the load and the store is fp32 in registers, in packed
// pairs, rounded to bf16 once.
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"
#include "seq.cuh"

namespace cpattn {

namespace {

constexpr int kNrThreads = 256;
constexpr int kUnit = 2;    // heads of one batch of copies
constexpr int kErrArg = 1;   // CPATTN_ERR_INVALID_ARG

// Four bf16 values as two packed pairs of floats.
__device__ __forceinline__ void unpack4(const uint2& u, float2* f) {
  f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ uint2 pack4(const float2* f) {
  return make_uint2(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y));
}
__device__ __forceinline__ float2 swap2(const float2& v) { return make_float2(v.y, v.x); }
__device__ __forceinline__ float2 both2(float v) { return make_float2(v, v); }

// Sum over the lanes of a row (groups of LG lanes never straddle a warp).
template <int LG>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's features are a (four at `lo`) and b (four at `hi`):
//   y_a = a ac + a' as,  y_b = b bc + b' bs,
// where a', b' are the pairs' other members: b and a (half split), or a and b
// with their pairs swapped (interleaved).
struct Turn {
  float2 ac[2], as[2], bc[2], bs[2];
  int lo, hi;
  bool on;  // the lane's features turn
};

__device__ __forceinline__ void place_lane(Turn& t, int c, int rot, bool interleaved) {
  t.on = c < (rot >> 3);
  const bool apart = t.on && !interleaved;
  t.lo = apart ? 4 * c : 8 * c;
  t.hi = apart ? (rot >> 1) + 4 * c : 8 * c + 4;
}

// Coefficients of the position whose table row is `row` (valid: the row may be
// read); `sgn` is 1 for the rotation and -1 for its inverse.
template <bool INTERLEAVED>
__device__ __forceinline__ void load_turn(Turn& t, const float* row, int rot, int c, bool valid,
                                          float sgn) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t.ac[i] = t.bc[i] = both2(1.f);
    t.as[i] = t.bs[i] = both2(0.f);
  }
  if (!t.on || !valid) return;
  const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 4 * c));
  const float4 sv = __ldg(reinterpret_cast<const float4*>(row + (rot >> 1) + 4 * c));
  const float cs[4] = {cv.x, cv.y, cv.z, cv.w};
  const float sn[4] = {sgn * sv.x, sgn * sv.y, sgn * sv.z, sgn * sv.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (INTERLEAVED) {
      t.ac[i] = both2(cs[i]);
      t.as[i] = make_float2(-sn[i], sn[i]);
      t.bc[i] = both2(cs[2 + i]);
      t.bs[i] = make_float2(-sn[2 + i], sn[2 + i]);
    } else {
      t.ac[i] = t.bc[i] = make_float2(cs[2 * i], cs[2 * i + 1]);
      t.as[i] = make_float2(-sn[2 * i], -sn[2 * i + 1]);
      t.bs[i] = make_float2(sn[2 * i], sn[2 * i + 1]);
    }
  }
}

template <bool INTERLEAVED>
__device__ __forceinline__ void apply_turn(const Turn& t, float2* a, float2* b) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 pa = INTERLEAVED ? swap2(a[i]) : b[i];
    const float2 pb = INTERLEAVED ? swap2(b[i]) : a[i];
    const float2 ya = __fmul2_rn(a[i], t.ac[i]), yb = __fmul2_rn(b[i], t.bc[i]);
    // Features that do not turn take no product with a partner (0 times an
    // infinity).
    a[i] = t.on ? __ffma2_rn(pa, t.as[i], ya) : ya;
    b[i] = t.on ? __ffma2_rn(pb, t.bs[i], yb) : yb;
  }
}

}  // namespace

template <int D, bool INTERLEAVED, bool PAGED, int NB>
__global__ void __launch_bounds__(kNrThreads, PAGED ? 4 : 5) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LG = D / 8;
  constexpr int run = NB * kUnit;  // heads of a unit
  extern __shared__ __align__(16) uint8_t ring[];  // [run][threads] pieces of 16 bytes
  constexpr int kGroups = kNrThreads / LG;
  const int lane = threadIdx.x & 31;
  const int c = lane % LG;
  const int uq = (p.q_heads + run - 1) / run;
  const int uk = (p.kv_heads + run - 1) / run;
  const int upt = uq + (PAGED ? 2 : 1) * uk;  // units of a token
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LG;
  const bool live = unit < p.total_tokens * upt;
  const int token = live ? static_cast<int>(static_cast<unsigned>(unit) / upt) : 0;
  int hu = live ? static_cast<int>(static_cast<unsigned>(unit) - token * upt) : 0;
  // Which of q (0), k (1), v (2) this unit belongs to.
  const int which = hu < uq ? 0 : (hu < uq + uk ? 1 : 2);
  hu -= which == 0 ? 0 : (which == 1 ? uq : uq + uk);
  const int h0 = hu * run;
  const int heads = live ? min(h0 + run, which == 0 ? p.q_heads : p.kv_heads) : 0;
  const __nv_bfloat16* in =
      (which == 0 ? p.q : which == 1 ? p.k : p.v) +
      static_cast<size_t>(token) *
          (which == 0 ? p.q_stride : which == 1 ? p.k_stride : p.v_stride);
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      const int i = nb * kUnit + u;
      if (h0 + i < heads) cp_async16(mine + i * (kNrThreads * 16), in + (h0 + i) * D + c * 8, 16);
    }
    cp_async_commit();
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

  Turn t;
  const bool turning = p.table != nullptr;
  const bool plain = PAGED && which == 2;  // values are copied as they are
  place_lane(t, c, turning ? p.rot : 0, INTERLEAVED);
  load_turn<INTERLEAVED>(t, p.table + static_cast<size_t>(ok ? pos : 0) * p.rot, p.rot, c,
                         ok && !plain, p.sign);
  // The weights go into the rotation's coefficients: with n = x r w,
  // y = r (x (w cos) + x' (w' sin)).
  const __nv_bfloat16* wp = which == 0 ? p.q_weight : p.k_weight;
  const bool normed = wp != nullptr;  // the same for every lane: both weights or no queries
  if (normed) {
    float2 wa[2], wb[2];
    unpack4(__ldg(reinterpret_cast<const uint2*>(wp + t.lo)), wa);
    unpack4(__ldg(reinterpret_cast<const uint2*>(wp + t.hi)), wb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t.ac[i] = __fmul2_rn(t.ac[i], wa[i]);
      t.bc[i] = __fmul2_rn(t.bc[i], wb[i]);
      t.as[i] = __fmul2_rn(t.as[i], INTERLEAVED ? swap2(wa[i]) : wb[i]);
      t.bs[i] = __fmul2_rn(t.bs[i], INTERLEAVED ? swap2(wb[i]) : wa[i]);
    }
  }
  const uint8_t* row = ring + (threadIdx.x - c) * 16;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    // This batch's rows have landed, every lane's part of them.
    if (nb == 0) cp_async_wait<NB - 1>();
    else if (nb == 1) cp_async_wait<(NB > 2 ? NB - 2 : 0)>();
    else if (nb == 2) cp_async_wait<(NB > 3 ? NB - 3 : 0)>();
    else cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      const int i = nb * kUnit + u, h = h0 + i;
      const uint2 xa = *reinterpret_cast<const uint2*>(row + i * (kNrThreads * 16) + t.lo * 2);
      const uint2 xb = *reinterpret_cast<const uint2*>(row + i * (kNrThreads * 16) + t.hi * 2);
      float2 a[2], b[2];
      unpack4(xa, a);
      unpack4(xb, b);
      if (normed) {
        float2 ss = __fmul2_rn(a[0], a[0]);
        ss = __ffma2_rn(a[1], a[1], ss);
        ss = __ffma2_rn(b[0], b[0], ss);
        ss = __ffma2_rn(b[1], b[1], ss);
        const float2 r = both2(rsqrtf(row_sum<LG>(ss.x + ss.y) * (1.f / D) + p.eps));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[k] = __fmul2_rn(a[k], r);
          b[k] = __fmul2_rn(b[k], r);
        }
      }
      apply_turn<INTERLEAVED>(t, a, b);
      if (ok && h < heads) {
        *reinterpret_cast<uint2*>(out + h * D + t.lo) = plain ? xa : pack4(a);
        *reinterpret_cast<uint2*>(out + h * D + t.hi) = plain ? xb : pack4(b);
      }
    }
  }
}

// Gradients.  A fixed number of CTAs walk the units (RUN batches of UNIT heads
// of one token): the first q_ctas take the query heads, the others the key heads, so
// a lane holds one weight's 8 features and their sums of g hat in registers.
// The CTA adds its lane groups in shared memory and norm_rope_dw_kernel adds
// the CTAs' rows: the same order in every run, no atomics.
template <int D, bool INTERLEAVED, int UNIT, int RUN>
__global__ void __launch_bounds__(kNrThreads, 3) norm_rope_bwd_kernel(const NormRopeBwdParams p) {
  constexpr int LG = D / 8;
  constexpr int kGroups = kNrThreads / LG;
  extern __shared__ __align__(16) uint8_t ring[];  // [2][gradients, inputs][UNIT][threads] x 16
  __shared__ __align__(16) float red[kGroups][D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int c = lane % LG;
  const int group = threadIdx.x / LG;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.q_ctas;
  const int cta = static_cast<int>(blockIdx.x) - (is_k ? p.q_ctas : 0);
  const int ctas = is_k ? static_cast<int>(gridDim.x) - p.q_ctas : p.q_ctas;
  const int heads = is_k ? p.kv_heads : p.q_heads;
  const int upt = (heads + RUN * UNIT - 1) / (RUN * UNIT);  // units of a token
  const long long units = p.total_tokens * upt;
  const __nv_bfloat16* xin = is_k ? p.k : p.q;
  const __nv_bfloat16* gin = is_k ? p.dk_out : p.dq_out;
  __nv_bfloat16* out = is_k ? p.dk : p.dq;
  const long long x_stride = is_k ? p.k_stride : p.q_stride;
  const long long g_stride = is_k ? p.dk_out_stride : p.dq_out_stride;
  const long long o_stride = is_k ? p.dk_stride : p.dq_stride;
  const bool turning = p.table != nullptr;
  Turn t;
  place_lane(t, c, turning ? p.rot : 0, INTERLEAVED);
  float2 wa[2], wb[2], dwa[2], dwb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) dwa[i] = dwb[i] = both2(0.f);
  const __nv_bfloat16* wp = is_k ? p.k_weight : p.q_weight;
  unpack4(__ldg(reinterpret_cast<const uint2*>(wp + t.lo)), wa);
  unpack4(__ldg(reinterpret_cast<const uint2*>(wp + t.hi)), wb);
  const long long stride = static_cast<long long>(ctas) * kGroups;
  // The next batch's rows (of this unit or the next) are copied to shared memory
  // while the current one's are used; a unit's batches share its angles.  Whole
  // warps stay in the loop together (the shuffles are warp-wide).
  struct Place {
    int token, h0, end, pos;
  };
  auto place = [&](long long u) {
    Place a = {0, 0, 0, 0};
    if (u < units) {
      a.token = static_cast<int>(static_cast<unsigned>(u) / upt);
      a.h0 = static_cast<int>(static_cast<unsigned>(u) - a.token * upt) * (RUN * UNIT);
      a.end = min(a.h0 + RUN * UNIT, heads);
      if (turning) a.pos = __ldg(p.positions + a.token);
    }
    return a;
  };
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const uint8_t* row = ring + (threadIdx.x - c) * 16;
  auto load = [&](const Place& a, int h0, int buf) {
#pragma unroll
    for (int u = 0; u < UNIT; ++u) {
      const int h = h0 + u;
      const uint32_t dst = mine + (buf * 2 * UNIT + u) * (kNrThreads * 16);
      if (h < a.end) {
        cp_async16(dst, gin + a.token * g_stride + h * D + c * 8, 16);
        cp_async16(dst + UNIT * (kNrThreads * 16), xin + a.token * x_stride + h * D + c * 8, 16);
      }
    }
    cp_async_commit();
  };
  long long unit = static_cast<long long>(cta) * kGroups + group;
  Place at = place(unit);
  load(at, at.h0, 0);
  int buf = 0;
  for (long long base = static_cast<long long>(cta) * kGroups; base < units; base += stride) {
    unit += stride;
    const Place ahead = place(unit);
    bool ok = at.end > 0;
    if (turning) {
      const bool good = at.pos >= 0 && at.pos < p.max_pos;
      if (ok && !good && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArg);
      ok = ok && good;
    }
    load_turn<INTERLEAVED>(t, p.table + static_cast<size_t>(ok ? at.pos : 0) * p.rot, p.rot, c, ok,
                           -1.f);
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      if (j + 1 < RUN) load(at, at.h0 + (j + 1) * UNIT, buf ^ 1);
      else load(ahead, ahead.h0, buf ^ 1);
      cp_async_wait<1>();
      __syncwarp();
#pragma unroll
      for (int u = 0; u < UNIT; ++u) {
        const int h = at.h0 + j * UNIT + u;
        const bool count = ok && h < at.end;
        const uint8_t* piece = row + (buf * 2 * UNIT + u) * (kNrThreads * 16);
        float2 a[2], b[2];
        unpack4(*reinterpret_cast<const uint2*>(piece + t.lo * 2), a);
        unpack4(*reinterpret_cast<const uint2*>(piece + t.hi * 2), b);
        apply_turn<INTERLEAVED>(t, a, b);  // g
        const uint8_t* px = piece + UNIT * (kNrThreads * 16);
        float2 xa[2], xb[2];
        unpack4(*reinterpret_cast<const uint2*>(px + t.lo * 2), xa);
        unpack4(*reinterpret_cast<const uint2*>(px + t.hi * 2), xb);
        float2 ss = both2(0.f), dot = both2(0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ss = __ffma2_rn(xa[k], xa[k], ss);
          ss = __ffma2_rn(xb[k], xb[k], ss);
          dot = __ffma2_rn(__fmul2_rn(a[k], wa[k]), xa[k], dot);
          dot = __ffma2_rn(__fmul2_rn(b[k], wb[k]), xb[k], dot);
        }
        const float sum = row_sum<LG>(ss.x + ss.y);
        const float prod = row_sum<LG>(dot.x + dot.y);
        const float r = rsqrtf(sum * (1.f / D) + p.eps);
        const float2 r2 = both2(r);
        const float2 m2 = both2(-prod * r * (1.f / D));  // -mean(u hat)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 ha = __fmul2_rn(xa[k], r2), hb = __fmul2_rn(xb[k], r2);
          if (count) {
            dwa[k] = __ffma2_rn(a[k], ha, dwa[k]);
            dwb[k] = __ffma2_rn(b[k], hb, dwb[k]);
          }
          a[k] = __fmul2_rn(__ffma2_rn(ha, m2, __fmul2_rn(a[k], wa[k])), r2);
          b[k] = __fmul2_rn(__ffma2_rn(hb, m2, __fmul2_rn(b[k], wb[k])), r2);
        }
        if (count) {
          __nv_bfloat16* dst = out + at.token * o_stride + h * D;
          *reinterpret_cast<uint2*>(dst + t.lo) = pack4(a);
          *reinterpret_cast<uint2*>(dst + t.hi) = pack4(b);
        }
      }
      __syncwarp();  // the buffer is refilled by all lanes
      buf ^= 1;
    }
    at = ahead;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    *reinterpret_cast<float2*>(&red[group][t.lo + 2 * k]) = dwa[k];
    *reinterpret_cast<float2*>(&red[group][t.hi + 2 * k]) = dwb[k];
  }
  __syncthreads();
  for (int f = threadIdx.x; f < D; f += kNrThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) s += red[g][f];
    p.partial[static_cast<size_t>(blockIdx.x) * D + f] = s;
  }
}

// Adds the CTAs' partial weight gradients: 32 warps share 32 features of one
// weight, each taking every 32nd row (a few hundred rows: two round trips of
// eight loads), and are added in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* partial, int q_rows, int rows, int D, float* dqw, float* dkw) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = D / 32;
  const bool is_k = static_cast<int>(blockIdx.x) >= per;
  const int col = (static_cast<int>(blockIdx.x) - (is_k ? per : 0)) * 32;
  const int r1 = is_k ? rows : q_rows;
  float s = 0.f;
#pragma unroll 8
  for (int r = (is_k ? q_rows : 0) + warp; r < r1; r += 32)
    s += __ldcg(partial + static_cast<size_t>(r) * D + col + lane);
  red[warp][lane] = s;
  __syncthreads();
  // Warp w adds the 32 sums of feature w.
  float t = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) (is_k ? dkw : dqw)[col + warp] = t;
}

template <int D, int NB>
static cudaError_t launch_norm_rope_t(const NormRopeParams& p, bool interleaved, long long units,
                                      cudaStream_t stream) {
  const int groups = kNrThreads / (D / 8);
  const unsigned grid = static_cast<unsigned>((units + groups - 1) / groups);
  constexpr int kSmem = NB * kUnit * kNrThreads * 16;
  const bool paged = p.page_table != nullptr;
  auto kern = paged ? (interleaved ? norm_rope_kernel<D, true, true, NB>
                                   : norm_rope_kernel<D, false, true, NB>)
                    : (interleaved ? norm_rope_kernel<D, true, false, NB>
                                   : norm_rope_kernel<D, false, false, NB>);
  static_assert(kSmem <= 48 * 1024, "no opt-in needed");
  kern<<<grid, kNrThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_norm_rope_d(const NormRopeParams& p, bool interleaved, int num_sms,
                                      cudaStream_t stream) {
  auto units_at = [&](int run) {
    const long long uq = (p.q_heads + run - 1) / run, uk = (p.kv_heads + run - 1) / run;
    return p.total_tokens * (uq + (p.page_table != nullptr ? 2 : 1) * uk);
  };
  // Eight heads a lane group share a position's angles and have four times the
  // loads in flight of two (16,384 tokens of 32 + 32 heads of 128: 85 us, four heads
  // 95 us, two 128 us), as long as they leave every SM several rounds of CTAs (a
  // decoding step wants its few rows spread out, 32 tokens of 32 + 8 heads of 128:
  // two heads 4.8 us, four 6.1 us) and not too many of their places go unused, as
  // those are computed too.  Less than half may in runs of eight, half in runs of
  // four (32,768 tokens, heads of 128 / 64, us in runs of eight, four and two: 5 + 5
  // heads, three eighths unused, 36.9, 43.0, 47.1 / 20.5, 24.6, 25.4; 4 + 4, half and
  // none, 34.7, 28.6, 33.0 / 18.5, 14.7, 18.5; 3 + 1, three quarters and half, 30.8,
  // 22.6, 24.6 / 16.5, 12.4, 13.7).
  const long long many = 12LL * num_sms * (kNrThreads / (D / 8));
  if (units_at(1) == 0) return cudaSuccess;
  auto fits = [&](int run) {
    const long long places = units_at(run) * run, most = 2 * units_at(1);
    return units_at(run) >= many && (run > 2 * kUnit ? places < most : places <= most);
  };
  if (fits(4 * kUnit))
    return launch_norm_rope_t<D, 4>(p, interleaved, units_at(4 * kUnit), stream);
  if (fits(2 * kUnit))
    return launch_norm_rope_t<D, 2>(p, interleaved, units_at(2 * kUnit), stream);
  return launch_norm_rope_t<D, 1>(p, interleaved, units_at(kUnit), stream);
}

cudaError_t launch_norm_rope(const NormRopeParams& p, int D, bool interleaved, int num_sms,
                             cudaStream_t stream) {
  return D == 64 ? launch_norm_rope_d<64>(p, interleaved, num_sms, stream)
                 : launch_norm_rope_d<128>(p, interleaved, num_sms, stream);
}

template <int D, int UNIT, int RUN>
static cudaError_t launch_norm_rope_bwd_t(NormRopeBwdParams p, bool interleaved, float* dqw,
                                          float* dkw, int num_sms, cudaStream_t stream) {
  constexpr int kSmem = 2 * 2 * UNIT * kNrThreads * 16;
  constexpr int kHeads = RUN * UNIT;
  const int groups = kNrThreads / (D / 8);
  const long long uq = (p.q_heads + kHeads - 1) / kHeads, uk = (p.kv_heads + kHeads - 1) / kHeads;
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
    auto kern = interleaved ? norm_rope_bwd_kernel<D, true, UNIT, RUN>
                            : norm_rope_bwd_kernel<D, false, UNIT, RUN>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kern<<<g, kNrThreads, kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // No tokens: both sums are empty (zero rows of partials) and come out zero.
  const bool any = p.total_tokens > 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * D / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = any ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(p.partial),
                            any ? p.q_ctas : 0, any ? static_cast<int>(g) : 0, D, dqw, dkw);
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdParams& p, int D, bool interleaved, float* dqw,
                                 float* dkw, int num_sms, cudaStream_t stream) {
  // Runs of four heads (two batches of two) share a position's angles and the
  // unit's bookkeeping: 14,000 tokens of 40 heads of 128 73 us, runs of two 82 us
  // (16,384 of 64 heads 126 us, runs of eight 135 us).  They have to leave every
  // lane group three units or the groups even out badly: 4,999 tokens of 20 heads
  // of 64 16.4 us, runs of two 14.5 us.
  const long long groups = 3LL * num_sms * (kNrThreads / (D / 8));
  const bool many = p.total_tokens * ((p.q_heads + 3) / 4 + (p.kv_heads + 3) / 4) >= 3 * groups;
  if (D == 64)
    return many ? launch_norm_rope_bwd_t<64, 2, 2>(p, interleaved, dqw, dkw, num_sms, stream)
                : launch_norm_rope_bwd_t<64, 2, 1>(p, interleaved, dqw, dkw, num_sms, stream);
  return many ? launch_norm_rope_bwd_t<128, 2, 2>(p, interleaved, dqw, dkw, num_sms, stream)
              : launch_norm_rope_bwd_t<128, 2, 1>(p, interleaved, dqw, dkw, num_sms, stream);
}

}  // namespace cpattn
