// A paged KV cache in 4 bits (fp4.cuh): quantising new tokens into it, reading
// tokens back, and reading a batch's caches into 16-bit pages for the tile kernel.
//
// Quantising, for 16 features x of a token and head (u the cache's power of two):
//   s = e4m3(min(max(max|x| / (6 u), 2^-9), 448)),  c = e2m1(x / (s u)),
// both to the nearest, halves to even, c saturating.  x has 8 significant bits and s
// four, so a border between two codes times s has at most 7: x is either on a border
// or off it by 2^-8 of it, and x times the rounded reciprocal of s, rounded to
// multiples of 2^-13, falls on the same side as the quotient (for s: 16
// significant bits).  The bytes are those that exact arithmetic gives.  A group with a
// NaN or an infinity gets the scale NaN.
//
// All three are HBM bound, 2.56 bytes a feature; the append spends 7 instructions on one
// where its bytes take the time of 14.  A lane takes 16 features of the append, one scale,
// and 8 of the others, 16 bytes of bf16.  60,000 tokens of 8 heads of 128 take 49.4 us in
// (6.4 TB/s with 4 us for the launch) and 51.5 us out; 16 caches of 300,000 tokens in all
// 304 us (6.4 TB/s); 34,816 tokens into pages 28 us (6.5 TB/s).
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "seq.cuh"

namespace cpattn {

namespace {

constexpr int kF4Threads = 256;
constexpr int kAppendRun = 2;  // heads of a unit of the append (of four: 47 registers more,
                               // a decoding step's pass 11.7 instead of 10.1 us)
constexpr int kGatherRun = 4;  // and of the gather (of two: 16 caches 324 instead of 304 us)
constexpr int kPagesCtas = 8;  // CTAs of an SM, the pages' kernel
constexpr int kErrArgF = 1;  // CPATTN_ERR_INVALID_ARG

// Place of a new token: its tile's first byte in head 0 of its page, or -1.
struct Fp4Place {
  long long at;
  int row;      // of the tile
  bool behind;  // behind the last sequence
};

template <int LG>
__device__ __forceinline__ Fp4Place find_place(const Fp4CacheParams& p, int tile_bytes, bool live,
                                               int token, int c, int lane) {
  Fp4Place r;
  const int b = find_seq<LG>(p.cu_seqlens, p.num_seqs, token, c, lane);
  const int lo = __ldg(p.cu_seqlens + b), hi = __ldg(p.cu_seqlens + b + 1);
  const int kv = __ldg(p.kv_lens + b);
  r.behind = token >= __ldg(p.cu_seqlens + p.num_seqs);
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  bool good = live && lo >= 0 && token >= lo && token < hi && kv >= 0 && kv <= cap;
  const int pos = good ? kv - (hi - token) : 0;
  good = good && pos >= 0;
  int page = -1;
  if (good) {
    page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages + (pos >> p.page_shift));
    good = page >= 0 && page < p.num_pages;
  }
  r.row = pos & (kFp4Tile - 1);
  const int tile = (pos & ((1 << p.page_shift) - 1)) / kFp4Tile;
  r.at = good && !r.behind
             ? static_cast<long long>(page) * p.page_stride + static_cast<long long>(tile) * tile_bytes
             : -1;
  return r;
}

// Eight codes without the signs of zeros.
__device__ __forceinline__ uint32_t plain_zeros(uint32_t w) {
  const uint32_t m = w & 0x77777777u;
  return w & ((m + 0x77777777u) | m);  // a half's top bit survives where its m is not 0
}

// The larger magnitude of each half, of a sign that does not matter; NaN if one is.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 bf16 values (two 16-byte pieces) to 8 bytes of codes and the scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4& a, const uint4& b, float inv_unit,
                                            uint32_t& scale) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = max_abs2(max_abs2(max_abs2(x[0], x[1]), max_abs2(x[2], x[3])),
                          max_abs2(max_abs2(x[4], x[5]), max_abs2(x[6], x[7])));
  top = max(top & 0x7fffu, (top >> 16) & 0x7fffu);  // a NaN or an infinity is above the rest
  // The quotient to 16 significant bits, which those between two scales pass exactly.
  const float t = __uint_as_float(
      (__float_as_uint(__uint_as_float(top << 16) * inv_unit * (1.f / kFp4Top)) + 0x80u) &
      0xffffff00u);
  float s;
  scale = to_e4m3(fminf(fmaxf(t, kFp4MinScale), kFp4MaxScale), s);
  const float inv = __fdividef(inv_unit, s);
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w = x[2 * i + j];
      q[j] = __ffma2_rn(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)),
                        make_float2(inv, inv), make_float2(1536.f, 1536.f));
      q[j] = __fadd2_rn(q[j], make_float2(-1536.f, -1536.f));  // multiples of 2^-13
    }
    code[i] = to_fp4x4(q[0].x, q[0].y, q[1].x, q[1].y);
  }
  if (top >= 0x7f80u) {
    scale = 0x7fu;
    return make_uint2(0u, 0u);
  }
  return make_uint2(plain_zeros(code[0] | code[1] << 16), plain_zeros(code[2] | code[3] << 16));
}

// Eight codes (a word) times their scale, as bf16.
__device__ __forceinline__ uint4 values8(uint32_t w, float s) {
  uint32_t h[4], o[4];
  fp4x8_to_f16(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f16x2_to_f32(h[i], lo, hi);
    o[i] = pack_bf16x2(lo * s, hi * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  float s, none;
  f16x2_to_f32(e4m3x2_to_f16(byte), s, none);
  return s;
}

}  // namespace

// A group of D / 16 lanes takes kAppendRun heads of a token, a lane 16 features (one
// scale); the groups of a warp take consecutive tokens, so that four of them fill a
// 32-byte piece of each strip.
template <int D>
__global__ void __launch_bounds__(kF4Threads) fp4_append_kernel(const Fp4CacheParams p) {
  constexpr int LG = D / 16;
  constexpr int kTokens = kF4Threads / LG;  // of a CTA
  const int lane = threadIdx.x & 31;
  const int c = lane % LG;
  const long long t = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x / LG;
  const bool live = t < p.total_tokens;
  const int token = live ? static_cast<int>(t) : 0;
  const int h0 = static_cast<int>(blockIdx.y) * kAppendRun;
  const int heads = live ? min(h0 + kAppendRun, p.kv_heads) : 0;
  uint4 x[2][kAppendRun][2];
#pragma unroll
  for (int i = 0; i < kAppendRun; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (h0 + i < heads) {
        const uint4* src = reinterpret_cast<const uint4*>(
            (w ? p.v + token * p.v_stride : p.k + token * p.k_stride) + (h0 + i) * D + c * 16);
        x[w][i][0] = __ldg(src);
        x[w][i][1] = __ldg(src + 1);
      }
  const Fp4Place at = find_place<LG>(p, Fp4<D>::kTileBytes, live, token, c, lane);
  if (at.at < 0) {
    if (live && !at.behind && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArgF);
    return;
  }
  const long long block = (1ll << p.page_shift) / kFp4Tile * Fp4<D>::kTileBytes;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint8_t* cache = (w ? p.v_cache : p.k_cache) + at.at;
#pragma unroll
    for (int i = 0; i < kAppendRun; ++i) {
      if (h0 + i >= heads) break;
      uint32_t scale;
      const uint2 code = quantise16(x[w][i][0], x[w][i][1], w ? p.v_scale : p.k_scale, scale);
      uint8_t* tile = cache + (h0 + i) * block;
      *reinterpret_cast<uint2*>(tile + Fp4<D>::place(c, at.row >> 1) + (at.row & 1) * 8) = code;
      tile[Fp4<D>::kScales + c * kFp4Tile + at.row] = static_cast<uint8_t>(scale);
    }
  }
}

// D / 8 lanes write a row, 16 bytes each; they take kGatherRun heads of a token, and a
// CTA consecutive tokens, whose codes lie in the same 32-byte pieces.
template <int D>
__global__ void __launch_bounds__(kF4Threads) fp4_gather_kernel(const Fp4CacheParams p) {
  constexpr int LG = D / 8;
  constexpr int kTokens = kF4Threads / LG;
  const int lane = threadIdx.x & 31;
  const int c = lane % LG, j = c >> 1;
  const long long t = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x / LG;
  const bool live = t < p.total_tokens;
  const int token = live ? static_cast<int>(t) : 0;
  const int h0 = static_cast<int>(blockIdx.y) * kGatherRun;
  const int heads = min(h0 + kGatherRun, p.kv_heads);
  const Fp4Place at = find_place<LG>(p, Fp4<D>::kTileBytes, live, token, c, lane);
  if (at.at < 0) {
    if (live && !at.behind && p.status != nullptr && c == 0) atomicCAS(p.status, 0, kErrArgF);
    return;
  }
  const long long block = (1ll << p.page_shift) / kFp4Tile * Fp4<D>::kTileBytes;
  const int code_at = Fp4<D>::place(j, at.row >> 1) + (at.row & 1) * 8 + (c & 1) * 4;
  const int scale_at = Fp4<D>::kScales + j * kFp4Tile + at.row;
  uint32_t code[2][kGatherRun], scale[2][kGatherRun];
#pragma unroll
  for (int i = 0; i < kGatherRun; ++i)
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (h0 + i < heads) {
        const uint8_t* tile = (w ? p.v_cache : p.k_cache) + at.at + (h0 + i) * block;
        code[w][i] = __ldg(reinterpret_cast<const uint32_t*>(tile + code_at));
        scale[w][i] = __ldg(tile + scale_at);
      }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    __nv_bfloat16* out =
        w ? p.v_out + token * p.v_stride : p.k_out + token * p.k_stride;
#pragma unroll
    for (int i = 0; i < kGatherRun; ++i)
      if (h0 + i < heads)
        *reinterpret_cast<uint4*>(out + (h0 + i) * D + c * 8) =
            values8(code[w][i], e4m3_value(scale[w][i]) * (w ? p.v_scale : p.k_scale));
  }
}

// Caches [0, kv_len) of every sequence with new tokens to 16-bit pages of 128 tokens, page
// i of sequence b at b * out_pages + i, with the table that says so.  A CTA has a KV head
// and every gridDim.x-th of the pages that there are (the bounds may be far above the
// lengths), a warp a tile of it.  Keys in bf16, values in fp16, both exactly and without
// the caches' powers of two: the softmax scale has the keys', the join of O the values'.
// Every warp goes through all sequences for its pages, about 0.5 us a sequence with 64 warps
// on an SM: what bounds it where there are many short caches (8 heads of 128: 1,025 caches of
// 20 to 79 keys 502 us, their bytes' floor 39; 257 of 100 to 399 149 us, floor 50), and
// beside the bytes where they are long (65 of 4,000 to 6,400: 290 us, floor 261).
template <int D>
__global__ void __launch_bounds__(kF4Threads) fp4_pages_kernel(const Fp4PagesParams p) {
  constexpr int LG = D / 8;
  constexpr int kRows = 32 / LG;  // rows of a warp's step
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % LG, j = c >> 1;
  const int h = static_cast<int>(blockIdx.y), step = static_cast<int>(gridDim.x);
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  const long long block = (1ll << p.page_shift) / kFp4Tile * Fp4<D>::kTileBytes;
  bool bad = false;
  int first = static_cast<int>(blockIdx.x);  // of this CTA's pages of sequence b
  int kv_next = __ldg(p.kv_lens), lo_next = __ldg(p.cu_seqlens), hi_next = __ldg(p.cu_seqlens + 1);
  for (int b = 0; b < p.num_seqs; ++b) {
    const int kv = kv_next, lo = lo_next, hi = hi_next;
    if (b + 1 < p.num_seqs) {
      kv_next = __ldg(p.kv_lens + b + 1);
      lo_next = hi;
      hi_next = __ldg(p.cu_seqlens + b + 2);
    }
    // A sequence without new tokens is not read.  (The schedule kernel reports lengths
    // that are not valid.)
    const bool valid = hi > lo && kv >= 0 && kv <= p.max_kv_len && kv <= cap;
    const int n_pages = valid ? (kv + kFp4OutPage - 1) / kFp4OutPage : 0;
    const int* pages = p.page_table + static_cast<size_t>(b) * p.max_pages;
    int pg = first;
    for (; pg < n_pages; pg += step) {
      const long long to = static_cast<long long>(b) * p.out_pages + pg;
      if (h == 0 && threadIdx.x == 0) p.out_table[to] = static_cast<int>(to);
      const int key0 = pg * kFp4OutPage + warp * kFp4Tile;
      if (key0 >= kv) continue;
      const int page = __ldg(pages + (key0 >> p.page_shift));
      const bool gone = page < 0 || page >= p.num_pages;
      bad = bad || gone;
      const long long at = static_cast<long long>(gone ? 0 : page) * p.page_stride + h * block +
                           ((key0 & ((1 << p.page_shift) - 1)) / kFp4Tile) * Fp4<D>::kTileBytes;
      const int n = min(kv - key0, kFp4Tile);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint8_t* tile = (w ? p.v_cache : p.k_cache) + at;
        uint16_t* out = (w ? p.v_out : reinterpret_cast<uint16_t*>(p.k_out)) +
                        ((to * kFp4OutPage + warp * kFp4Tile) * p.kv_heads + h) * D + c * 8;
        uint32_t code[kFp4Tile / kRows], scale[kFp4Tile / kRows];
#pragma unroll
        for (int i = 0; i < kFp4Tile / kRows; ++i) {
          const int r = i * kRows + lane / LG;
          code[i] = __ldg(reinterpret_cast<const uint32_t*>(
              tile + Fp4<D>::place(j, r >> 1) + (r & 1) * 8 + (c & 1) * 4));
          scale[i] = __ldg(tile + Fp4<D>::kScales + j * kFp4Tile + r);
        }
#pragma unroll
        for (int i = 0; i < kFp4Tile / kRows; ++i) {
          const int r = i * kRows + lane / LG;
          uint4 v;
          if (w) {
            const uint32_t s = __byte_perm(e4m3x2_to_f16(scale[i]), 0, 0x1010);
            uint32_t x[4];
            fp4x8_to_f16(code[i], x);
            v = make_uint4(mul_f16x2(x[0], s), mul_f16x2(x[1], s), mul_f16x2(x[2], s),
                           mul_f16x2(x[3], s));
          } else {
            v = values8(code[i], e4m3_value(scale[i]));
          }
          if (r < n)
            *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * p.kv_heads * D) =
                gone ? make_uint4(0u, 0u, 0u, 0u) : v;
        }
      }
    }
    first = pg - n_pages;  // the pages of all sequences are dealt out in turn
  }
  // The schedule before this clears the error word.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad && lane == 0) atomicCAS(&p.hdr->error, 0, kPagedBad);
}

static dim3 fp4_grid(const Fp4CacheParams& p, int lanes, int run) {
  const long long tokens = kF4Threads / lanes;
  return dim3(static_cast<unsigned>((p.total_tokens + tokens - 1) / tokens),
              static_cast<unsigned>((p.kv_heads + run - 1) / run));
}

cudaError_t launch_fp4_append(const Fp4CacheParams& p, int D, cudaStream_t stream) {
  const dim3 grid = fp4_grid(p, D / 16, kAppendRun);
  if (D == 64) fp4_append_kernel<64><<<grid, kF4Threads, 0, stream>>>(p);
  else fp4_append_kernel<128><<<grid, kF4Threads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fp4_gather(const Fp4CacheParams& p, int D, cudaStream_t stream) {
  const dim3 grid = fp4_grid(p, D / 8, kGatherRun);
  if (D == 64) fp4_gather_kernel<64><<<grid, kF4Threads, 0, stream>>>(p);
  else fp4_gather_kernel<128><<<grid, kF4Threads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fp4_pages(const Fp4PagesParams& p, int D, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  // Two rounds of CTAs over all heads, and no more than there can be pages.
  const long long pages = static_cast<long long>(p.num_seqs) * p.out_pages;
  const long long share = (num_sms * kPagesCtas + p.kv_heads - 1) / p.kv_heads;
  cfg.gridDim = dim3(static_cast<unsigned>(pages < share ? pages : share),
                     static_cast<unsigned>(p.kv_heads));
  cfg.blockDim = dim3(kF4Threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return D == 64 ? cudaLaunchKernelEx(&cfg, fp4_pages_kernel<64>, p)
                 : cudaLaunchKernelEx(&cfg, fp4_pages_kernel<128>, p);
}

}  // namespace cpattn
