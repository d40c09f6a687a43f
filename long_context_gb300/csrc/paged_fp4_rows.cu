// Attention of few rows over a paged KV cache in 4 bits (fp4.cuh): one token a
// sequence, or a few, for every query head that shares a KV head.
//
// A CTA of 4 warps has one block of 8, 16 or 32 rows of one KV head and one split of the
// keys, and each warp takes every fourth step of the split on its own, with its own
// ring of stages, its own softmax state and no barrier until the states are joined
// (as for the bf16 cache, paged_rows.cu).  What differs is what bounds it: a key and its
// value are 9 D / 8 bytes instead of 4 D, so at the copy bandwidth an SM has 98 cycles
// for a tile of 16 keys of 128 features and their values, in which 4,096 codes become
// fp16 operands.  Measured rates of an SM, a cycle: 64 conversions of two codes, as many packed
// multiplications, permutations or logic operations, and 0.57 matrix instructions.  So:
// * keys and values are the left operand of 16 x 8 x 16 matrix instructions, whose
//   16 rows they fill, and the queries are the right one: 8 rows cost 8 instructions
//   for a tile's scores, not 16;
// * scores come out as [keys, rows]; the matrix transpose that P needs between the
//   products is one instruction for 8 x 8;
// * a byte of codes (features 2 i and 2 i + 1 of one key) is a pair of fp16 as it comes
//   out of one conversion, and keys take it as it is.  The values' operand has pairs of
//   keys: the halves of two keys' words are exchanged before the conversion, 16
//   operations a tile and lane (permutations behind it, 32; without them, the other
//   feature's column of P zero and twice the products: a token each of 64 caches, 32 / 8
//   heads of 128, 247 instead of 238 us);
// * codes times scales are exact in fp16, the queries (each row times a power of two,
//   which the score's factor takes back) too; P is rounded to fp16 (2^-11);
// * K and V come by bulk copies, one a page and operand, a few lanes issuing them;
// * a step is 64 keys of 128 features and its scores are taken together: with 32 at a
//   time, and four CTAs of an SM instead of three, 277 instead of 247 us.
// That case is at 5.9 TB/s (1.40 GB in 238 us; the same copies without the arithmetic
// take 214): 242 instructions a tile and warp at half of the issue rate, by latencies of
// the chain copy, conversion, scores, exponentials, P V in 12 warps of 150 registers.
// With 32 rows the products are four times as many (17 caches of up to 20,000 keys, 4
// KV heads of 64, 25 rows: 37 us, 9 of them the products' and their operands'); their
// queries are in shared memory (in registers, which spilled, 72 instead of 62 us for
// 32 rows over 17 caches of 128 features, now 56).
//
// Softmax: p = 2^(s scale log2 e - m + 11) with a running reference m per row.  It is
// the largest score of the first keys and moves to a new largest only when a lane's sum
// of a pass would leave fp16's range, so p is below 2^15 and the largest weight's at
// least 2^11: fp16 keeps its 11 bits of weights down to 2^-25 of the largest.  O and l
// share the reference, so O / l and m + ln l do not depend on it.  l sums p in fp32.
//
// The splits come from the schedule kernel's list, from the lengths in every warp
// (paged_plan.cuh), or, where sequences are short, are equal parts of a sequence that a
// cluster of CTAs takes, whose states meet through distributed shared memory.
#include <cuda_bf16.h>

#include <type_traits>

#include "fp4.cuh"
#include "kernels.h"
#include "paged_plan.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

constexpr int kF4Warps = 4;
constexpr int kF4RowsThreads = kF4Warps * 32;
constexpr float kNegInfF = -__builtin_huge_valf();
constexpr float kLn2F = 0.69314718055994530942f;
constexpr float kLog2eF = 1.44269504088896340736f;
constexpr float kLiftF = 11.f;       // powers of two of a weight at the reference
constexpr float kMaxSumF = 32768.f;  // of a lane's weights of a row in one pass

constexpr int kF4MaxParts = 8;       // CTAs of a portable cluster

// Where a CTA's work comes from.
enum class Fp4Work {
  kList,   // the schedule kernel's list
  kPlan,   // worked out by every warp (paged_plan.cuh)
  kStatic  // a cluster of CTAs has one sequence and KV head, in equal parts
};

template <int D, int NT>
struct Fp4RowsCfg {
  static constexpr int kTiles = (NT == 1 ? 4 : 2) * (128 / D);  // tiles of a step
  static constexpr int kKeys = kTiles * kFp4Tile;
  static constexpr int kHalf = kTiles * Fp4<D>::kTileBytes;  // K (or V) of a step
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kRing = kF4Warps * kStages * kStage;  // 74 or 55 KB
  static constexpr int kRows = 8 * NT;
  static constexpr int kJoin = kF4Warps * kRows * D * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  static constexpr int kPass = NT == 1 ? 4 : 2;  // tiles whose scores are taken together
  static constexpr int kCtas = NT == 4 ? 2 : 3;  // of an SM
};

// The low halves of lo's bytes and the high halves of hi's.
__device__ __forceinline__ uint32_t halves(uint32_t lo, uint32_t hi) {
  return (lo & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u);
}

__device__ __forceinline__ void sts128_zero(uint32_t a) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
}

}  // namespace

template <int D, int NT, Fp4Work W>
__global__ void __launch_bounds__(kF4RowsThreads, Fp4RowsCfg<D, NT>::kCtas)
    fp4_rows_kernel(const Fp4RowsParams fp) {
  using C = Fp4RowsCfg<D, NT>;
  constexpr bool kPlan = W == Fp4Work::kPlan;
  constexpr bool kStatic = W == Fp4Work::kStatic;
  using F = Fp4<D>;
  const PagedParams& p = fp.p;
  constexpr int kRows = C::kRows;
  constexpr bool kMany = NT > 1;    // the queries are in shared memory
  constexpr int kM = D / 16;        // products of a tile's scores
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kF4Warps][kRows], s_l[kF4Warps][kRows];
  __shared__ __align__(8) uint64_t s_full[kF4Warps][C::kStages];
  __shared__ float s_back[kRows];
  __shared__ int s_lim[kRows];
  __shared__ uint4 s_q[kMany ? NT * (kM / 2) * 32 : 1];
  __shared__ int s_last, s_abort, s_bad;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int Hk = p.num_kv_heads, G = p.group;
  const int rank = kStatic ? static_cast<int>(blockIdx.x) % fp.parts : 0;
  const int eh = kStatic ? static_cast<int>(blockIdx.x) / fp.parts : static_cast<int>(blockIdx.x);
  const int e = eh / Hk;
  const int h = eh - e * Hk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  PagedWork w;
  if (kStatic) {
    // Every CTA checks all lengths (as the schedule kernels do) and takes its own.
    w.seq = e;
    w.tok0 = __ldg(p.cu_seqlens + e);
    w.q_len = __ldg(p.cu_seqlens + e + 1) - w.tok0;
    w.kv_len = __ldg(p.kv_lens + e);
    bool bad = false;
    const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
    for (int b = threadIdx.x; b < p.num_seqs; b += kF4RowsThreads) {
      const int lo = __ldg(p.cu_seqlens + b), hi = __ldg(p.cu_seqlens + b + 1);
      const int kv = __ldg(p.kv_lens + b);
      bad = bad || lo < 0 || hi < lo || hi > p.total_q || hi - lo > p.max_seqlen || kv < 0 ||
            kv > p.max_kv_len || kv > cap || (b == 0 && lo != 0);
    }
    bad = __syncthreads_or(bad);
    if (bad || w.q_len == 0) {
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (bad) p.hdr->error = kPagedBad;
      }
      return;
    }
    const int units = (w.kv_len + p.shape.unit - 1) / p.shape.unit;
    const int per = (units + fp.parts - 1) / fp.parts * p.shape.unit;
    w.blk = 0;
    w.kv_lo = min(rank * per, w.kv_len);
    w.kv_hi = min(w.kv_lo + per, w.kv_len);
    w.slot = -1;
  } else if (kPlan) {
    const PagedPlan plan = make_plan(p, lane);
    if (e >= plan.splits) return;
    w = plan_split(p, plan, e);
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n_work = __ldcg(&p.hdr->n_items);
    const int err0 = __ldcg(&p.hdr->error);
    const int4* wp = reinterpret_cast<const int4*>(p.work + e);
    const int4 w0 = __ldcg(wp), w1 = __ldcg(wp + 1), w2 = __ldcg(wp + 2);
    if (e >= n_work) return;
    if (__syncthreads_or(says_timeout(err0))) return;
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

  // Steps of this warp: keys [kv_lo + (warp + 4 i) span, + span), the span a step's
  // kKeys or, in a short split, less, so that all warps have some.
  int span = C::kKeys;
  while (span > kFp4Tile && kv_hi - kv_lo <= span * kF4Warps / 2) span /= 2;
  const int all_steps = (kv_hi - kv_lo + span - 1) / span;
  const int steps = all_steps > warp ? (all_steps - warp + kF4Warps - 1) / kF4Warps : 0;
  const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);
  uint64_t* full = s_full[warp];
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) mbar_init(full + i, 1);
    fence_mbarrier_init();
  }
  if (threadIdx.x == 0) s_abort = s_bad = 0;
  __syncthreads();
  // A step's tiles come in runs that share a page; lane 2 r copies run r of K, lane
  // 2 r + 1 of V.  Its page number is read a step ahead.
  const int page_tiles = 1 << (p.page_shift - 4);
  // (Aligned as the split's first key is, so that no run crosses a page's end: a step may
  // have 128 keys, and a split starts at a multiple of 64.)
  const int aligned = kv_lo > 0 ? max((kv_lo & -kv_lo) / kFp4Tile, 1) : page_tiles;
  const int run_tiles = min(min(span / kFp4Tile, page_tiles), aligned);
  const int run_at = (lane >> 1) * run_tiles;
  const int copy_end = run_at * kFp4Tile < span ? kv_hi : 0;
  const int* pages = p.page_table + static_cast<size_t>(seq) * p.max_pages;
  const uint8_t* cache = ((lane & 1) ? fp.v_cache : fp.k_cache) +
                         static_cast<size_t>(h) * page_tiles * F::kTileBytes;
  int copy_key = kv_lo + warp * span + run_at * kFp4Tile;  // of the next copy
  uint32_t copy_to = ring + (lane & 1) * C::kHalf + run_at * F::kTileBytes;
  uint32_t copy_bar = smem_u32(full);
  const uint32_t page_units = fp.page_units;
  int copy_left = steps;
  int next_page = copy_key < copy_end ? __ldg(pages + (copy_key >> p.page_shift)) : 0;
  bool bad_page = false;
  auto copy = [&]() {
    if (copy_left <= 0) return;
    --copy_left;
    const int page = next_page, key = copy_key;
    copy_key += kF4Warps * span;
    if (copy_key < copy_end) next_page = __ldg(pages + (copy_key >> p.page_shift));
#ifdef CPATTN_FAULT_INJECT_DROP_P
    const bool drop = blockIdx.x == 0 && warp == 0 && copy_left == steps - 1;
#else
    constexpr bool drop = false;
#endif
    if (key < copy_end) {
      const int n = min(run_tiles, (copy_end - key + kFp4Tile - 1) / kFp4Tile);
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
        const unsigned at = (key >> 4) & (page_tiles - 1);
        const uint32_t bytes = n * F::kTileBytes;
        mbar_expect_tx(copy_bar, bytes);
        if (!drop)
          bulk_load(copy_to,
                    cache + (static_cast<uint64_t>(static_cast<unsigned>(page)) * page_units +
                             at * (F::kTileBytes / 16)) * 16,
                    bytes, copy_bar);
      } else {
        // Its keys or values count as zeros: their scales are.
        bad_page = true;
        for (int x = 0; x < n; ++x)
          for (int y = 0; y < D; y += 16)
            sts128_zero(copy_to + x * F::kTileBytes + F::kScales + y);
        fence_proxy_async_smem();
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_at(copy_bar);
    const bool wrap = copy_bar == smem_u32(full + C::kStages - 1);
    copy_to += wrap ? (1 - C::kStages) * C::kStage : C::kStage;
    copy_bar += wrap ? (1 - C::kStages) * 8 : 8;
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) copy();

  // The queries as right operands: lane (g, t) has row g of each block of eight,
  // features [t D / 4, + D / 4), as fp16 times a power of two that brings the row's
  // largest below 2^15.  With more than one block each warp makes one, and all read
  // them from shared memory.
  uint32_t q[kM][2];
  float2 sc[NT];    // from a score to the exponent, rows 2 t and 2 t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (kMany && warp != nt) continue;
    const int row = row0 + nt * 8 + g;
    const bool in = row >= 0;
    const int tok = in ? row / G : 0;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + (static_cast<size_t>(tok0 + tok) * p.num_heads + h * G + (in ? row - tok * G : 0)) * D +
        t * (D / 4));
    uint32_t x[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, x[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(14 - exponent of the largest); its inverse is a normal number too.
    const int up = min(252, 268 - static_cast<int>(top >> 7));
    const float f = __uint_as_float(static_cast<uint32_t>(up) << 23);
    const float back = __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        q[m][i] = pack_f16x2(__uint_as_float(x[2 * m + i] << 16) * f,
                                 __uint_as_float(x[2 * m + i] & 0xffff0000u) * f);
    if (kMany) {
#pragma unroll
      for (int m = 0; m < kM; m += 2)
        s_q[(nt * (kM / 2) + m / 2) * 32 + lane] =
            make_uint4(q[m][0], q[m][1], q[m + 1][0], q[m + 1][1]);
    }
    if (t == 0) {
      s_back[nt * 8 + g] = back;
      // Keys below it are visible.
      s_lim[nt * 8 + g] = p.causal && in ? kv_len - q_len + tok + 1 : kv_len;
    }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // A normal number: masked scores (-inf) and zeros are multiplied by it.
      (i ? sc[nt].y : sc[nt].x) =
          fminf(fmaxf(s_back[nt * 8 + 2 * t + i] * p.scale_log2, 1.17549435e-38f), 3.40282347e38f);
    }
  }
  // Steps ending at or below this key need no mask (rows are in order, so the block's
  // first row sees the fewest keys; what rows that are not there see does not matter).
  const int free_end = p.causal ? kv_len - q_len + max(row0, 0) / G + 1 : kv_len;

  // Lane (g, t) accumulates rows 2 t and 2 t + 1 of features g D / 8 + 2 i and + 1, i
  // below D / 16: [i][feature][row].
  float o[NT][D / 16][4];
  float m[NT][2];          // the references
  float2 off[NT], l[NT];   // 11 - m (11 without a reference) and the sums, by rows
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = kNegInfF;
    off[nt] = make_float2(kLiftF, kLiftF);
    l[nt] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[nt][i][x] = 0.f;
  }
  bool fresh = true;  // some row has no reference yet

  bool failed = false;
  int step = 0, st = 0, key0 = kv_lo + warp * span;
  uint32_t parity = 0;
  const int k_at = t * (D / 64);           // first group of this lane's keys
  const int v_at = D == 128 ? g : g >> 1;  // group of its values
  // One step.  kWhole: all of its keys are there and every row sees them.
  auto take = [&](auto whole, const uint8_t* stage, int left) {
    constexpr bool kWhole = decltype(whole)::value;
#pragma unroll(NT == 4 ? 1 : 4)
    for (int pass = 0; pass < C::kTiles; pass += C::kPass) {
      if (!kWhole && pass > 0 && pass * kFp4Tile >= left) break;
      float s[C::kPass][NT][4];
      // (A tile behind the split's end holds what an earlier step left.)
      // Rows of the left operand: token 2 g, and 2 g + 1 as row g + 8.
#pragma unroll
      for (int gg = 0; gg < D / 64; ++gg) {
        const int j = k_at + gg;
        uint4 k4[C::kPass];
        uint32_t s0[C::kPass], s1[C::kPass];
#pragma unroll
        for (int u = 0; u < C::kPass; ++u) {
          const uint8_t* tile = stage + (pass + u) * F::kTileBytes;
          k4[u] = *reinterpret_cast<const uint4*>(tile + F::place(j, g));
          const uint32_t both = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(
              tile + F::kScales + j * kFp4Tile + 2 * g));
          s0[u] = __byte_perm(both, 0, 0x1010);
          s1[u] = __byte_perm(both, 0, 0x3232);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int mm = gg * 4 + half * 2;
          uint4 qs[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            qs[nt] = kMany ? s_q[(nt * (kM / 2) + mm / 2) * 32 + lane]
                           : make_uint4(q[mm][0], q[mm][1], q[mm + 1][0], q[mm + 1][1]);
#pragma unroll
          for (int u = 0; u < C::kPass; ++u) {
            uint32_t a[4], b[4];
            fp4x8_to_f16(half ? k4[u].y : k4[u].x, a);
            fp4x8_to_f16(half ? k4[u].w : k4[u].z, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = mul_f16x2(a[i], s0[u]);
              b[i] = mul_f16x2(b[i], s1[u]);
            }
            const uint32_t op0[4] = {a[0], b[0], a[1], b[1]}, op1[4] = {a[2], b[2], a[3], b[3]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (mm == 0) mma_16816_f16_first(s[u][nt], op0, qs[nt].x, qs[nt].y);
              else mma_16816_f16(s[u][nt], op0, qs[nt].x, qs[nt].y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816_f16(s[u][nt], op1, qs[nt].z, qs[nt].w);
          }
        }
      }
      const int pass_end = (pass + C::kPass) * kFp4Tile;
      if (!kWhole && (key0 + pass_end > free_end || pass_end > left)) {
#pragma unroll
        for (int u = 0; u < C::kPass; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = key0 + (pass + u) * kFp4Tile + 2 * g + (x >> 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (key >= s_lim[nt * 8 + 2 * t + (x & 1)] || key >= key0 + left) s[u][nt][x] = kNegInfF;
          }
      }
      // The exponentials against the references as they are; again, against new ones,
      // if a lane's sum leaves fp16's range or a row has none yet.
      float2 e2[C::kPass][NT][2], sum[NT];
      auto exponentials = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sum[nt] = make_float2(0.f, 0.f);
#pragma unroll
          for (int u = 0; u < C::kPass; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float2 x = __ffma2_rn(make_float2(s[u][nt][2 * y], s[u][nt][2 * y + 1]), sc[nt],
                                          off[nt]);
              e2[u][nt][y] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              sum[nt] = __fadd2_rn(sum[nt], e2[u][nt][y]);
            }
        }
      };
#pragma unroll 1
      for (int round = 0;; ++round) {
        exponentials();
        if (round > 0) break;
        bool move = fresh;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          move = move || !(sum[nt].x <= kMaxSumF) || !(sum[nt].y <= kMaxSumF);
        if (!__any_sync(0xffffffffu, move)) break;
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = kNegInfF;
#pragma unroll
            for (int u = 0; u < C::kPass; ++u) v = fmax3(v, s[u][nt][i], s[u][nt][i + 2]);
            v *= i ? sc[nt].y : sc[nt].x;
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float mn = fmaxf(m[nt][i], v);
            const float alpha = m[nt][i] == kNegInfF ? 0.f : ex2_approx(m[nt][i] - mn);
            m[nt][i] = mn;
            const float to = mn == kNegInfF ? kLiftF : kLiftF - mn;
            if (i) off[nt].y = to;
            else off[nt].x = to;
            if (i) l[nt].y *= alpha;
            else l[nt].x *= alpha;
            fresh = fresh || mn == kNegInfF;
#pragma unroll
            for (int f = 0; f < D / 16; ++f) {
              o[nt][f][i] *= alpha;
              o[nt][f][i + 2] *= alpha;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) l[nt] = __fadd2_rn(l[nt], sum[nt]);
#pragma unroll
      for (int u = 0; u < C::kPass; ++u) {
        if (!kWhole && u > 0 && (pass + u) * kFp4Tile >= left) break;
        // P of this lane's row g: pa tokens 4 t and 4 t + 2, pb 4 t + 1 and 4 t + 3.
        uint32_t pa[NT], pb[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pa[nt] = transpose_8x8(pack_f16x2(e2[u][nt][0].x, e2[u][nt][0].y));
          pb[nt] = transpose_8x8(pack_f16x2(e2[u][nt][1].x, e2[u][nt][1].y));
        }
        const uint8_t* tile = stage + C::kHalf + (pass + u) * F::kTileBytes;
        const uint4 v01 = *reinterpret_cast<const uint4*>(tile + F::place(v_at, 2 * t));
        const uint4 v23 = *reinterpret_cast<const uint4*>(tile + F::place(v_at, 2 * t + 1));
        uint32_t sb =
            *reinterpret_cast<const uint32_t*>(tile + F::kScales + v_at * kFp4Tile + 4 * t);
        // What lies behind the cache's end has weight 0, and a NaN there is one.
        if (!kWhole && left < (pass + u + 1) * kFp4Tile) {
          const int n = kv_len - (key0 + (pass + u) * kFp4Tile) - 4 * t;
          sb = n <= 0 ? 0u : (n >= 4 ? sb : sb & ((1u << (8 * n)) - 1u));
        }
        sb = __byte_perm(sb, 0, 0x3120);
        const uint32_t s02 = e4m3x2_to_f16(sb), s13 = e4m3x2_to_f16(sb >> 16);
        // Words of the four tokens, eight features each.
        constexpr int kW = D / 64;
        uint32_t wd[4][kW];
        if (D == 128) {
          wd[0][0] = v01.x;
          wd[0][kW - 1] = v01.y;
          wd[1][0] = v01.z;
          wd[1][kW - 1] = v01.w;
          wd[2][0] = v23.x;
          wd[2][kW - 1] = v23.y;
          wd[3][0] = v23.z;
          wd[3][kW - 1] = v23.w;
        } else {
          const bool hi = g & 1;
          wd[0][0] = hi ? v01.y : v01.x;
          wd[1][0] = hi ? v01.w : v01.z;
          wd[2][0] = hi ? v23.y : v23.x;
          wd[3][0] = hi ? v23.w : v23.z;
        }
#pragma unroll
        for (int k = 0; k < kW; ++k) {
          uint32_t x[2][2][4];  // tokens (0, 2) or (1, 3), even or odd feature
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            fp4x8_to_f16(halves(wd[z][k], wd[z + 2][k] << 4), x[z][0]);
            fp4x8_to_f16(halves(wd[z][k] >> 4, wd[z + 2][k]), x[z][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t op[4] = {mul_f16x2(x[0][0][i], s02), mul_f16x2(x[0][1][i], s02),
                                    mul_f16x2(x[1][0][i], s13), mul_f16x2(x[1][1][i], s13)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][k * 4 + i], op, pa[nt], pb[nt]);
          }
        }
      }
    }
  };

#pragma unroll 1
  for (; step < steps; ++step) {
    if (!__all_sync(0xffffffffu, mbar_try_wait_sleep(full + st, parity, kWaitSleepNs)) &&
        __any_sync(0xffffffffu, !wait_bounded(full + st, parity, &s_abort))) {
      failed = true;
      break;
    }
    copy();
    const uint8_t* stage = smem + warp * (C::kStages * C::kStage) + st * C::kStage;
    const int left = min(kv_hi - key0, span);  // keys of the step
    if (key0 + C::kKeys <= free_end && left >= C::kKeys) take(std::true_type(), stage, left);
    else take(std::false_type(), stage, left);
    key0 += kF4Warps * span;
    st = st + 1 == C::kStages ? 0 : st + 1;
    parity ^= st == 0;
    __syncwarp();  // the stage may be filled again
  }
  if (failed) {
    s_abort = 1;
    // Copies in flight still write to this CTA's memory.
    for (int i = step; i < min(steps, step + C::kStages - 1); ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(full + st, parity) && global_timer_ns() - t0 < 200000000ull) {
      }
      st = st + 1 == C::kStages ? 0 : st + 1;
      parity ^= st == 0;
    }
  }

  // Join the warps' states (their rings are done with) and write the rows.
  if (bad_page) s_bad = 1;
  __syncthreads();
  const int error = s_abort ? kPagedLate : (s_bad ? kPagedBad : 0);
  if (!kStatic && threadIdx.x == 0) {
    if (kPlan) p.cta_error[blockIdx.x] = error;
    else if (error) atomicCAS(&p.hdr->error, 0, error);
  }
  float* so = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = nt * 8 + 2 * t + i;
      float sum = i ? l[nt].y : l[nt].x;
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (g == 0) {
        s_m[warp][r] = m[nt][i] - kLiftF;
        s_l[warp][r] = sum;
      }
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
        *reinterpret_cast<float2*>(so + r * D + g * (D / 8) + 2 * f) =
            make_float2(o[nt][f][i], o[nt][f][i + 2]);
    }
  __syncthreads();
  // One row's four features from c on, joined: to the output (to < 0) or to the partial
  // results of `to`, a slot.
  auto put = [&](int to, int r, int c, const float4& acc, float top, float den, float unit) {
    const float inv = den == 0.f ? 0.f : unit / den;
    const float lse = den == 0.f ? kNegInfF : (top + __log2f(den)) * kLn2F;
    const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (to >= 0) {
      const size_t part = (static_cast<size_t>(to) * Hk + h) * kRows + r;
      *reinterpret_cast<float4*>(p.o_part + part * D + c) = v;
      if (c == 0) p.lse_part[part] = lse;
    } else {
      const int row = row0 + r, tok = row / G;
      const size_t at_row = static_cast<size_t>(tok0 + tok) * p.num_heads + h * G + (row - tok * G);
      *reinterpret_cast<uint2*>(p.out + at_row * D + c) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      if (c == 0 && p.lse != nullptr) p.lse[at_row] = lse;
    }
  };
  // A state joins with 2^(its reference - the largest).  One without a visible key has
  // l = 0 and O = 0 (or NaN in both, which the row then shows).
  auto weight = [](float ref, float top) { return ref == kNegInfF ? 1.f : ex2_approx(ref - top); };
  auto add = [](float4& acc, float f, const float4& v) {
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  };
  // Joins this CTA's warps' states, times `unit`.
  auto join = [&](int to, float unit) {
    const float* all = reinterpret_cast<const float*>(smem);
    for (int x = threadIdx.x; x < kRows * (D / 4); x += kF4RowsThreads) {
      const int r = x / (D / 4), c = (x % (D / 4)) * 4;
      if (row0 + r < 0) continue;
      float top = kNegInfF;
#pragma unroll
      for (int v = 0; v < kF4Warps; ++v) top = fmaxf(top, s_m[v][r]);
      float den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kF4Warps; ++v) {
        const float f = weight(s_m[v][r], top);
        den = fmaf(f, s_l[v][r], den);
        add(acc, f, *reinterpret_cast<const float4*>(all + (v * kRows + r) * D + c));
      }
      put(to, r, c, acc, top, den, unit);
    }
  };
  if (kStatic) {
    if (fp.parts == 1) {
      join(-1, fp.v_scale);
    } else {
      // Each CTA of the cluster joins its share of the rows' features over all warps of
      // all CTAs, four lanes to four features, a warp's state of every CTA each.
      cluster_sync();
      const int share = (kRows * (D / 4) + fp.parts - 1) / fp.parts;
      const int end = min(kRows * (D / 4), (rank + 1) * share);
      const int v = threadIdx.x & 3;
      const uint32_t at_m = smem_u32(&s_m[v][0]), at_l = smem_u32(&s_l[v][0]);
      const uint32_t at_o = smem_u32(smem) + v * kRows * D * 4;
      for (int x0 = rank * share; x0 < end; x0 += kF4RowsThreads / 4) {
        const int x = x0 + (threadIdx.x >> 2);
        const int r = min(x, end - 1) / (D / 4), c = (min(x, end - 1) % (D / 4)) * 4;
        float ref[kF4MaxParts], top = kNegInfF;
#pragma unroll
        for (int i = 0; i < kF4MaxParts; ++i) {
          ref[i] = i < fp.parts ? ld_cluster(at_m + r * 4, i) : kNegInfF;
          top = fmaxf(top, ref[i]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kF4MaxParts; ++i)
          if (i < fp.parts) {
            const float f = weight(ref[i], top);
            den = fmaf(f, ld_cluster(at_l + r * 4, i), den);
            add(acc, f, ld_cluster4(at_o + (r * D + c) * 4, i));
          }
#pragma unroll
        for (int z = 1; z < 4; z <<= 1) {
          den += __shfl_xor_sync(0xffffffffu, den, z);
          acc.x += __shfl_xor_sync(0xffffffffu, acc.x, z);
          acc.y += __shfl_xor_sync(0xffffffffu, acc.y, z);
          acc.z += __shfl_xor_sync(0xffffffffu, acc.z, z);
          acc.w += __shfl_xor_sync(0xffffffffu, acc.w, z);
        }
        if (v == 0 && x < end && row0 + r >= 0) put(-1, r, c, acc, top, den, fp.v_scale);
      }
      cluster_sync();  // the others have read this CTA's memory
    }
    // The kernel before this one clears the error word; one CTA waits for its end, so that
    // what follows this kernel follows that one.
    if (threadIdx.x == 0 && (error || blockIdx.x == 0)) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (error) atomicCAS(&p.hdr->error, 0, error);
    }
    return;
  }
  join(slot, fp.v_scale);
  if (slot < 0 || kPlan || NT > 2) return;  // else paged_merge_kernel joins them

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
      mx[i] = kNegInfF;
      sum[i] = 0.f;
#pragma unroll
      for (int z = 0; z < kPer; ++z) acc[i][z] = 0.f;
    }
    for (int s0 = warp; s0 < splits; s0 += kAhead * kF4Warps) {
      float x[kAbreast][kAhead], v[kAbreast][kAhead][kPer];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int s = s0 + u * kF4Warps;
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) {
          x[i][u] = kNegInfF;
#pragma unroll
          for (int z = 0; z < kPer; ++z) v[i][u][z] = 0.f;
          if (s < splits && r0 + i < kRows) {
            const size_t part = part0 + s * pitch + r0 + i;
            x[i][u] = __ldcg(p.lse_part + part) * kLog2eF;
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
        const float alpha = mx[i] == kNegInfF ? 0.f : ex2_approx(mx[i] - mn);
        mx[i] = mn;
        sum[i] *= alpha;
#pragma unroll
        for (int z = 0; z < kPer; ++z) acc[i][z] *= alpha;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float f = x[i][u] == kNegInfF ? 0.f : ex2_approx(x[i][u] - mn);
          sum[i] += f;
#pragma unroll
          for (int z = 0; z < kPer; ++z) acc[i][z] = fmaf(f, v[i][u][z], acc[i][z]);
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
      for (int z = 0; z < kPer; z += 2)
        *reinterpret_cast<float2*>(so + r * D + lane * kPer + z) =
            make_float2(acc[i][z], acc[i][z + 1]);
    }
  }
  __syncthreads();
  join(-1, 1.f);
}

// Before the static kernel, which runs beside it.
__global__ void fp4_begin_kernel(WsHeader* hdr) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  hdr->error = 0;
  hdr->n_items = 0;
}

template <int D, int NT, Fp4Work W>
static cudaError_t launch_fp4_rows_t(const Fp4RowsParams& p, cudaStream_t stream) {
  using C = Fp4RowsCfg<D, NT>;
  auto kern = fp4_rows_kernel<D, NT, W>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
      W == Fp4Work::kStatic ? static_cast<long long>(p.p.num_seqs) * p.p.num_kv_heads * p.parts
                            : p.p.max_work * p.p.num_kv_heads));
  cfg.blockDim = dim3(kF4RowsThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.parts);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // After the schedule kernel, or the one above.
  cfg.numAttrs = W == Fp4Work::kPlan ? 0 : (W == Fp4Work::kStatic && p.parts > 1 ? 2 : 1);
  if (W == Fp4Work::kStatic) {
    fp4_begin_kernel<<<1, 1, 0, stream>>>(p.p.hdr);
    const cudaError_t b = cudaGetLastError();
    if (b != cudaSuccess) return b;
  }
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D, int NT>
static cudaError_t launch_fp4_rows_w(const Fp4RowsParams& p, cudaStream_t stream) {
  if (p.parts > 0) return launch_fp4_rows_t<D, NT, Fp4Work::kStatic>(p, stream);
  return p.p.shape.plan ? launch_fp4_rows_t<D, NT, Fp4Work::kPlan>(p, stream)
                        : launch_fp4_rows_t<D, NT, Fp4Work::kList>(p, stream);
}

template <int D>
static cudaError_t launch_fp4_rows_d(const Fp4RowsParams& p, cudaStream_t stream) {
  return p.p.shape.rows == 8    ? launch_fp4_rows_w<D, 1>(p, stream)
         : p.p.shape.rows == 16 ? launch_fp4_rows_w<D, 2>(p, stream)
                                : launch_fp4_rows_w<D, 4>(p, stream);
}

cudaError_t launch_fp4_rows(const Fp4RowsParams& p, int D, cudaStream_t stream) {
  return D == 64 ? launch_fp4_rows_d<64>(p, stream) : launch_fp4_rows_d<128>(p, stream);
}

}  // namespace cpattn
