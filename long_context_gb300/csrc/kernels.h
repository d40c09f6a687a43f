// Internal interface between the host library (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace cpattn {

// Geometry of the attention kernel.
constexpr int kBM = 128;               // query rows per Q tile (= TMEM lanes)
constexpr int kBN = 128;               // keys per KV tile
constexpr int kNQ = 2;                 // Q tiles per CTA, ping-ponged
constexpr int kRowsPerItem = kBM * kNQ;
constexpr int kThreads = 384;          // 2 softmax warpgroups + control WG
// Register split (setmaxnreg): the kernel is launched at kLaunchRegs per
// thread; the control warpgroup drops to kCtrlRegs and the two softmax
// warpgroups rise to kSoftmaxRegs.  The shares add up to the launch total:
// 384 * 168 = 256 * 224 + 128 * 56.
constexpr int kLaunchRegs = 168;
constexpr int kSoftmaxRegs = 224;
constexpr int kCtrlRegs = 56;
static_assert(kThreads * kLaunchRegs == 256 * kSoftmaxRegs + 128 * kCtrlRegs,
              "register split must match the launch allocation");
constexpr int kMaxCp = 64;

// Workspace layout (all offsets 256-byte aligned):
//   [0, 256)                 WsHeader
//   [256, +4*(B+1))          first CTA of each sample (in schedule order)
//   [.., +8*max_items)       schedule order of the samples (B ints used)
//   [.., +16*max_items*H)    work table: one CtaWork per attention CTA
//   [.., ...)                unfused mode only: o_steps, m_steps, l_steps
struct WsHeader {
  int error;    // cpattn_status of the last kernels run on this workspace
  int n_items;  // CTAs of the attention grid that have work
  int pad[62];
};

struct WsLayout {
  size_t prefix_off, items_off, table_off, o_off, m_off, l_off, total;
  int64_t max_items;
};

// One attention CTA's work, written by the schedule kernel so that a CTA
// finds it with a single 16-byte load:
//   x = first token of the sample, y = sample length L,
//   z = (head << 8) | CP size c,  w = (query block << 8) | CP rank.
// (head < 2^16, c <= 64, rank < c, block < 2^23 since L < 2^31.)
using CtaWork = int4;

WsLayout ws_layout(int64_t T, int32_t B, int32_t H, int32_t D, int32_t max_cp,
                   bool with_partials);

struct SchedParams {
  const int* cu_seqlens;
  const int* cp_size;  // may be null: every sample at CP 1
  int num_seqs;
  int num_heads;
  long long total_tokens;
  int max_seqlen;
  int max_cp;
  WsHeader* hdr;
  int* first_cta;      // [B + 1]: first CTA of the sample at each order position
  int* order;          // [B]: samples by decreasing length
  CtaWork* table;      // [max_ctas]: work of each CTA (first n_items used)
  // Optional second table over the same items in the opposite order within
  // each (sample, head): increasing item index (null: not written).
  CtaWork* table_asc;
  long long max_ctas;  // grid size the host launches
  int rows_per_item;   // query (or key) rows per item
};

struct FwdParams {
  const CtaWork* table;  // [grid]: written by the schedule kernel
  int num_heads;
  int num_steps;        // ring steps walked: max_cp (fused) or S (partials)
  int causal;
  float scale_log2;     // softmax_scale * log2(e)
  __nv_bfloat16* out;   // fused: [T, H, D]
  float* lse;           // fused: [T, H] or null
  float* o_steps;       // partials: [S, T, H, D]
  float* m_steps;       // partials: [S, T, H]
  float* l_steps;
  long long total_tokens;
  WsHeader* hdr;
  int num_sms;          // CTA x_cta + num_sms is, in table order, a likely next CTA
};

// Backward kernels (attn_bwd.cu).  Gradients are bf16 [T, H, D]; `lse` is
// the forward's natural-log LSE [T, H]; `delta` = rowsum(dO * O) [T, H].
struct BwdParams {
  const CtaWork* table;  // this kernel's work table (written by the schedule kernel)
  const float* lse;
  const float* delta;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int num_heads;
  int causal;
  float scale;       // softmax scale (applied to dQ and dK at the end)
  float scale_log2;  // softmax scale * log2(e)
  WsHeader* hdr;
  long long total_tokens;  // T (bounds of the debug build's checks)
};

struct MergeParams {
  const float* o_steps;
  const float* m_steps;
  const float* l_steps;  // null: every l_s is 1 (normalised partials, m_s = their LSE)
  int num_steps;
  long long rows;       // T * H
  float* out_o;         // public merge: O / l in fp32
  float* out_m;
  float* out_l;
  __nv_bfloat16* out_bf16;  // unfused forward: O / l in bf16
  float* out_lse;           // m + ln l (written when not null)
};

// Host-side forward arguments and the launch sequence shared by the entry
// points (api.cu).
struct FwdArgs {
  const void *q, *k, *v;
  const int32_t *cu, *cp;
  int32_t B;
  int64_t T;
  int32_t max_seqlen, max_cp, H, D;
  float scale;
  int32_t causal;
};

bool aligned(const void* p, size_t a);

struct DeviceInfo {
  int num_sms = 0;
  int cc_major = 0;
  int cc_minor = 0;
};

// Properties of the current device (cached); a cpattn_status.
int device_info(DeviceInfo* out);

// Tensor map over a bf16 array of `rank` dimensions (innermost first; strides
// in bytes from the second on), 128-byte swizzle; a cpattn_status.  Needs an
// earlier device_info call.
int encode_bf16_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box);

// Host-checkable argument rules of the forward calls; a cpattn_status.
int check_fwd(const FwdArgs& a);

// Schedule kernel + attention kernel on `stream`, using `workspace` (at least
// ws_layout(T, B, H, D, max_cp, false).total bytes) for the error word and the
// work list; a cpattn_status.
int run_attention(const FwdArgs& a, bool partials, int32_t num_steps,
                  __nv_bfloat16* out, float* lse, float* o_steps,
                  float* m_steps, float* l_steps, void* workspace,
                  cudaStream_t stream);

cudaError_t launch_schedule(const SchedParams& p, cudaStream_t stream);

// Dynamic shared memory the attention kernel needs for head_dim D.
int attn_smem_bytes(int D);

cudaError_t launch_attn(const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const CUtensorMap& to, const FwdParams& p, int D,
                        bool partials, long long grid, cudaStream_t stream);

// Decode-time CP partials (decode.cu): q [B, H, D] bf16 (one new token per
// sequence), the KV cache k, v [T, H, D] bf16 packed by cu_seqlens [B + 1];
// shard s of sequence b is its keys [s*ceil(L/c), min((s+1)*ceil(L/c), L)).
// Outputs the normalised partials o_steps [c, B, H, D] and their natural-log
// LSE lse_steps [c, B, H] (an empty shard: 0 and -inf).
struct DecodeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int* cu_seqlens;
  int num_seqs, num_heads, cp;
  long long total_tokens;
  float scale_log2;
  float* o_steps;
  float* lse_steps;
};

cudaError_t launch_decode_partials(const DecodeParams& p, int D, cudaStream_t stream);


// delta[r] = sum_d dO[r, d] * O[r, d] for rows r < rows (= T * H).
cudaError_t launch_bwd_delta(const __nv_bfloat16* out, const __nv_bfloat16* dout,
                             float* delta, long long rows, int D, int num_sms,
                             cudaStream_t stream);

// dK/dV kernel (one CTA per 128-key tile) and dQ kernel (one CTA per 128-query
// tile); the four tensor maps are Q, K, V, dO.
cudaError_t launch_bwd_dkdv(const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, const CUtensorMap& tdo,
                            const BwdParams& p, int D, long long grid, cudaStream_t stream);
cudaError_t launch_bwd_dq(const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const CUtensorMap& tdo,
                          const BwdParams& p, int D, long long grid, cudaStream_t stream);

cudaError_t launch_merge(const MergeParams& p, int D, bool bf16_out,
                         int num_sms, cudaStream_t stream);

// Norm + rotation (norm_rope.cu).  Inputs and outputs are token-major rows of
// whole heads, [T, heads, D] with a token stride in elements; `table` (null: no
// rotation) is float [max_pos, rot]; both weights are null or neither.  With a
// page table the kernel also copies v, takes positions from cu_seqlens and
// kv_lens, and k_out / v_out are the paged caches (q_heads 0: no queries).
struct NormRopeParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out, *v_out;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  const __nv_bfloat16 *q_weight, *k_weight;
  const int* positions;
  const float* table;
  int rot, max_pos, q_heads, kv_heads;
  long long total_tokens;
  float eps;
  float sign;  // of the rotation: 1, or -1 for its inverse
  int* status;
  const int *cu_seqlens, *kv_lens, *page_table;
  int num_seqs, num_pages, page_shift, max_pages;
  long long page_stride;
};

cudaError_t launch_norm_rope(const NormRopeParams& p, int D, bool interleaved, int num_sms,
                             cudaStream_t stream);

constexpr int kNormRopeBwdCtas = 1024;  // at most this many rows of partial weight gradients

struct NormRopeBwdParams {
  const __nv_bfloat16 *dq_out, *dk_out, *q, *k;
  __nv_bfloat16 *dq, *dk;
  long long dq_out_stride, dk_out_stride, q_stride, k_stride, dq_stride, dk_stride;
  const __nv_bfloat16 *q_weight, *k_weight;
  const int* positions;
  const float* table;
  int rot, max_pos, q_heads, kv_heads;
  long long total_tokens;
  float eps;
  int* status;
  float* partial;  // [CTAs, D]
  int q_ctas;      // CTAs that take the query heads (set by the launch)
};

cudaError_t launch_norm_rope_bwd(const NormRopeBwdParams& p, int D, bool interleaved, float* dqw,
                                 float* dkw, int num_sms, cudaStream_t stream);

// Attention over a paged KV cache (paged_*.cu).  A row is one (token, query
// head of the KV head's group) pair; the rows of a sequence for one KV head are
// numbered token * group + head and cut into blocks of `rows` aligned to their
// end (block 0 may be short).  An item is one block; an item's visible keys
// are cut into splits of whole units (of `unit` keys), and the attention
// kernels run one CTA per (split, KV head).
constexpr int kPagedMaxGroup = 128;

// One split, written by the schedule kernel (three 16-byte loads).
struct alignas(16) PagedWork {
  int tok0, q_len, kv_len, seq;
  int blk;           // row block
  int kv_lo, kv_hi;  // keys [kv_lo, kv_hi), kv_lo a multiple of the unit
  int slot;          // slot of the partial results; -1: the item is whole
  int slot0, n;      // a split item: its first slot and its splits
  int item;          // a split item: its number among them
  int pad;
};

// One item whose splits the merge kernel joins.
struct alignas(16) PagedMerge {
  int tok0, q_len, blk, slot0;
  int n, pad[3];
};

struct PagedLayout {
  size_t first_off, work_off, merge_off, arrived_off, error_off, o_off, lse_off, total;
  int64_t max_work;   // splits of one KV head
  int64_t max_slots;  // slots of one KV head
};

// How the rows are cut for a group size, and how far splits go.
struct PagedShape {
  bool tiles;      // the tensor-memory kernel (else the register kernel)
  int rows;        // rows of a block
  int unit;        // keys of a unit
  int min_units;   // tiles, and few rows of many items: a split has at least so many units
  int whole;       // items of up to so many units stay whole
  int keep;        // and lists that have no larger items than this
  int ctas;        // a split does at least 1 / ctas of the whole work
  int round;       // CTAs resident at once (at most ctas)
  bool join;       // the last CTA of a split item joins it (else a merge kernel)
  bool plan;       // no schedule kernel: every warp works the list out (paged_plan.cuh)
};

struct PagedParams {
  const __nv_bfloat16 *q, *k_cache, *v_cache;
  const int *cu_seqlens, *kv_lens, *page_table;
  int num_seqs, num_heads, num_kv_heads, group;
  int num_pages, page_shift, max_pages, causal;
  int max_seqlen, max_kv_len;
  long long total_q, page_stride;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;  // [total_q, num_heads] or null
  WsHeader* hdr;
  int* first;         // [num_seqs + 1]: first item of each sequence
  PagedWork* work;    // [max_work]
  PagedMerge* merge;  // [max_slots / 2]
  int* arrived;       // [max_slots / 2, num_kv_heads]: splits that are done (join)
  int* cta_error;     // [max_work, num_kv_heads]: bad pages seen (plan)
  float* o_part;      // [max_slots, num_kv_heads, rows, D], normalised
  float* lse_part;    // [max_slots, num_kv_heads, rows], natural log
  long long max_work, max_slots;
  PagedShape shape;
};

// Units of a split when there are few rows: with few items the splits are made to
// fit one round of resident CTAs (sum of ceil(u / target) <= all / target + items),
// else to be several rounds that even out, of at least min_units: a join costs as
// much as about 20 units (with 4, 24 and 32: 65 caches of 327 to 655 keys, 4 heads,
// 27.0, 18.5 and 18.4 us; 90 of 601 to 4,808 keys, 2 heads, 60.8, 59.4 and 64.6).
__device__ __forceinline__ int paged_rows_target(const PagedShape& s, long long all, int items,
                                                 int heads) {
  const long long lanes = static_cast<long long>(items) * heads;
  const bool one = 2 * lanes <= s.round;
  const long long share = one ? s.round - lanes : s.ctas;
  const long long target = (all * heads + share - 1) / share;
  const long long least = one ? 1 : s.min_units;
  return static_cast<int>(target < least ? least : (target > (1 << 30) ? (1 << 30) : target));
}

cudaError_t launch_paged_schedule(const PagedParams& p, cudaStream_t stream);
cudaError_t launch_paged_rows(const PagedParams& p, int D, cudaStream_t stream);
cudaError_t launch_paged_tile(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const PagedParams& p, int D,
                              cudaStream_t stream);
cudaError_t launch_paged_merge(const PagedParams& p, int D, int num_sms, cudaStream_t stream);

}  // namespace cpattn
