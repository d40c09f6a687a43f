// Host side of the C ABI's norm + rotation and paged-cache calls (declared in
// include/cpattn.h): argument checks, workspace layout and kernel launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cpattn.h"
#include "kernels.h"
#include "paged_plan.cuh"

namespace cpattn {

namespace {

constexpr size_t kServeAlign = 256;
constexpr int64_t kInt31 = int64_t(1) << 31;

inline size_t serve_align(size_t x) { return (x + kServeAlign - 1) / kServeAlign * kServeAlign; }

// sm_103a only, as every kernel of the library.
int serve_device(DeviceInfo* dev) {
  const int st = device_info(dev);
  if (st != CPATTN_OK) return st;
  return dev->cc_major == 10 && dev->cc_minor == 3 ? CPATTN_OK : CPATTN_ERR_UNSUPPORTED;
}

// Token-major rows of `heads` whole heads, read or written 16 bytes at a time.
bool rows_ok(const void* p, int64_t stride, int64_t heads, int32_t D) {
  return p != nullptr && aligned(p, 16) && stride >= heads * D && stride % 8 == 0;
}

// What the norm + rotation calls share; rope_table null: no rotation.
int check_turn(const float* table, int32_t rot, int32_t max_pos, const void* wq, const void* wk,
               bool both_weights, float eps, int32_t interleaved, int32_t D) {
  if (D != 64 && D != 128) return CPATTN_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return CPATTN_ERR_INVALID_ARG;
  if (table != nullptr &&
      (!aligned(table, 16) || rot < 16 || rot > D || rot % 16 != 0 || max_pos < 1))
    return CPATTN_ERR_INVALID_ARG;
  if (both_weights && (wq == nullptr) != (wk == nullptr)) return CPATTN_ERR_INVALID_ARG;
  if ((wq && !aligned(wq, 16)) || (wk && !aligned(wk, 16))) return CPATTN_ERR_INVALID_ARG;
  if ((wq || wk) && !(std::isfinite(eps) && eps > 0.f)) return CPATTN_ERR_INVALID_ARG;
  return CPATTN_OK;
}

// Heads and tokens within what one launch can number (a unit is a token's run
// of heads; T * heads < 2^31 covers every kernel).
bool counts_ok(int64_t T, int64_t heads) {
  return T >= 0 && heads >= 1 && heads <= 3 * 65535 && T < kInt31 && T * heads < kInt31;
}

int page_shift_of(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// The shares are those of a GB300's 152 SMs, not of the device at hand, because the
// workspace's size follows from them and is asked for without a device; on a part
// with fewer only the balance would suffer.
PagedShape paged_shape(int64_t group, int32_t max_seqlen, int32_t num_seqs) {
  PagedShape s;
  const int64_t rows = group * max_seqlen;
  s.tiles = rows > 32;
  // A sequence's rows are one block, a lane's to plan.
  s.plan = !s.tiles && num_seqs <= kPlanSeqs;
  s.join = rows <= 16 && !s.plan;
  if (s.tiles) {
    s.rows = kNQ * static_cast<int>(kBM / group * group);
    s.unit = kBN;
    // A key tile takes 1.4-1.5 us and cutting a list about as long as 14 of them
    // (the schedule has the figures).  In a list that is cut, pieces of four tiles
    // pay for items above eight (an item of 19 among 28: 30 us, cut above 14: 40 us).
    s.min_units = 4;
    s.whole = 8;
    s.keep = 14;
    s.ctas = 152;
    s.round = 152;
  } else {
    s.rows = rows <= 16 ? 16 : 32;
    s.unit = 64;
    s.min_units = 24;
    s.whole = s.keep = 1;
    s.ctas = 608;
    s.round = 304;
  }
  return s;
}

// Q or O: [T, H, D] in boxes of 64 features x one KV head's query heads x a Q
// tile's tokens.
int q_tile_map(CUtensorMap* map, const void* base, const PagedParams& p, int D) {
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.num_heads),
                              static_cast<cuuint64_t>(p.total_q)};
  const cuuint64_t strides[2] = {row, row * p.num_heads};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group),
                             static_cast<cuuint32_t>(p.shape.rows / (kNQ * p.group))};
  return encode_bf16_map(map, base, 3, dims, strides, box);
}

// A cache: [pages, page size, KV heads, D] in boxes of 64 features x one head
// x a page's rows (at most a key tile's).
int cache_map(CUtensorMap* map, const void* base, const PagedParams& p, int D) {
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const int size = 1 << p.page_shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.num_kv_heads),
                              static_cast<cuuint64_t>(size),
                              static_cast<cuuint64_t>(p.num_pages)};
  const cuuint64_t strides[3] = {row, row * p.num_kv_heads,
                                 static_cast<cuuint64_t>(p.page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(size < kBN ? size : kBN), 1};
  return encode_bf16_map(map, base, 4, dims, strides, box);
}

PagedLayout paged_layout(int64_t total_q, int32_t B, int32_t H, int32_t Hk, int32_t D,
                         const PagedShape& s) {
  PagedLayout l;
  l.max_work = total_q * (H / Hk) / s.rows + B + s.ctas / Hk;
  l.max_slots = 2 * static_cast<int64_t>(s.ctas) / Hk;
  size_t off = serve_align(sizeof(WsHeader));
  l.first_off = off;
  off = serve_align(off + sizeof(int) * (static_cast<size_t>(B) + 1));
  l.work_off = off;
  off = serve_align(off + sizeof(PagedWork) * static_cast<size_t>(l.max_work));
  l.merge_off = off;
  off = serve_align(off + sizeof(PagedMerge) * static_cast<size_t>(l.max_slots / 2 + 1));
  l.arrived_off = off;
  off = serve_align(off + sizeof(int) * static_cast<size_t>(l.max_slots / 2 + 1) * Hk);
  l.error_off = off;
  if (s.plan) off = serve_align(off + sizeof(int) * static_cast<size_t>(l.max_work) * Hk);
  const size_t rows = static_cast<size_t>(l.max_slots) * Hk * s.rows;
  l.o_off = off;
  off = serve_align(off + rows * D * sizeof(float));
  l.lse_off = off;
  off = serve_align(off + rows * sizeof(float));
  l.total = off;
  return l;
}

// Bytes for this batch and every smaller one (fewer tokens, sequences or new tokens
// of a sequence): the largest layout of the shapes among them, which change at 16
// and at 32 rows and at kPlanSeqs sequences.
size_t paged_workspace(int64_t total_q, int32_t B, int32_t H, int32_t Hk, int32_t D,
                       int32_t max_seqlen) {
  const int64_t group = H / Hk;
  size_t most = 0;
  for (const int64_t rows : {int64_t(16), int64_t(32), group * max_seqlen}) {
    const int32_t len = static_cast<int32_t>(std::min<int64_t>(max_seqlen, rows / group));
    for (const int32_t seqs : {B, std::min(B, kPlanSeqs)})
      most = std::max(
          most, paged_layout(total_q, seqs, H, Hk, D, paged_shape(group, len, seqs)).total);
  }
  return most;
}

bool paged_sizes_ok(int64_t total_q, int32_t B, int32_t H, int32_t Hk, int32_t max_seqlen) {
  if (total_q < 0 || total_q >= kInt31 || B < 0 || H < 1 || H > 65535 || Hk < 1 || H % Hk != 0 ||
      max_seqlen < 0)
    return false;
  const int64_t group = H / Hk;
  return max_seqlen * group < (int64_t(1) << 30);
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cpattn_qk_norm_rope(const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const int32_t* positions,
                                   const float* rope_table, int32_t rotary_dim,
                                   int32_t max_position, const void* q_weight,
                                   const void* k_weight, float eps, int32_t interleaved,
                                   int64_t total_tokens, int32_t num_heads, int32_t num_kv_heads,
                                   int32_t head_dim, void* q_out, int64_t q_out_stride,
                                   void* k_out, int64_t k_out_stride, int32_t* status,
                                   void* stream) {
  int st = check_turn(rope_table, rotary_dim, max_position, q_weight, k_weight, true, eps,
                      interleaved, head_dim);
  if (st != CPATTN_OK) return st;
  if (rope_table == nullptr && q_weight == nullptr) return CPATTN_ERR_INVALID_ARG;
  if (num_heads < 1 || num_kv_heads < 1 ||
      !counts_ok(total_tokens, static_cast<int64_t>(num_heads) + num_kv_heads))
    return CPATTN_ERR_INVALID_ARG;
  if (status != nullptr && !aligned(status, 4)) return CPATTN_ERR_INVALID_ARG;
  if (total_tokens == 0) return CPATTN_OK;
  if (!rows_ok(q, q_stride, num_heads, head_dim) || !rows_ok(k, k_stride, num_kv_heads, head_dim) ||
      !rows_ok(q_out, q_out_stride, num_heads, head_dim) ||
      !rows_ok(k_out, k_out_stride, num_kv_heads, head_dim))
    return CPATTN_ERR_INVALID_ARG;
  if (rope_table != nullptr && (positions == nullptr || !aligned(positions, 4)))
    return CPATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  st = serve_device(&dev);
  if (st != CPATTN_OK) return st;
  NormRopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.positions = positions;
  p.table = rope_table;
  p.rot = rotary_dim;
  p.max_pos = max_position;
  p.q_heads = num_heads;
  p.kv_heads = num_kv_heads;
  p.total_tokens = total_tokens;
  p.eps = eps;
  p.sign = 1.f;
  p.status = status;
  return launch_norm_rope(p, head_dim, interleaved != 0, dev.num_sms,
                          static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

extern "C" size_t cpattn_qk_norm_rope_bwd_workspace_size(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return sizeof(float) * static_cast<size_t>(kNormRopeBwdCtas) * head_dim;
}

extern "C" int cpattn_qk_norm_rope_bwd(
    const void* dq_out, int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride,
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
    const float* rope_table, int32_t rotary_dim, int32_t max_position, const void* q_weight,
    const void* k_weight, float eps, int32_t interleaved, int64_t total_tokens, int32_t num_heads,
    int32_t num_kv_heads, int32_t head_dim, void* dq, int64_t dq_stride, void* dk,
    int64_t dk_stride, float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
    int32_t* status, void* stream) {
  int st = check_turn(rope_table, rotary_dim, max_position, q_weight, k_weight, true, eps,
                      interleaved, head_dim);
  if (st != CPATTN_OK) return st;
  if (rope_table == nullptr && q_weight == nullptr) return CPATTN_ERR_INVALID_ARG;
  if (num_heads < 1 || num_kv_heads < 1 ||
      !counts_ok(total_tokens, static_cast<int64_t>(num_heads) + num_kv_heads))
    return CPATTN_ERR_INVALID_ARG;
  if (status != nullptr && !aligned(status, 4)) return CPATTN_ERR_INVALID_ARG;
  const bool normed = q_weight != nullptr;
  if (normed) {
    if (dq_weight == nullptr || dk_weight == nullptr || !aligned(dq_weight, 4) ||
        !aligned(dk_weight, 4))
      return CPATTN_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, kServeAlign)) return CPATTN_ERR_INVALID_ARG;
    if (workspace_bytes < cpattn_qk_norm_rope_bwd_workspace_size(head_dim))
      return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  }
  if (total_tokens > 0) {
    if (!rows_ok(dq_out, dq_out_stride, num_heads, head_dim) ||
        !rows_ok(dk_out, dk_out_stride, num_kv_heads, head_dim) ||
        !rows_ok(dq, dq_stride, num_heads, head_dim) ||
        !rows_ok(dk, dk_stride, num_kv_heads, head_dim))
      return CPATTN_ERR_INVALID_ARG;
    // Without norms the inputs are not read.
    if (normed && (!rows_ok(q, q_stride, num_heads, head_dim) ||
                   !rows_ok(k, k_stride, num_kv_heads, head_dim)))
      return CPATTN_ERR_INVALID_ARG;
    if (rope_table != nullptr && (positions == nullptr || !aligned(positions, 4)))
      return CPATTN_ERR_INVALID_ARG;
  }
  DeviceInfo dev;
  st = serve_device(&dev);
  if (st != CPATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!normed) {  // the inverse rotation of the gradients
    if (total_tokens == 0) return CPATTN_OK;
    NormRopeParams f{};
    f.q = static_cast<const __nv_bfloat16*>(dq_out);
    f.k = static_cast<const __nv_bfloat16*>(dk_out);
    f.q_out = static_cast<__nv_bfloat16*>(dq);
    f.k_out = static_cast<__nv_bfloat16*>(dk);
    f.q_stride = dq_out_stride;
    f.k_stride = dk_out_stride;
    f.q_out_stride = dq_stride;
    f.k_out_stride = dk_stride;
    f.positions = positions;
    f.table = rope_table;
    f.rot = rotary_dim;
    f.max_pos = max_position;
    f.q_heads = num_heads;
    f.kv_heads = num_kv_heads;
    f.total_tokens = total_tokens;
    f.sign = -1.f;
    f.status = status;
    return launch_norm_rope(f, head_dim, interleaved != 0, dev.num_sms, s) == cudaSuccess
               ? CPATTN_OK
               : CPATTN_ERR_CUDA;
  }
  NormRopeBwdParams p{};
  p.dq_out = static_cast<const __nv_bfloat16*>(dq_out);
  p.dk_out = static_cast<const __nv_bfloat16*>(dk_out);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dq_out_stride = dq_out_stride;
  p.dk_out_stride = dk_out_stride;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.dq_stride = dq_stride;
  p.dk_stride = dk_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.positions = positions;
  p.table = rope_table;
  p.rot = rotary_dim;
  p.max_pos = max_position;
  p.q_heads = num_heads;
  p.kv_heads = num_kv_heads;
  p.total_tokens = total_tokens;
  p.eps = eps;
  p.status = status;
  p.partial = static_cast<float*>(workspace);
  return launch_norm_rope_bwd(p, head_dim, interleaved != 0, dq_weight, dk_weight, dev.num_sms,
                              s) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

extern "C" int cpattn_paged_append(
    const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* k_cache,
    void* v_cache, int64_t num_pages, int32_t page_size, int64_t page_stride,
    const int32_t* page_table, int32_t max_pages, const int32_t* cu_seqlens,
    const int32_t* kv_lens, int32_t num_seqs, int64_t total_tokens, int32_t num_kv_heads,
    int32_t head_dim, const float* rope_table, int32_t rotary_dim, int32_t max_position,
    int32_t interleaved, const void* q_weight, const void* k_weight, float eps, const void* q,
    int64_t q_stride, int32_t num_heads, void* q_out, int64_t q_out_stride, int32_t* status,
    void* stream) {
  // Queries of no tokens may have a null address.
  const bool with_q = q != nullptr || (total_tokens == 0 && num_heads > 0);
  int st = check_turn(rope_table, rotary_dim, max_position, q_weight, k_weight, with_q, eps,
                      interleaved, head_dim);
  if (st != CPATTN_OK) return st;
  if (!with_q && (q_weight != nullptr || q_out != nullptr || num_heads != 0))
    return CPATTN_ERR_INVALID_ARG;
  if (with_q && num_heads < 1) return CPATTN_ERR_INVALID_ARG;
  if (num_kv_heads < 1 || num_heads < 0 || num_seqs < 0 ||
      !counts_ok(total_tokens, static_cast<int64_t>(num_heads) + 2 * static_cast<int64_t>(num_kv_heads)))
    return CPATTN_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0) return CPATTN_ERR_UNSUPPORTED;
  if (num_pages < 1 || num_pages >= kInt31 || max_pages < 0 ||
      page_stride < static_cast<int64_t>(page_size) * num_kv_heads * head_dim ||
      page_stride % 8 != 0)
    return CPATTN_ERR_INVALID_ARG;
  if (status != nullptr && !aligned(status, 4)) return CPATTN_ERR_INVALID_ARG;
  if (total_tokens == 0 || num_seqs == 0) return CPATTN_OK;
  if (!rows_ok(k, k_stride, num_kv_heads, head_dim) || !rows_ok(v, v_stride, num_kv_heads, head_dim))
    return CPATTN_ERR_INVALID_ARG;
  if (q != nullptr && (!rows_ok(q, q_stride, num_heads, head_dim) ||
                       !rows_ok(q_out, q_out_stride, num_heads, head_dim)))
    return CPATTN_ERR_INVALID_ARG;
  if (k_cache == nullptr || v_cache == nullptr || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      k_cache == v_cache)
    return CPATTN_ERR_INVALID_ARG;
  if (page_table == nullptr || cu_seqlens == nullptr || kv_lens == nullptr ||
      !aligned(page_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
    return CPATTN_ERR_INVALID_ARG;
  DeviceInfo dev;
  st = serve_device(&dev);
  if (st != CPATTN_OK) return st;
  NormRopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_cache);
  p.v_out = static_cast<__nv_bfloat16*>(v_cache);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.table = rope_table;
  p.rot = rotary_dim;
  p.max_pos = max_position;
  p.q_heads = num_heads;
  p.kv_heads = num_kv_heads;
  p.total_tokens = total_tokens;
  p.eps = eps;
  p.sign = 1.f;
  p.status = status;
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = kv_lens;
  p.page_table = page_table;
  p.num_seqs = num_seqs;
  p.num_pages = static_cast<int>(num_pages);
  p.page_shift = shift;
  p.max_pages = max_pages;
  p.page_stride = page_stride;
  return launch_norm_rope(p, head_dim, interleaved != 0, dev.num_sms,
                          static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

extern "C" size_t cpattn_paged_attn_workspace_size(int64_t total_q, int32_t num_seqs,
                                                   int32_t num_heads, int32_t num_kv_heads,
                                                   int32_t head_dim, int32_t max_seqlen) {
  if (!paged_sizes_ok(total_q, num_seqs, num_heads, num_kv_heads, max_seqlen) ||
      (head_dim != 64 && head_dim != 128) || num_heads / num_kv_heads > kPagedMaxGroup)
    return 0;
  return paged_workspace(total_q, num_seqs, num_heads, num_kv_heads, head_dim, max_seqlen);
}

extern "C" int cpattn_paged_attn(const void* q, const void* k_cache, const void* v_cache,
                                 int64_t num_pages, int32_t page_size, int64_t page_stride,
                                 const int32_t* page_table, int32_t max_pages,
                                 const int32_t* cu_seqlens, const int32_t* kv_lens,
                                 int32_t num_seqs, int64_t total_q, int32_t max_seqlen,
                                 int32_t max_kv_len, int32_t num_heads, int32_t num_kv_heads,
                                 int32_t head_dim, float softmax_scale, int32_t causal, void* out,
                                 float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (head_dim != 64 && head_dim != 128) return CPATTN_ERR_UNSUPPORTED;
  if (!paged_sizes_ok(total_q, num_seqs, num_heads, num_kv_heads, max_seqlen) || max_kv_len < 0 ||
      max_kv_len > (1 << 30))
    return CPATTN_ERR_INVALID_ARG;
  const int group = num_heads / num_kv_heads;
  const int shift = page_shift_of(page_size);
  if (group > kPagedMaxGroup || shift < 0) return CPATTN_ERR_UNSUPPORTED;
  if (!(std::isfinite(softmax_scale) && softmax_scale > 0.f) || (causal != 0 && causal != 1))
    return CPATTN_ERR_INVALID_ARG;
  if (num_pages < 1 || num_pages >= kInt31 || max_pages < 0 ||
      page_stride < static_cast<int64_t>(page_size) * num_kv_heads * head_dim ||
      page_stride % 8 != 0)
    return CPATTN_ERR_INVALID_ARG;
  const bool any = total_q > 0 && num_seqs > 0;
  if (any) {
    for (const void* ptr : {q, k_cache, v_cache, static_cast<const void*>(out)})
      if (ptr == nullptr || !aligned(ptr, 16)) return CPATTN_ERR_INVALID_ARG;
    if (out == q) return CPATTN_ERR_INVALID_ARG;
    if (max_seqlen < 1) return CPATTN_ERR_INVALID_ARG;
    // A batch without cached keys may come without a table.
    if (max_pages > 0 && (page_table == nullptr || !aligned(page_table, 4)))
      return CPATTN_ERR_INVALID_ARG;
  }
  if (num_seqs > 0 && (cu_seqlens == nullptr || kv_lens == nullptr || !aligned(cu_seqlens, 4) ||
                       !aligned(kv_lens, 4)))
    return CPATTN_ERR_INVALID_ARG;
  if (lse != nullptr && !aligned(lse, 4)) return CPATTN_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, kServeAlign)) return CPATTN_ERR_INVALID_ARG;
  PagedParams p{};
  p.shape = paged_shape(group, max_seqlen, num_seqs);
  const PagedLayout lay =
      paged_layout(total_q, num_seqs, num_heads, num_kv_heads, head_dim, p.shape);
  if (workspace_bytes < lay.total) return CPATTN_ERR_WORKSPACE_TOO_SMALL;
  if (lay.max_work * num_kv_heads >= kInt31) return CPATTN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  const int st = serve_device(&dev);
  if (st != CPATTN_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  p.cu_seqlens = cu_seqlens;
  p.kv_lens = kv_lens;
  p.page_table = page_table;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.num_pages = static_cast<int>(num_pages);
  p.page_shift = shift;
  p.max_pages = max_pages;
  p.causal = causal;
  p.max_seqlen = max_seqlen;
  p.max_kv_len = max_kv_len;
  p.total_q = total_q;
  p.page_stride = page_stride;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.first = reinterpret_cast<int*>(ws + lay.first_off);
  p.work = reinterpret_cast<PagedWork*>(ws + lay.work_off);
  p.merge = reinterpret_cast<PagedMerge*>(ws + lay.merge_off);
  p.arrived = reinterpret_cast<int*>(ws + lay.arrived_off);
  p.cta_error = reinterpret_cast<int*>(ws + lay.error_off);
  p.o_part = reinterpret_cast<float*>(ws + lay.o_off);
  p.lse_part = reinterpret_cast<float*>(ws + lay.lse_off);
  // The grid: no more splits than units, nor (a plan's items are at most num_seqs)
  // than one round when they are made to fit one.  CTAs without work cost a small
  // step a round of their own.
  p.max_work = lay.max_work;
  const int64_t units = (static_cast<int64_t>(max_kv_len) + p.shape.unit - 1) / p.shape.unit;
  const int64_t items = total_q * group / p.shape.rows + num_seqs;
  if (units < 1) p.max_work = p.max_work < items ? p.max_work : items;
  else if (p.max_work / units >= items) p.max_work = items * units;
  const int64_t lanes = static_cast<int64_t>(num_seqs) * num_kv_heads;
  if (p.shape.plan && 2 * lanes <= p.shape.round && p.max_work > p.shape.round / num_kv_heads)
    p.max_work = p.shape.round / num_kv_heads;
  p.max_slots = lay.max_slots;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Without rows there is still the error word to write.
  if ((!p.shape.plan || !any) && launch_paged_schedule(p, s) != cudaSuccess)
    return CPATTN_ERR_CUDA;
  if (!any) return CPATTN_OK;
  if (p.shape.tiles) {
    CUtensorMap tq, tk, tv, to;
    if (q_tile_map(&tq, q, p, head_dim) != CPATTN_OK ||
        q_tile_map(&to, out, p, head_dim) != CPATTN_OK ||
        cache_map(&tk, k_cache, p, head_dim) != CPATTN_OK ||
        cache_map(&tv, v_cache, p, head_dim) != CPATTN_OK)
      return CPATTN_ERR_CUDA;
    if (launch_paged_tile(tq, tk, tv, to, p, head_dim, s) != cudaSuccess) return CPATTN_ERR_CUDA;
  } else if (launch_paged_rows(p, head_dim, s) != cudaSuccess) {
    return CPATTN_ERR_CUDA;
  }
  // Lists of short items are never cut; after a plan the merge also writes the error word.
  if (!p.shape.join && (p.shape.plan || max_kv_len > p.shape.keep * p.shape.unit) &&
      launch_paged_merge(p, head_dim, dev.num_sms, s) != cudaSuccess)
    return CPATTN_ERR_CUDA;
  return CPATTN_OK;
}
