// attention.hip -- attention over a paged key-value cache on gfx950.
//
// Kernels and the C ABI declared in include/qemb_attention.h:
//   * norm_rope_kernel   norms of queries and keys, rotation, append (norm_rope.inc)
//   * prompt_*           causal / windowed attention of prompts (prompt.inc)
//   * decode_*           attention of one new token over the pages (decode.inc)
//   * shared_*           attention of new tokens whose sequences share prefixes (shared.inc)
//   * evict_*            selection by accumulated mass and the copy (evict.inc)
// rows.inc holds the row formats: 16-bit rows and the library's packed rows.
//
// Built without fast-math and without contraction (a packed row must round
// exactly as the range rule of qemb.h says); fused multiply-adds are written
// out where a kernel wants them.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "qemb_attention.h"

namespace {

constexpr int kWave = 64;
constexpr int kBlock = 256;
constexpr int64_t kMaxBlocks = (1 << 24) - 1;  // of kBlock threads: a launch counts threads in 32 bits
constexpr int64_t kMostPlaces = INT32_MAX - 1023;  // rows, keys and slots are counted in 32 bits, up to a step past the last

#include "../common.inc"
#include "rows.inc"
#include "norm_rope.inc"
#include "prompt.inc"
#include "decode.inc"
#include "shared.inc"
#include "evict.inc"

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool is_pow2(int32_t v) { return v > 0 && (v & (v - 1)) == 0; }
inline int log2_of(int32_t v) { return 31 - __builtin_clz((unsigned)v); }

// Sizes that every entry point with heads checks alike.
inline int check_heads(int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype) {
  if (q_heads < 1 || kv_heads < 1 || dim < 1) return QEMB_E_INVALID_ARG;
  if (dtype != QEMB_DTYPE_BF16 && dtype != QEMB_DTYPE_FP16) return QEMB_E_INVALID_ARG;
  if (dim > QEMB_MAX_HEAD_DIM || dim % 8) return QEMB_E_UNSUPPORTED;
  return QEMB_OK;
}

// ... and the attentions besides: query heads share kv heads evenly.
inline int check_groups(int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype) {
  if (int rc = check_heads(q_heads, kv_heads, dim, dtype)) return rc;
  return q_heads % kv_heads ? QEMB_E_INVALID_ARG : QEMB_OK;
}

inline bool strides_fit(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0;
}

// Scores are taken as powers of two.
inline bool scale_fits(float scale) { return isfinite(scale * 1.44269504088896340736f); }

// A stride along one token or one head is never taken, so it may be anything.
inline int64_t taken(int64_t stride, int64_t count, int32_t dim) { return count > 1 ? stride : dim; }

inline int64_t row_bytes_of(int32_t dim, int32_t bits) {
  return bits == 16 ? 2 * (int64_t)dim : ((int64_t)dim * bits / 8 + 4 + 15) / 16 * 16;
}

}  // namespace

extern "C" {

int qemb_norm_rope_axes(const void* q, const void* k, const void* v, int64_t tokens, int32_t q_heads,
                        int32_t kv_heads, int32_t dim, int32_t dtype, int64_t q_token_stride,
                        int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const void* positions,
                        int32_t axes, const uint8_t* pair_axes, int32_t index_type, const float* cos_sin,
                        int64_t places, int32_t rot_dim, int32_t interleaved, int32_t norm,
                        const void* q_weight, const void* k_weight, float eps, void* q_out, void* k_out,
                        void* k_pages, void* v_pages, const int64_t* slots, int64_t pages,
                        int32_t page_size, int32_t bits, int32_t* err_count, qemb_stream_t stream) {
  if (tokens < 0 || places < 0 || pages < 0 || rot_dim < 0 || rot_dim > dim) return QEMB_E_INVALID_ARG;
  if (axes < 1 || axes > QEMB_MAX_AXES || (axes > 1 && rot_dim && !pair_axes) || (!norm && (q_weight || k_weight))) return QEMB_E_INVALID_ARG;
  if (index_type != QEMB_INDEX_INT32 && index_type != QEMB_INDEX_INT64) return QEMB_E_INVALID_ARG;
  if (int rc = check_heads(q_heads, kv_heads, dim, dtype)) return rc;
  if (rot_dim % 16) return QEMB_E_UNSUPPORTED;
  const bool cached = k_pages || v_pages;
  if (q_heads + (cached ? 2 : 1) * (int64_t)kv_heads > kMostPlaces) return QEMB_E_UNSUPPORTED;
  if (cached) {
    if (!k_pages || !v_pages || !is_pow2(page_size)) return QEMB_E_INVALID_ARG;
    if (bits != 16 && bits != 8 && bits != 4) return QEMB_E_INVALID_ARG;
  }
  q_token_stride = taken(q_token_stride, tokens, dim), q_head_stride = taken(q_head_stride, q_heads, dim);
  k_token_stride = taken(k_token_stride, tokens, dim), k_head_stride = taken(k_head_stride, kv_heads, dim);
  v_token_stride = taken(v_token_stride, tokens, dim), v_head_stride = taken(v_head_stride, kv_heads, dim);
  if (!strides_fit(q_token_stride, q_head_stride) || !strides_fit(k_token_stride, k_head_stride) ||
      (cached && !strides_fit(v_token_stride, v_head_stride)))
    return QEMB_E_MISALIGNED;
  if (tokens == 0) return QEMB_OK;
  if (!q || !k || !q_out || !positions || (rot_dim && !cos_sin) || (cached ? !v || !slots : !k_out))
    return QEMB_E_INVALID_ARG;
  for (const void* p : {q, k, (const void*)(cached ? v : nullptr), (const void*)q_out, (const void*)k_out,
                        (const void*)k_pages, (const void*)v_pages, (const void*)cos_sin, q_weight, k_weight})
    if (!aligned(p, 16)) return QEMB_E_MISALIGNED;
  if (!aligned(pair_axes, 4)) return QEMB_E_MISALIGNED;
  if (!aligned(positions, index_type == QEMB_INDEX_INT64 ? 8 : 4) || !aligned(slots, 8)) return QEMB_E_MISALIGNED;
  NormRopeArgs a;
  a.x[0] = q, a.x[1] = k, a.x[2] = v;
  a.token_stride[0] = q_token_stride, a.token_stride[1] = k_token_stride, a.token_stride[2] = v_token_stride;
  a.head_stride[0] = q_head_stride, a.head_stride[1] = k_head_stride, a.head_stride[2] = v_head_stride;
  a.weight[0] = q_weight, a.weight[1] = k_weight;
  a.out[0] = q_out, a.out[1] = k_out;
  a.pages[0] = k_pages, a.pages[1] = v_pages;
  a.tokens = tokens;
  a.q_heads = q_heads, a.kv_heads = kv_heads, a.dim = dim;
  a.rows = q_heads + (cached ? 2 : 1) * kv_heads;
  a.positions = positions, a.idx64 = index_type == QEMB_INDEX_INT64;
  a.axes = axes, a.pair_axes = pair_axes, a.norm = norm != 0;
  a.cos_sin = cos_sin, a.places = places, a.rot = rot_dim, a.interleaved = interleaved != 0;
  a.eps = eps;
  a.slots = cached ? slots : nullptr;
  a.n_pages = pages, a.page_log2 = cached ? log2_of(page_size) : 0;
  a.row_bytes = cached ? row_bytes_of(dim, bits) : 0;
  a.err_count = err_count;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int row_bits = cached ? bits : 16;
  // one axis with a norm keeps the kernel that loads its angles in whole pieces
  const bool plain = axes == 1 && !pair_axes && norm;
  if (dtype == QEMB_DTYPE_BF16) return plain ? launch_norm_rope<__bf16, false>(a, row_bits, st) : launch_norm_rope<__bf16, true>(a, row_bits, st);
  return plain ? launch_norm_rope<_Float16, false>(a, row_bits, st) : launch_norm_rope<_Float16, true>(a, row_bits, st);
}

int qemb_norm_rope(const void* q, const void* k, const void* v, int64_t tokens, int32_t q_heads,
                   int32_t kv_heads, int32_t dim, int32_t dtype, int64_t q_token_stride,
                   int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                   int64_t v_token_stride, int64_t v_head_stride, const void* positions,
                   int32_t index_type, const float* cos_sin, int64_t places, int32_t rot_dim,
                   int32_t interleaved, const void* q_weight, const void* k_weight, float eps,
                   void* q_out, void* k_out, void* k_pages, void* v_pages, const int64_t* slots,
                   int64_t pages, int32_t page_size, int32_t bits, int32_t* err_count,
                   qemb_stream_t stream) {
  return qemb_norm_rope_axes(q, k, v, tokens, q_heads, kv_heads, dim, dtype, q_token_stride, q_head_stride, k_token_stride,
                             k_head_stride, v_token_stride, v_head_stride, positions, 1, nullptr, index_type, cos_sin, places,
                             rot_dim, interleaved, 1, q_weight, k_weight, eps, q_out, k_out, k_pages, v_pages, slots, pages,
                             page_size, bits, err_count, stream);
}

int qemb_prompt_attention(const void* q, const void* k, const void* v, int64_t q_tokens,
                          int64_t k_tokens, int32_t batch, int32_t q_heads, int32_t kv_heads,
                          int32_t dim, int32_t dtype, int64_t q_token_stride, int64_t q_head_stride,
                          int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                          int64_t v_head_stride, const int32_t* q_offsets, const int32_t* k_offsets,
                          int64_t max_q, int32_t window, int32_t sinks, float scale, void* out,
                          float* lse, int32_t* err_count, qemb_stream_t stream) {
  if (q_tokens < 0 || k_tokens < 0 || batch < 0 || window < 0 || sinks < 0 || max_q < 0) return QEMB_E_INVALID_ARG;
  if (!scale_fits(scale)) return QEMB_E_INVALID_ARG;
  if (q_tokens > kMostPlaces || k_tokens > kMostPlaces) return QEMB_E_UNSUPPORTED;
  if (int rc = check_groups(q_heads, kv_heads, dim, dtype)) return rc;
  q_token_stride = taken(q_token_stride, q_tokens, dim), q_head_stride = taken(q_head_stride, q_heads, dim);
  k_token_stride = taken(k_token_stride, k_tokens, dim), k_head_stride = taken(k_head_stride, kv_heads, dim);
  v_token_stride = taken(v_token_stride, k_tokens, dim), v_head_stride = taken(v_head_stride, kv_heads, dim);
  // a tile's byte offsets are 32 bits wide
  if (k_token_stride > kMaxTokenStride || v_token_stride > kMaxTokenStride) return QEMB_E_UNSUPPORTED;
  if (!strides_fit(q_token_stride, q_head_stride) || !strides_fit(k_token_stride, k_head_stride) ||
      !strides_fit(v_token_stride, v_head_stride))
    return QEMB_E_MISALIGNED;
  if (q_tokens == 0 || batch == 0) return QEMB_OK;
  if (!q || !out || !q_offsets || !k_offsets || (k_tokens > 0 && (!k || !v))) return QEMB_E_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(q_offsets, 4) ||
      !aligned(k_offsets, 4) || !aligned(lse, 4))
    return QEMB_E_MISALIGNED;
  PromptArgs a;
  a.q = q, a.k = k, a.v = v;
  a.qt = q_token_stride, a.qh = q_head_stride, a.kt = k_token_stride, a.kh = k_head_stride;
  a.vt = v_token_stride, a.vh = v_head_stride;
  a.q_tokens = (int)q_tokens, a.k_tokens = (int)k_tokens, a.batch = batch;
  a.q_heads = q_heads, a.kv_heads = kv_heads, a.dim = dim;
  a.q_offsets = q_offsets, a.k_offsets = k_offsets;
  a.window = window < k_tokens ? window : 0;  // one as long as all keys hides none
  a.sinks = a.window ? (int)(sinks < k_tokens ? sinks : k_tokens) : 0;  // steps are counted past them in 32 bits
  a.scale = scale;
  a.out = out, a.lse = lse, a.err_count = err_count;
  if (max_q == 0 || max_q > q_tokens) max_q = q_tokens;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == QEMB_DTYPE_BF16 ? launch_prompt<__bf16>(a, (int)max_q, st) : launch_prompt<_Float16>(a, (int)max_q, st);
}

size_t qemb_decode_workspace_bytes(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim,
                                   int32_t width, int32_t page_size, int32_t window, int32_t sinks,
                                   int32_t with_mass) {
  if (batch < 1 || check_groups(q_heads, kv_heads, dim, QEMB_DTYPE_BF16) != QEMB_OK || width < 1 || !is_pow2(page_size) ||
      window < 0 || sinks < 0 || (int64_t)width * page_size > kMostPlaces)
    return 0;
  return decode_plan(batch, q_heads, kv_heads, dim, (int64_t)width * page_size, window, sinks, with_mass != 0).bytes;
}

int qemb_decode_attention(const void* q, const void* k_pages, const void* v_pages, int64_t pages,
                          int32_t page_size, int32_t bits, int32_t batch, int32_t q_heads,
                          int32_t kv_heads, int32_t dim, int32_t dtype, const int32_t* block_table,
                          int32_t width, const int32_t* seq_lens, int32_t window, int32_t sinks,
                          float scale, float* mass, int64_t mass_len, void* out, float* lse,
                          void* workspace, int32_t* err_count, qemb_stream_t stream) {
  if (batch < 0 || width < 0 || pages < 0 || window < 0 || sinks < 0 || !is_pow2(page_size)) return QEMB_E_INVALID_ARG;
  if (!scale_fits(scale)) return QEMB_E_INVALID_ARG;
  if (bits != 16 && bits != 8 && bits != 4) return QEMB_E_INVALID_ARG;
  if (int rc = check_groups(q_heads, kv_heads, dim, dtype)) return rc;
  if ((int64_t)width * page_size > kMostPlaces) return QEMB_E_UNSUPPORTED;
  if ((int64_t)kv_heads * page_size > INT32_MAX || (int64_t)kv_heads * page_size * row_bytes_of(dim, bits) > INT32_MAX)
    return QEMB_E_UNSUPPORTED;  // a page's bytes are counted in 32 bits
  if (batch == 0) return QEMB_OK;
  if (!q || !out || !seq_lens || (width > 0 && !block_table) || (pages > 0 && (!k_pages || !v_pages)))
    return QEMB_E_INVALID_ARG;
  if (mass && mass_len < 0) return QEMB_E_INVALID_ARG;
  for (const void* p : {q, k_pages, v_pages, (const void*)out, (const void*)workspace})
    if (!aligned(p, 16)) return QEMB_E_MISALIGNED;
  for (const void* p : {(const void*)block_table, (const void*)seq_lens, (const void*)mass, (const void*)lse})
    if (!aligned(p, 4)) return QEMB_E_MISALIGNED;
  const DecodePlan plan = decode_plan(batch, q_heads, kv_heads, dim, (int64_t)width * page_size, window, sinks, mass != nullptr);
  if (plan.bytes && !workspace) return QEMB_E_INVALID_ARG;
  DecodeArgs a;
  a.q = q;
  a.pages[0] = k_pages, a.pages[1] = v_pages;
  a.n_pages = pages, a.page_log2 = log2_of(page_size), a.row_bytes = row_bytes_of(dim, bits);
  a.batch = batch, a.q_heads = q_heads, a.kv_heads = kv_heads, a.dim = dim;
  a.block_table = block_table, a.width = width, a.seq_lens = seq_lens;
  a.window = window, a.sinks = window ? sinks : 0;
  a.scale = scale;
  a.mass = mass, a.mass_len = mass_len;
  a.out = out, a.lse = lse, a.workspace = (float*)workspace, a.err_count = err_count;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == QEMB_DTYPE_BF16 ? launch_decode<__bf16>(a, plan, bits, st) : launch_decode<_Float16>(a, plan, bits, st);
}

size_t qemb_shared_workspace_bytes(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t groups,
                                   int32_t prefix_width, int32_t width, int32_t page_size, int32_t bits) {
  if (batch < 1 || (bits != 16 && bits != 8 && bits != 4) || check_groups(q_heads, kv_heads, dim, QEMB_DTYPE_BF16) != QEMB_OK || groups < 1 || prefix_width < 0 || width < 0 ||
      !is_pow2(page_size) || (int64_t)width * page_size > kMostPlaces || (int64_t)prefix_width * page_size > kMostPlaces)
    return 0;
  return shared_plan(batch, q_heads, kv_heads, dim, groups, (int64_t)prefix_width * page_size, (int64_t)width * page_size, bits).bytes;
}

int qemb_shared_attention(const void* q, const void* k_pages, const void* v_pages, int64_t pages, int32_t page_size,
                          int32_t bits, int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                          const int32_t* prefix_table, int32_t prefix_width, const int32_t* prefix_lens,
                          const int32_t* group_offsets, int32_t groups, const int32_t* block_table, int32_t width,
                          const int32_t* seq_lens, float scale, void* out, float* lse, void* workspace,
                          int32_t* err_count, qemb_stream_t stream) {
  if (batch < 0 || width < 0 || prefix_width < 0 || pages < 0 || groups < 1 || !is_pow2(page_size)) return QEMB_E_INVALID_ARG;
  if (!scale_fits(scale) || (groups > 1 && !group_offsets)) return QEMB_E_INVALID_ARG;
  if (bits != 16 && bits != 8 && bits != 4) return QEMB_E_INVALID_ARG;
  if (int rc = check_groups(q_heads, kv_heads, dim, dtype)) return rc;
  if ((int64_t)width * page_size > kMostPlaces || (int64_t)prefix_width * page_size > kMostPlaces) return QEMB_E_UNSUPPORTED;
  if ((int64_t)batch * q_heads > kMostPlaces) return QEMB_E_UNSUPPORTED;
  if ((int64_t)kv_heads * page_size > INT32_MAX || (int64_t)kv_heads * page_size * row_bytes_of(dim, bits) > INT32_MAX)
    return QEMB_E_UNSUPPORTED;  // a page's bytes are counted in 32 bits
  if (batch == 0) return QEMB_OK;
  if (!q || !out || !seq_lens || !prefix_lens || (width > 0 && !block_table) || (prefix_width > 0 && !prefix_table) ||
      (pages > 0 && (!k_pages || !v_pages)))
    return QEMB_E_INVALID_ARG;
  for (const void* p : {q, k_pages, v_pages, (const void*)out, (const void*)workspace})
    if (!aligned(p, 16)) return QEMB_E_MISALIGNED;
  for (const void* p : {(const void*)block_table, (const void*)seq_lens, (const void*)prefix_table, (const void*)prefix_lens,
                        (const void*)group_offsets, (const void*)lse})
    if (!aligned(p, 4)) return QEMB_E_MISALIGNED;
  const SharedPlan plan = shared_plan(batch, q_heads, kv_heads, dim, groups, (int64_t)prefix_width * page_size, (int64_t)width * page_size, bits);
  if (!workspace) return QEMB_E_INVALID_ARG;
  SharedArgs a;
  a.q = q;
  a.pages[0] = k_pages, a.pages[1] = v_pages;
  a.n_pages = pages, a.page_log2 = log2_of(page_size), a.row_bytes = row_bytes_of(dim, bits);
  a.batch = batch, a.q_heads = q_heads, a.kv_heads = kv_heads, a.dim = dim, a.groups = groups;
  a.prefix_table = prefix_table, a.prefix_width = prefix_width, a.prefix_lens = prefix_lens;
  a.group_offsets = group_offsets, a.block_table = block_table, a.width = width, a.seq_lens = seq_lens;
  a.scale = scale;
  a.out = out, a.lse = lse, a.workspace = (float*)workspace, a.err_count = err_count;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == QEMB_DTYPE_BF16 ? launch_shared<__bf16>(a, plan, bits, st) : launch_shared<_Float16>(a, plan, bits, st);
}

int qemb_evict(const void* k_pages, const void* v_pages, int64_t pages, int32_t page_size,
               int64_t row_bytes, int32_t batch, int32_t kv_heads, const int32_t* block_table,
               int32_t width, const int32_t* seq_lens, const float* mass, int64_t mass_len,
               int32_t keep, int32_t sinks, int32_t recent, void* new_k_pages, void* new_v_pages,
               int64_t new_pages, const int32_t* new_block_table, int32_t new_width, int32_t* kept,
               float* new_mass, int64_t new_mass_len, int32_t* new_lens, int32_t* err_count,
               qemb_stream_t stream) {
  if (batch < 0 || kv_heads < 1 || pages < 0 || new_pages < 0 || width < 0 || mass_len < 0 || !is_pow2(page_size))
    return QEMB_E_INVALID_ARG;
  if (keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep || row_bytes < 16) return QEMB_E_INVALID_ARG;
  if ((int64_t)new_width * page_size < keep || new_mass_len < keep) return QEMB_E_INVALID_ARG;
  if (row_bytes % 16) return QEMB_E_MISALIGNED;
  if (row_bytes > (1 << 16) || (int64_t)width * page_size > INT32_MAX || (int64_t)new_width * page_size > INT32_MAX ||
      mass_len > INT32_MAX || new_mass_len > INT32_MAX || (int64_t)batch * kv_heads > INT32_MAX)
    return QEMB_E_UNSUPPORTED;
  if ((int64_t)width * page_size > kMostPlaces && mass_len > kMostPlaces) return QEMB_E_UNSUPPORTED;  // both bound a length
  if (batch == 0) return QEMB_OK;
  if (!seq_lens || !new_block_table || !kept || !new_mass || !new_lens || (width > 0 && (!block_table)) ||
      (mass_len > 0 && !mass) || (pages > 0 && (!k_pages || !v_pages)) || (new_pages > 0 && (!new_k_pages || !new_v_pages)))
    return QEMB_E_INVALID_ARG;
  for (const void* p : {k_pages, v_pages, (const void*)new_k_pages, (const void*)new_v_pages})
    if (!aligned(p, 16)) return QEMB_E_MISALIGNED;
  for (const void* p : {(const void*)block_table, (const void*)seq_lens, (const void*)mass, (const void*)new_block_table,
                        (const void*)kept, (const void*)new_mass, (const void*)new_lens})
    if (!aligned(p, 4)) return QEMB_E_MISALIGNED;
  EvictArgs a;
  a.pages[0] = k_pages, a.pages[1] = v_pages;
  a.new_pages[0] = new_k_pages, a.new_pages[1] = new_v_pages;
  a.n_pages = pages, a.n_new_pages = new_pages;
  a.page_log2 = log2_of(page_size), a.row_bytes = (int)row_bytes;
  a.batch = batch, a.kv_heads = kv_heads;
  a.block_table = block_table, a.width = width, a.new_block_table = new_block_table, a.new_width = new_width;
  a.seq_lens = seq_lens, a.mass = mass, a.mass_len = mass_len;
  a.keep = keep, a.sinks = sinks, a.recent = recent;
  a.kept = kept, a.new_mass = new_mass, a.new_mass_len = new_mass_len, a.new_lens = new_lens;
  a.err_count = err_count;
  return launch_evict(a, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
