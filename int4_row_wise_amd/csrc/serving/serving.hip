// serving.hip -- what stands around the attention in a serving loop, on gfx950.
//
// Kernels and the C ABI declared in include/qemb_serving.h:
//   * add_norm_kernel  residual addition and norm, 16 or 8 bits out (add_norm.inc)
//   * logprobs_*       log probabilities, entropies, the most likely tokens (logprobs.inc)
//
// Built without fast-math and without contraction (a packed row must round
// exactly as the range rule of qemb.h says); fused multiply-adds are written
// out where a kernel wants them.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "qemb_serving.h"

namespace {

constexpr int kWave = 64;
constexpr int kBlock = 256;
constexpr int64_t kMaxBlocks = (1 << 24) - 1;  // of kBlock threads: a launch counts threads in 32 bits

#include "../common.inc"
#include "../attention/rows.inc"
#include "add_norm.inc"
#include "logprobs.inc"

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

extern "C" {

int qemb_add_norm(const void* x, const void* residual, const void* weight, int64_t rows, int32_t dim,
                  int32_t dtype, int64_t x_stride, int64_t residual_stride, int64_t sum_stride,
                  float eps, int32_t form, int32_t group, void* out, float* scales, void* sum_out,
                  qemb_stream_t stream) {
  if (rows < 0 || dim < 1 || (dtype != QEMB_DTYPE_BF16 && dtype != QEMB_DTYPE_FP16)) return QEMB_E_INVALID_ARG;
  if (form < QEMB_FORM_VALUES || form > QEMB_FORM_ROWS8) return QEMB_E_INVALID_ARG;
  const bool scaled = form == QEMB_FORM_INT8 || form == QEMB_FORM_E4M3;
  if (group && (!scaled || group < 32 || group > 512 || (group & (group - 1)) || dim % group)) return QEMB_E_INVALID_ARG;
  if (dim > QEMB_MAX_NORM_DIM || dim % 8 || (form == QEMB_FORM_ROWS8 && dim > QEMB_MAX_DIM)) return QEMB_E_UNSUPPORTED;
  if (rows > kMaxBlocks) return QEMB_E_UNSUPPORTED;
  if (rows <= 1) x_stride = residual_stride = sum_stride = dim;
  if (x_stride < 0 || x_stride % 8 || (residual && (residual_stride < 0 || residual_stride % 8)) ||
      (sum_out && (sum_stride < dim || sum_stride % 8)))
    return QEMB_E_MISALIGNED;
  if (rows == 0) return QEMB_OK;
  if (!x || !out || (scaled && !scales)) return QEMB_E_INVALID_ARG;
  for (const void* p : {x, residual, weight, (const void*)out, (const void*)sum_out})
    if (!aligned(p, 16)) return QEMB_E_MISALIGNED;
  if (!aligned(scales, 4)) return QEMB_E_MISALIGNED;
  AddNormArgs a;
  a.x = x, a.residual = residual, a.weight = weight;
  a.rows = rows, a.dim = dim;
  a.x_stride = x_stride, a.residual_stride = residual_stride, a.sum_stride = sum_stride;
  a.eps = eps, a.group = group;
  a.out = out, a.scales = scales, a.sum_out = sum_out;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == QEMB_DTYPE_BF16 ? launch_add_norm<__bf16>(a, form, st) : launch_add_norm<_Float16>(a, form, st);
}

size_t qemb_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype, int32_t top) {
  if (rows < 1 || vocab < 1 || vocab > kMaxVocab || dtype < 0 || dtype > QEMB_DTYPE_FP32 || top < 0 || top > QEMB_MAX_TOP) return 0;
  return logprobs_plan(rows, vocab, dtype, top).bytes;
}

int qemb_token_logprobs(const void* logits, int64_t rows, int64_t vocab, int32_t dtype,
                        int64_t row_stride, const void* targets, int32_t index_type, int32_t top,
                        float* logprobs, float* entropy, float* lse, int32_t* top_ids,
                        float* top_logprobs, void* workspace, int32_t* err_count,
                        qemb_stream_t stream) {
  if (rows < 0 || vocab < 1 || dtype < 0 || dtype > QEMB_DTYPE_FP32 || top < 0 || top > QEMB_MAX_TOP) return QEMB_E_INVALID_ARG;
  if (index_type != QEMB_INDEX_INT32 && index_type != QEMB_INDEX_INT64) return QEMB_E_INVALID_ARG;
  if (vocab > kMaxVocab || rows > kMaxBlocks) return QEMB_E_UNSUPPORTED;
  if (rows <= 1) row_stride = vocab;
  if (row_stride < 0) return QEMB_E_INVALID_ARG;
  if (rows == 0) return QEMB_OK;
  if (!logits || (!targets) != (!logprobs) || (top > 0 && (!top_ids || !top_logprobs))) return QEMB_E_INVALID_ARG;
  if (!aligned(logits, dtype == QEMB_DTYPE_FP32 ? 4 : 2) || !aligned(targets, index_type == QEMB_INDEX_INT64 ? 8 : 4))
    return QEMB_E_MISALIGNED;
  for (const void* p : {(const void*)logprobs, (const void*)entropy, (const void*)lse, (const void*)top_ids, (const void*)top_logprobs})
    if (!aligned(p, 4)) return QEMB_E_MISALIGNED;
  if (!aligned(workspace, 16)) return QEMB_E_MISALIGNED;
  const LogprobsPlan plan = logprobs_plan(rows, vocab, dtype, top);
  if (plan.bytes && !workspace) return QEMB_E_INVALID_ARG;
  LogprobsArgs a;
  a.logits = logits, a.rows = rows, a.vocab = (int)vocab, a.row_stride = row_stride;
  a.targets = targets, a.idx64 = index_type == QEMB_INDEX_INT64, a.top = top;
  a.logprobs = logprobs, a.entropy = entropy, a.lse = lse, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
  a.workspace = workspace, a.err_count = err_count;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == QEMB_DTYPE_BF16   ? launch_logprobs<__bf16>(a, plan, st)
         : dtype == QEMB_DTYPE_FP16 ? launch_logprobs<_Float16>(a, plan, st)
                                    : launch_logprobs<float>(a, plan, st);
}

}  // extern "C"
