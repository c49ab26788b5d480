// draft_fp4.cu -- the draft LM head kept in 4 bits and the ranking of its logits in one call: the
// features are quantised (quantize.cu), multiplied (fp4_linear.cu) and the bf16 logits ranked
// (draft.cu).  The head is what such a call reads: 0.28 GB instead of 1.05 GB for 128256 x 4096.
#include "fp4.cuh"

namespace svk {

namespace {

struct DraftFp4Layout {
  size_t codes, scales, logits, total;
  int64_t pitch;
};

DraftFp4Layout draft_fp4_layout(int32_t R, int32_t V, int32_t d, spec_fp4_format format) {
  DraftFp4Layout L{};
  L.pitch = ((int64_t)V + 7) / 8 * 8;
  L.codes = 0;
  L.scales = align_up(spec_fp4_code_bytes(R, d), 256);
  L.logits = align_up(L.scales + spec_fp4_scale_bytes(R, d, format), 256);
  L.total = align_up(L.logits + (size_t)R * (size_t)L.pitch * 2, 256);
  return L;
}

}  // namespace

}  // namespace svk

using namespace svk;

extern "C" size_t spec_draft_fused_fp4_workspace_size(int32_t R, int32_t V, int32_t d, int32_t k,
                                                      spec_fp4_format format) {
  if (R < 1 || V < 1 || d < 1 || k < 1 || k > 32 || k > V || V > SPEC_MAX_VOCAB || R > SPEC_FP4_MAX_DIM ||
      d > SPEC_FP4_MAX_DIM || (format != SPEC_FP4_MX && format != SPEC_FP4_NV))
    return 0;
  return draft_fp4_layout(R, V, d, format).total;
}

extern "C" int spec_draft_topk_fused_fp4(const void* features, float feature_scale, const void* w_codes,
                                         const void* w_scales, spec_fp4_format format,
                                         float weight_scale, int32_t d, int32_t R, int32_t V, int32_t k,
                                         float temperature, void* out_logits, int64_t logits_pitch,
                                         int32_t* out_tokens, float* out_probs, int32_t* out_status,
                                         void* workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (format != SPEC_FP4_MX && format != SPEC_FP4_NV) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (R < 0 || V < 1 || d < 1 || k < 1 || k > 32 || k > V) return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_VOCAB || R > SPEC_FP4_MAX_DIM || d > SPEC_FP4_MAX_DIM) return SPEC_ERR_TOO_LARGE;
  if (!(temperature > 0.0f) || !(temperature <= 3.402823466e38f)) return SPEC_ERR_INVALID_ARG;
  if (!fp4_tensor_scale_ok(feature_scale) || !(weight_scale > 0.0f) ||
      (format == SPEC_FP4_MX && (feature_scale != 1.0f || weight_scale != 1.0f)))
    return SPEC_ERR_INVALID_ARG;
  // the scales' product, 24 bits times a power of two, has to be a float: beyond the largest all
  // logits would be infinite, below the smallest all 0
  const double alpha = (double)feature_scale * (double)weight_scale;
  if (!(alpha <= 3.402823466e38) || (double)(float)alpha != alpha) return SPEC_ERR_INVALID_ARG;
  if (R == 0) return SPEC_OK;
  if (!features || !w_codes || !w_scales || !out_tokens || !out_probs || !workspace)
    return SPEC_ERR_INVALID_ARG;
  const uintptr_t all = reinterpret_cast<uintptr_t>(features) | reinterpret_cast<uintptr_t>(w_codes) |
                        reinterpret_cast<uintptr_t>(w_scales);
  if ((all & 15u) || d % 8 != 0) return SPEC_ERR_MISALIGNED;
  if (out_logits) {
    if (logits_pitch < V) return SPEC_ERR_INVALID_ARG;
    if (logits_pitch > INT64_MAX / 16) return SPEC_ERR_TOO_LARGE;
    if ((reinterpret_cast<uintptr_t>(out_logits) & 15u) || (logits_pitch * 2) % 16 != 0)
      return SPEC_ERR_MISALIGNED;
  }
  const DraftFp4Layout L = draft_fp4_layout(R, V, d, format);
  if (workspace_bytes < (out_logits ? L.logits : L.total)) return SPEC_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return SPEC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  void* logits = out_logits ? out_logits : static_cast<void*>(ws + L.logits);
  const int64_t pitch = out_logits ? logits_pitch : L.pitch;
  int rc = spec_fp4_quantize(features, SPEC_BF16, R, d, d, format, feature_scale, ws + L.codes,
                             ws + L.scales, stream);
  if (rc == SPEC_OK)
    rc = spec_fp4_linear(ws + L.codes, ws + L.scales, w_codes, w_scales, format, R, V, d, (float)alpha,
                         logits, SPEC_BF16, pitch, stream);
  if (rc == SPEC_OK)
    rc = spec_draft_topk(logits, SPEC_BF16, R, V, pitch, k, temperature, out_tokens, out_probs,
                         out_status, stream);
  return rc;
}
