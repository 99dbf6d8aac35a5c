// layer_api.cu -- the extern "C" entry points of the router, the gated
// activation, the experts' products and their 8-bit forms (declared and
// documented in include/moe.h): argument validation on the host, then the launches.
#include <math.h>

#include "moe_internal.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int check_route(const moe_route_desc_t* d, moe::RouteParams* p) {
  if (!d) return MOE_ERR_INVALID_ARG;
  const int E = d->num_experts, G = d->num_groups;
  if (d->num_tokens < 0 || E < 1 || E > MOE_MAX_EXPERTS || d->topk < 1 || d->topk > MOE_MAX_TOPK || G < 1 ||
      G > MOE_MAX_GROUPS)
    return MOE_ERR_SHAPE;
  if (E % G || d->topk_groups < 1 || d->topk_groups > G || d->topk > d->topk_groups * (E / G)) return MOE_ERR_SHAPE;
  if ((int64_t)d->num_tokens * d->topk >= ((int64_t)1 << 31)) return MOE_ERR_SHAPE;
  if (d->logits_stride != 0 && d->logits_stride < E) return MOE_ERR_SHAPE;
  if ((d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID) ||
      (d->group_score != MOE_GROUP_MAX && d->group_score != MOE_GROUP_TOP2_SUM) ||
      (d->logits_kind != MOE_LOGITS_F32 && d->logits_kind != MOE_LOGITS_BF16) || !isfinite(d->scale))
    return MOE_ERR_INVALID_ARG;
  p->num_tokens = d->num_tokens;
  p->num_experts = E;
  p->topk = d->topk;
  p->num_groups = G;
  p->topk_groups = d->topk_groups;
  p->score = d->score;
  p->group_score = d->group_score;
  p->renormalize = d->renormalize != 0;
  p->logits_kind = d->logits_kind;
  p->stride = d->logits_stride ? d->logits_stride : E;
  p->scale = d->scale;
  return MOE_OK;
}

int check_glu(const moe_glu_desc_t* d, const int32_t* num_rows, moe::GluParams* p) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->rows < 0 || d->rows >= ((int64_t)1 << 31) || d->width < 8 || d->width > 65536 || d->width % 8)
    return MOE_ERR_SHAPE;
  if (!aligned(num_rows, 4)) return MOE_ERR_ALIGNMENT;
  p->num_rows = num_rows;
  p->rows = d->rows;
  p->width = d->width;
  return MOE_OK;
}

// Checks that every expert call shares. out_rows: rows of w per expert.
int check_expert(const moe_expert_desc_t* d, const int32_t* row_begin, const int32_t* row_end,
                 moe::ExpertParams* p) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->num_experts < 1 || d->num_experts > MOE_MAX_EXPERTS) return MOE_ERR_SHAPE;
  if (d->rows < 0 || d->rows >= ((int64_t)1 << 31) - 128) return MOE_ERR_SHAPE;
  if (d->in_features < 8 || d->in_features > 65536 || d->in_features % 8) return MOE_ERR_SHAPE;
  if (d->out_features < 8 || d->out_features > 65536 || d->out_features % 8) return MOE_ERR_SHAPE;
  if (d->x_stride != 0 && (d->x_stride < d->in_features || d->x_stride % 8 || d->x_stride >= ((int64_t)1 << 36)))
    return MOE_ERR_SHAPE;
  if (!row_begin || !row_end) return MOE_ERR_INVALID_ARG;
  if (!aligned(row_begin, 4) || !aligned(row_end, 4)) return MOE_ERR_ALIGNMENT;
  p->row_begin = row_begin;
  p->row_end = row_end;
  p->rows = d->rows;
  p->x_stride = d->x_stride ? d->x_stride : d->in_features;
  p->num_experts = d->num_experts;
  p->in_features = d->in_features;
  p->out_features = d->out_features;
  return MOE_OK;
}

int check_quant(const moe_quant_desc_t* d, const int32_t* num_rows, moe::QuantParams* p) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->rows < 0 || d->rows >= ((int64_t)1 << 31) || d->width < 16 || d->width > 65536 || d->width % 16)
    return MOE_ERR_SHAPE;
  if (d->x_stride != 0 && (d->x_stride < d->width || d->x_stride % 8 || d->x_stride >= ((int64_t)1 << 36)))
    return MOE_ERR_SHAPE;
  if (d->scale_stride != 0 && d->scale_stride != 1 && d->scale_stride != 4) return MOE_ERR_SHAPE;
  if (d->x_kind != MOE_ROWS_BF16 && d->x_kind != MOE_ROWS_F32) return MOE_ERR_INVALID_ARG;
  if (!aligned(num_rows, 4)) return MOE_ERR_ALIGNMENT;
  p->num_rows = num_rows;
  p->rows = d->rows;
  p->x_stride = d->x_stride ? d->x_stride : d->width;
  p->width = d->width;
  p->x_kind = d->x_kind;
  p->scale_stride = d->scale_stride == 4 ? 4 : 1;
  return MOE_OK;
}

int check_expert_i8(const moe_expert_i8_desc_t* d, const void* x, const float* x_scales, const int32_t* row_begin,
                    const int32_t* row_end, const void* w, const float* w_scales, void* out, moe::ExpertI8Params* p) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->num_experts < 1 || d->num_experts > MOE_MAX_EXPERTS) return MOE_ERR_SHAPE;
  if (d->rows < 0 || d->rows >= ((int64_t)1 << 31) - 128) return MOE_ERR_SHAPE;
  if (d->in_features < 16 || d->in_features > 65536 || d->in_features % 16) return MOE_ERR_SHAPE;
  if (d->out_features < 8 || d->out_features > 65536 || d->out_features % 8) return MOE_ERR_SHAPE;
  if (d->x_stride != 0 && (d->x_stride < d->in_features || d->x_stride % 16 || d->x_stride >= ((int64_t)1 << 36)))
    return MOE_ERR_SHAPE;
  if (d->x_scale_stride < 0 || d->x_scale_stride >= ((int64_t)1 << 36)) return MOE_ERR_SHAPE;
  if (!row_begin || !row_end) return MOE_ERR_INVALID_ARG;
  if (!aligned(row_begin, 4) || !aligned(row_end, 4)) return MOE_ERR_ALIGNMENT;
  p->rows = d->rows;
  if (p->rows == 0) return MOE_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4))
    return MOE_ERR_ALIGNMENT;
  p->row_begin = row_begin;
  p->row_end = row_end;
  p->x = (const int8_t*)x;
  p->x_scales = x_scales;
  p->w = (const int8_t*)w;
  p->w_scales = w_scales;
  p->out = (uint8_t*)out;
  p->x_stride = d->x_stride ? d->x_stride : d->in_features;
  p->x_scale_stride = d->x_scale_stride ? d->x_scale_stride : 1;
  p->num_experts = d->num_experts;
  p->in_features = d->in_features;
  p->out_features = d->out_features;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route(const moe_route_desc_t* desc, const void* logits, const float* bias, int32_t* topk_idx,
              float* topk_weights, moe_stream_t stream) {
  moe::RouteParams p = {};
  int rc = check_route(desc, &p);
  if (rc != MOE_OK || p.num_tokens == 0) return rc;
  if (!logits || !topk_idx || !topk_weights) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, p.logits_kind == MOE_LOGITS_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_weights, 4))
    return MOE_ERR_ALIGNMENT;
  p.logits = logits;
  p.bias = bias;
  p.topk_idx = topk_idx;
  p.topk_weights = topk_weights;
  return cuda_status(moe::launch_route(p, (cudaStream_t)stream));
}

int moe_route_backward(const moe_route_desc_t* desc, const void* logits, const int32_t* topk_idx,
                       const float* grad_weights, void* grad_logits, moe_stream_t stream) {
  moe::RouteParams p = {};
  int rc = check_route(desc, &p);
  if (rc != MOE_OK || p.num_tokens == 0) return rc;
  if (!logits || !topk_idx || !grad_weights || !grad_logits) return MOE_ERR_INVALID_ARG;
  const uintptr_t a = p.logits_kind == MOE_LOGITS_BF16 ? 2 : 4;
  if (!aligned(logits, a) || !aligned(grad_logits, a) || !aligned(topk_idx, 4) || !aligned(grad_weights, 4))
    return MOE_ERR_ALIGNMENT;
  p.logits = logits;
  p.topk_idx = const_cast<int32_t*>(topk_idx);
  p.grad_weights = grad_weights;
  p.grad_logits = grad_logits;
  return cuda_status(moe::launch_route_backward(p, (cudaStream_t)stream));
}

int moe_swiglu(const moe_glu_desc_t* desc, const int32_t* num_rows, const void* gate_up, void* act, void* ckpt,
               float* ckpt_scales, moe_stream_t stream) {
  moe::GluParams p = {};
  int rc = check_glu(desc, num_rows, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!gate_up || (!act && !ckpt) || !ckpt != !ckpt_scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(gate_up, 16) || !aligned(act, 16) || !aligned(ckpt, 8) || !aligned(ckpt_scales, 4))
    return MOE_ERR_ALIGNMENT;
  p.gate_up = (const uint8_t*)gate_up;
  p.act = (uint8_t*)act;
  p.ckpt = (uint8_t*)ckpt;
  p.scales = ckpt_scales;
  return cuda_status(moe::launch_swiglu(p, (cudaStream_t)stream));
}

int moe_swiglu_backward(const moe_glu_desc_t* desc, const int32_t* num_rows, const void* ckpt,
                        const float* ckpt_scales, const void* grad_act, void* grad_gate_up, void* act,
                        moe_stream_t stream) {
  moe::GluParams p = {};
  int rc = check_glu(desc, num_rows, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!ckpt || !ckpt_scales || !grad_act || !grad_gate_up) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_act, 16) || !aligned(grad_gate_up, 16) || !aligned(act, 16) || !aligned(ckpt, 8) ||
      !aligned(ckpt_scales, 4))
    return MOE_ERR_ALIGNMENT;
  p.ckpt = (uint8_t*)const_cast<void*>(ckpt);
  p.scales = const_cast<float*>(ckpt_scales);
  p.grad_act = (const uint8_t*)grad_act;
  p.grad_gate_up = (uint8_t*)grad_gate_up;
  p.act = (uint8_t*)act;
  return cuda_status(moe::launch_swiglu_backward(p, (cudaStream_t)stream));
}

int moe_expert_product(const moe_expert_desc_t* desc, const void* x, const int32_t* row_begin,
                       const int32_t* row_end, const void* w, void* y, moe_stream_t stream) {
  moe::ExpertParams p = {};
  int rc = check_expert(desc, row_begin, row_end, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16)) return MOE_ERR_ALIGNMENT;
  p.x = (const uint8_t*)x;
  p.w = (const uint8_t*)w;
  p.out = (uint8_t*)y;
  return cuda_status(moe::launch_expert_product(p, (cudaStream_t)stream));
}

int moe_expert_swiglu(const moe_expert_desc_t* desc, const void* x, const int32_t* row_begin,
                      const int32_t* row_end, const void* w, void* act, void* ckpt, float* ckpt_scales,
                      moe_stream_t stream) {
  moe::ExpertParams p = {};
  int rc = check_expert(desc, row_begin, row_end, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!x || !w || !act || !ckpt != !ckpt_scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(act, 16) || !aligned(ckpt, 8) || !aligned(ckpt_scales, 4))
    return MOE_ERR_ALIGNMENT;
  p.x = (const uint8_t*)x;
  p.w = (const uint8_t*)w;
  p.out = (uint8_t*)act;
  p.ckpt = (uint8_t*)ckpt;
  p.scales = ckpt_scales;
  return cuda_status(moe::launch_expert_swiglu(p, (cudaStream_t)stream));
}

int moe_expert_product_backward_input(const moe_expert_desc_t* desc, const void* grad_y,
                                      const int32_t* row_begin, const int32_t* row_end, const void* w,
                                      void* grad_x, moe_stream_t stream) {
  moe::ExpertParams p = {};
  int rc = check_expert(desc, row_begin, row_end, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!grad_y || !w || !grad_x) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_y, 16) || !aligned(w, 16) || !aligned(grad_x, 16)) return MOE_ERR_ALIGNMENT;
  p.x = (const uint8_t*)grad_y;
  p.w = (const uint8_t*)w;
  p.out = (uint8_t*)grad_x;
  return cuda_status(moe::launch_expert_grad_input(p, (cudaStream_t)stream));
}

int moe_expert_product_backward_weight(const moe_expert_desc_t* desc, const void* grad_y, const void* x,
                                       const int32_t* row_begin, const int32_t* row_end, void* grad_w,
                                       int grad_kind, moe_stream_t stream) {
  moe::ExpertParams p = {};
  int rc = check_expert(desc, row_begin, row_end, &p);
  if (rc != MOE_OK) return rc;
  if (grad_kind != MOE_GRAD_BF16 && grad_kind != MOE_GRAD_F32 && grad_kind != MOE_GRAD_F32_ADD)
    return MOE_ERR_INVALID_ARG;
  if (!grad_w || (p.rows > 0 && (!grad_y || !x))) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_y, 16) || !aligned(x, 16) || !aligned(grad_w, 16)) return MOE_ERR_ALIGNMENT;
  p.x = (const uint8_t*)grad_y;
  p.x2 = (const uint8_t*)x;
  p.out = (uint8_t*)grad_w;
  p.grad_kind = grad_kind;
  if (p.rows == 0) {  // no row anywhere: every expert's gradient is zero
    if (grad_kind == MOE_GRAD_F32_ADD) return MOE_OK;
    const size_t bytes = (size_t)p.num_experts * p.in_features * p.out_features * (grad_kind == MOE_GRAD_BF16 ? 2 : 4);
    return cuda_status(cudaMemsetAsync(grad_w, 0, bytes, (cudaStream_t)stream));
  }
  return cuda_status(moe::launch_expert_grad_weight(p, (cudaStream_t)stream));
}

int moe_quantize_rows(const moe_quant_desc_t* desc, const int32_t* num_rows, const void* x, int8_t* q, float* scales,
                      moe_stream_t stream) {
  moe::QuantParams p = {};
  int rc = check_quant(desc, num_rows, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  if (!x || !q || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, p.scale_stride == 4 ? 16 : 4)) return MOE_ERR_ALIGNMENT;
  p.x = (const uint8_t*)x;
  p.q = q;
  p.scales = scales;
  return cuda_status(moe::launch_quantize(p, (cudaStream_t)stream));
}

int moe_expert_product_i8(const moe_expert_i8_desc_t* desc, const int8_t* x, const float* x_scales, const int32_t* row_begin,
                          const int32_t* row_end, const int8_t* w, const float* w_scales, void* y, moe_stream_t stream) {
  moe::ExpertI8Params p = {};
  int rc = check_expert_i8(desc, x, x_scales, row_begin, row_end, w, w_scales, y, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  return cuda_status(moe::launch_expert_product_i8(p, (cudaStream_t)stream));
}

int moe_expert_swiglu_i8(const moe_expert_i8_desc_t* desc, const int8_t* x, const float* x_scales, const int32_t* row_begin,
                         const int32_t* row_end, const int8_t* w, const float* w_scales, void* act, moe_stream_t stream) {
  moe::ExpertI8Params p = {};
  int rc = check_expert_i8(desc, x, x_scales, row_begin, row_end, w, w_scales, act, &p);
  if (rc != MOE_OK || p.rows == 0) return rc;
  return cuda_status(moe::launch_expert_swiglu_i8(p, (cudaStream_t)stream));
}

}  // extern "C"
