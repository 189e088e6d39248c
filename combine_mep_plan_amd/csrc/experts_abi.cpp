// Host side of the router and expert calls declared in include/mep.h: argument
// checks and launches.  These calls keep no state between each other, so they
// take a config instead of a handle; every check runs before any HIP call.
#include <initializer_list>

#include "mep_internal.h"

namespace {

constexpr int32_t kMaxTokens = 1 << 26;
constexpr size_t kCounterBytes = 256;    // balance workspace: the blocks' counter

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}
bool all_aligned(std::initializer_list<const void*> ps) {  // null pointers pass
  for (const void* p : ps)
    if (!aligned(p)) return false;
  return true;
}

int hip_rc(hipError_t e) { return e == hipSuccess ? MEP_OK : MEP_ERR_HIP; }

int check_gate(const mep_gate_config* c, int32_t T) {
  if (!c) return MEP_ERR_NULL;
  if (c->num_experts < 1 || c->num_experts > mep::kMaxExperts) return MEP_ERR_CONFIG;
  if (c->top_k < 1 || c->top_k > mep::kMaxTopk || c->top_k > c->num_experts)
    return MEP_ERR_CONFIG;
  if (c->score != MEP_SCORE_SOFTMAX && c->score != MEP_SCORE_SIGMOID) return MEP_ERR_CONFIG;
  if (c->dtype != MEP_FP32 && c->dtype != MEP_BF16) return MEP_ERR_CONFIG;
  if (T < 0 || T > kMaxTokens) return MEP_ERR_SHAPE;
  return MEP_OK;
}

int check_groups(const mep_gate_config& c, int32_t groups, int32_t top, int32_t by) {
  if (groups < 1 || groups > mep::kMaxGroups || c.num_experts % groups != 0)
    return MEP_ERR_CONFIG;
  const int32_t size = c.num_experts / groups;
  if (top < 1 || top > groups || c.top_k > top * size) return MEP_ERR_CONFIG;
  if (by != MEP_GROUP_MAX && by != MEP_GROUP_TOP2) return MEP_ERR_CONFIG;
  return by == MEP_GROUP_TOP2 && size < 2 ? MEP_ERR_CONFIG : MEP_OK;
}

// What mep_gate and mep_gate_grouped share; cfg and T are checked.
int gate_args(const mep_gate_config& c, const void* logits, const float* bias, int32_t T,
              int32_t* indices, float* weights, mep::GateArgs& a) {
  if (bias && c.score != MEP_SCORE_SIGMOID) return MEP_ERR_CONFIG;
  if (T > 0 && any_null({logits, indices, weights})) return MEP_ERR_NULL;
  if (!all_aligned({logits, bias, indices, weights})) return MEP_ERR_ALIGN;
  a.logits = logits;
  a.bias = bias;
  a.indices = indices;
  a.weights = weights;
  a.T = T;
  a.E = c.num_experts;
  a.k = c.top_k;
  a.score = c.score;
  a.dtype = c.dtype;
  a.normalize = c.normalize != 0;
  a.scale = c.scale;
  return MEP_OK;
}

bool counts_fit(const mep_gate_config& c, int32_t T) {
  return (int64_t)T * c.top_k <= INT32_MAX;
}

int check_linear(const mep_linear_config* c, int64_t cap_em) {
  if (!c) return MEP_ERR_NULL;
  if (c->num_experts < 1 || c->num_experts > mep::kMaxExperts) return MEP_ERR_CONFIG;
  if (c->act < MEP_ACT_NONE || c->act > MEP_ACT_SILU_GLU) return MEP_ERR_CONFIG;
  if (c->quant != MEP_QUANT_NONE && c->quant != MEP_QUANT_FP8_E4M3_BLOCK128)
    return MEP_ERR_CONFIG;
  const int unit = c->quant == MEP_QUANT_NONE ? 8 : 128;
  for (const int32_t d : {c->in_dim, c->out_dim})
    if (d <= 0 || d % unit != 0 || d > (1 << 20)) return MEP_ERR_CONFIG;
  if (cap_em < 0 || cap_em > INT32_MAX) return MEP_ERR_SHAPE;
  return MEP_OK;
}

int32_t weight_rows(const mep_linear_config& c) {
  return c.act == MEP_ACT_SILU_GLU ? 2 * c.out_dim : c.out_dim;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t grad_z_bytes(const mep_linear_config& c, int64_t cap_em) {
  return c.act == MEP_ACT_NONE ? 0 : align256((size_t)cap_em * weight_rows(c) * 2);
}

size_t part_bytes(const mep_linear_config& c, int64_t cap_em) {
  return (size_t)((cap_em + mep::kSegRows - 1) / mep::kSegRows) * weight_rows(c) * sizeof(float);
}

}  // namespace

extern "C" {

int mep_gate(const mep_gate_config* cfg, const void* logits, const float* bias, int32_t T,
             int32_t* indices, float* weights, void* stream) {
  mep::GateArgs a{};
  int rc = check_gate(cfg, T);
  if (rc == MEP_OK) rc = gate_args(*cfg, logits, bias, T, indices, weights, a);
  return rc != MEP_OK ? rc : hip_rc(mep::launch_gate(a, (hipStream_t)stream));
}

int mep_gate_grouped(const mep_gate_config* cfg, int32_t num_groups, int32_t top_groups,
                     int32_t group_score, const void* logits, const float* bias, int32_t T,
                     int32_t* indices, float* weights, void* stream) {
  mep::GateArgs a{};
  int rc = check_gate(cfg, T);
  if (rc == MEP_OK) rc = check_groups(*cfg, num_groups, top_groups, group_score);
  if (rc == MEP_OK) rc = gate_args(*cfg, logits, bias, T, indices, weights, a);
  if (rc != MEP_OK) return rc;
  a.groups = num_groups;
  a.top_groups = top_groups;
  a.group_score = group_score;
  return hip_rc(mep::launch_gate(a, (hipStream_t)stream));
}

size_t mep_balance_workspace_bytes(const mep_gate_config* cfg, int32_t T) {
  if (check_gate(cfg, T) != MEP_OK || !counts_fit(*cfg, T)) return 0;
  const size_t rows = (size_t)mep::balance_blocks(cfg->num_experts, T);
  return kCounterBytes + align256(rows * cfg->num_experts * sizeof(float)) +
         rows * (cfg->num_experts + 1) * sizeof(int32_t);
}

int mep_balance_loss(const mep_gate_config* cfg, const void* logits, const int32_t* indices,
                     const uint8_t* token_mask, int32_t T, int32_t* counts, float* prob_mean,
                     float* loss, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_gate(cfg, T);
  if (rc != MEP_OK) return rc;
  if (!counts_fit(*cfg, T)) return MEP_ERR_SHAPE;
  if (any_null({counts, prob_mean, loss, workspace})) return MEP_ERR_NULL;
  if (T > 0 && any_null({logits, indices})) return MEP_ERR_NULL;
  if (!all_aligned({logits, indices, token_mask, counts, prob_mean, loss, workspace}))
    return MEP_ERR_ALIGN;
  if (workspace_bytes < mep_balance_workspace_bytes(cfg, T)) return MEP_ERR_SHAPE;
  const size_t rows = (size_t)mep::balance_blocks(cfg->num_experts, T);
  unsigned char* ws = (unsigned char*)workspace;
  mep::BalanceArgs a{};
  a.logits = logits;
  a.indices = indices;
  a.mask = token_mask;
  a.counts = counts;
  a.prob_mean = prob_mean;
  a.loss = loss;
  a.done = (uint32_t*)ws;
  a.part_sum = (float*)(ws + kCounterBytes);
  a.part_cnt =
      (int32_t*)(ws + kCounterBytes + align256(rows * cfg->num_experts * sizeof(float)));
  a.T = T;
  a.E = cfg->num_experts;
  a.k = cfg->top_k;
  a.score = cfg->score;
  a.dtype = cfg->dtype;
  a.coef = cfg->balance_coef;
  return hip_rc(mep::launch_balance(a, (hipStream_t)stream));
}

int mep_gate_backward(const mep_gate_config* cfg, const void* logits, const int32_t* indices,
                      const uint8_t* token_mask, int32_t T, const float* grad_weights,
                      const int32_t* counts, const float* grad_loss, void* grad_logits,
                      void* stream) {
  int rc = check_gate(cfg, T);
  if (rc != MEP_OK) return rc;
  if (!grad_weights && !counts) return MEP_ERR_NULL;
  if (!counts != !grad_loss) return MEP_ERR_NULL;
  if (T > 0 && any_null({logits, indices, grad_logits})) return MEP_ERR_NULL;
  if (!all_aligned({logits, indices, token_mask, grad_weights, counts, grad_loss, grad_logits}))
    return MEP_ERR_ALIGN;
  mep::GateBackwardArgs a{};
  a.logits = logits;
  a.indices = indices;
  a.mask = token_mask;
  a.grad_weights = grad_weights;
  a.counts = counts;
  a.grad_loss = grad_loss;
  a.grad_logits = grad_logits;
  a.T = T;
  a.E = cfg->num_experts;
  a.k = cfg->top_k;
  a.score = cfg->score;
  a.dtype = cfg->dtype;
  a.normalize = cfg->normalize != 0;
  a.scale = cfg->scale;
  a.coef = cfg->balance_coef;
  return hip_rc(mep::launch_gate_backward(a, (hipStream_t)stream));
}

int mep_expert_linear(const mep_linear_config* cfg, const void* em_x, const float* em_scales,
                      const int32_t* em_counts, const int32_t* em_offsets, int64_t cap_em,
                      int64_t num_rows, const void* w, const float* w_scales, const float* bias,
                      const void* residual, void* y, void* z, void* stream) {
  int rc = check_linear(cfg, cap_em);
  if (rc != MEP_OK) return rc;
  if (num_rows < 0) return MEP_ERR_SHAPE;
  if (any_null({em_counts, em_offsets})) return MEP_ERR_NULL;
  if (cap_em > 0 && any_null({em_x, w, y})) return MEP_ERR_NULL;
  const bool fp8 = cfg->quant != MEP_QUANT_NONE;
  if (fp8 && cap_em > 0 && any_null({em_scales, w_scales})) return MEP_ERR_NULL;
  if (!all_aligned({em_x, em_scales, em_counts, em_offsets, w, w_scales, bias, residual, y, z}))
    return MEP_ERR_ALIGN;
  mep::LinearArgs a{};
  a.x = em_x;
  a.x_scales = em_scales;
  a.w = w;
  a.w_scales = w_scales;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.z = z;
  a.counts = em_counts;
  a.offsets = em_offsets;
  a.cap = cap_em;
  a.num_rows = num_rows;
  a.E = cfg->num_experts;
  a.K = cfg->in_dim;
  a.N = cfg->out_dim;
  a.Nz = weight_rows(*cfg);
  a.act = cfg->act;
  a.quant = cfg->quant;
  return hip_rc(mep::launch_linear(a, (hipStream_t)stream));
}

size_t mep_linear_workspace_bytes(const mep_linear_config* cfg, int64_t cap_em) {
  if (check_linear(cfg, cap_em) != MEP_OK || cfg->quant != MEP_QUANT_NONE) return 0;
  const size_t n = grad_z_bytes(*cfg, cap_em) + part_bytes(*cfg, cap_em);
  return n ? n : 16;
}

int mep_expert_linear_backward(const mep_linear_config* cfg, const void* grad_y, const void* z,
                               const void* em_x, const void* w, const int32_t* em_counts,
                               const int32_t* em_offsets, int64_t cap_em, int64_t num_rows,
                               void* grad_x, void* grad_w, float* grad_bias, void* workspace,
                               size_t workspace_bytes, void* stream) {
  int rc = check_linear(cfg, cap_em);
  if (rc != MEP_OK) return rc;
  if (cfg->quant != MEP_QUANT_NONE) return MEP_ERR_CONFIG;
  if (num_rows < 0) return MEP_ERR_SHAPE;
  if (any_null({em_counts, em_offsets, workspace})) return MEP_ERR_NULL;
  if (!grad_x && !grad_w && !grad_bias) return MEP_ERR_NULL;
  if (cap_em > 0) {
    if (!grad_y || (cfg->act != MEP_ACT_NONE && !z)) return MEP_ERR_NULL;
    if ((grad_x && !w) || (grad_w && !em_x)) return MEP_ERR_NULL;
  }
  if (!all_aligned({grad_y, z, em_x, w, em_counts, em_offsets, grad_x, grad_w, grad_bias,
                    workspace}))
    return MEP_ERR_ALIGN;
  if (workspace_bytes < mep_linear_workspace_bytes(cfg, cap_em)) return MEP_ERR_SHAPE;
  unsigned char* ws = (unsigned char*)workspace;
  mep::LinearBackwardArgs a{};
  a.grad_y = grad_y;
  a.z = z;
  a.x = em_x;
  a.w = w;
  a.counts = em_counts;
  a.offsets = em_offsets;
  a.grad_x = grad_x;
  a.grad_w = grad_w;
  a.grad_bias = grad_bias;
  a.grad_z = cfg->act == MEP_ACT_NONE ? const_cast<void*>(grad_y) : ws;
  a.part = (float*)(ws + grad_z_bytes(*cfg, cap_em));
  a.cap = cap_em;
  a.num_rows = num_rows;
  a.E = cfg->num_experts;
  a.K = cfg->in_dim;
  a.N = cfg->out_dim;
  a.Nz = weight_rows(*cfg);
  a.act = cfg->act;
  return hip_rc(mep::launch_linear_backward(a, (hipStream_t)stream));
}

}  // extern "C"
