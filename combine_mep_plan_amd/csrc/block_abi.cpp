// Host side of the norms around a block and of the calls over many gradients, declared
// in include/mep.h: argument checks and launches.  No state is kept between calls; every
// check runs before any HIP call.
#include <cmath>
#include <initializer_list>

#include "mep_internal.h"

namespace {

constexpr int32_t kMaxTokens = 1 << 26;
constexpr int32_t kMaxGrads = 65536;

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool all_aligned(std::initializer_list<const void*> ps) {  // null pointers pass
  for (const void* p : ps)
    if (!aligned(p)) return false;
  return true;
}

int hip_rc(hipError_t e) { return e == hipSuccess ? MEP_OK : MEP_ERR_HIP; }

bool is_norm(int32_t kind) { return kind >= MEP_NORM_NONE && kind <= MEP_NORM_LAYER; }

int check_norm(const mep_norm_config* c, int32_t T) {
  if (!c) return MEP_ERR_NULL;
  if (c->hidden_dim <= 0 || c->hidden_dim % 8 != 0 || c->hidden_dim > mep::kMaxNormRow)
    return MEP_ERR_CONFIG;
  if (c->dtype != MEP_FP32 && c->dtype != MEP_BF16) return MEP_ERR_CONFIG;
  if (!is_norm(c->post) || !is_norm(c->pre)) return MEP_ERR_CONFIG;
  if (c->gate < MEP_BLOCK_GATE_NONE || c->gate > MEP_BLOCK_GATE_ELEMENT) return MEP_ERR_CONFIG;
  if (!(c->eps > 0.0f) || !std::isfinite(c->eps)) return MEP_ERR_CONFIG;
  if (T < 0 || T > kMaxTokens) return MEP_ERR_SHAPE;
  return MEP_OK;
}

int check_grads(const mep_grad* g, int32_t n) {
  if (n < 0 || n > kMaxGrads) return MEP_ERR_SHAPE;
  if (n > 0 && !g) return MEP_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    if (g[i].dtype != MEP_FP32 && g[i].dtype != MEP_BF16) return MEP_ERR_CONFIG;
    if (g[i].reserved != 0) return MEP_ERR_CONFIG;
    if (g[i].numel < 0 || g[i].numel > ((int64_t)1 << 44)) return MEP_ERR_SHAPE;
  }
  return MEP_OK;
}

// Calls f(table) for each launch's share of the tensors, then says how it went.
template <class F>
int by_tables(const mep_grad* g, int32_t n, F f) {
  int32_t i = 0;
  do {
    mep::GradTable t{};
    uint64_t chunks = 0;
    while (i < n && t.n < mep::kGradsALaunch) {
      const bool bf16 = g[i].dtype == MEP_BF16;
      const uint32_t c = mep::grad_chunks(g[i].numel, bf16);
      if (chunks + c > mep::kMaxChunks) break;
      if (c > 0) {
        t.data[t.n] = g[i].data;
        t.out[t.n] = g[i].out;
        t.numel_type[t.n] = 2 * g[i].numel + bf16;
        t.first[t.n++] = (uint32_t)chunks;
        chunks += c;
      }
      ++i;
    }
    t.first[t.n] = (uint32_t)chunks;
    if (const int rc = f(t); rc != MEP_OK) return rc;
  } while (i < n);
  return MEP_OK;
}

}  // namespace

extern "C" {

int mep_block_norm(const mep_norm_config* cfg, const void* x, const void* y, const void* gate,
                   const float* post_weight, const float* post_bias, const float* pre_weight,
                   const float* pre_bias, int32_t T, void* s, void* n, void* n_codes,
                   float* n_scales, void* stream) {
  int rc = check_norm(cfg, T);
  if (rc != MEP_OK) return rc;
  if (n_codes && cfg->hidden_dim % 128 != 0) return MEP_ERR_CONFIG;
  if (gate && cfg->gate == MEP_BLOCK_GATE_NONE) return MEP_ERR_CONFIG;
  if (T > 0) {
    if ((!x && !y) || (!s && !n && !n_codes)) return MEP_ERR_NULL;
    if (y ? cfg->gate != MEP_BLOCK_GATE_NONE && !gate : gate != nullptr) return MEP_ERR_NULL;
    if (!n_codes != !n_scales) return MEP_ERR_NULL;
  }
  if (!all_aligned({x, y, gate, post_weight, post_bias, pre_weight, pre_bias, s, n, n_codes,
                    n_scales}))
    return MEP_ERR_ALIGN;
  mep::NormArgs a{};
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.post_weight = post_weight;
  a.post_bias = post_bias;
  a.pre_weight = pre_weight;
  a.pre_bias = pre_bias;
  a.s = s;
  a.n = n;
  a.codes = n_codes;
  a.scales = n_scales;
  a.T = T;
  a.H = cfg->hidden_dim;
  a.dtype = cfg->dtype;
  a.post = cfg->post;
  a.pre = cfg->pre;
  // without a block there is no gate, whatever the config names: the kernels load a
  // row's factor wherever the kind says that there is one
  a.gate_kind = y ? cfg->gate : MEP_BLOCK_GATE_NONE;
  a.sigmoid = cfg->gate_sigmoid != 0;
  a.eps = cfg->eps;
  a.offset = cfg->weight_offset;
  a.residual_scale = cfg->residual_scale;
  a.block_scale = cfg->block_scale;
  return hip_rc(mep::launch_block_norm(a, (hipStream_t)stream));
}

size_t mep_block_norm_workspace_bytes(const mep_norm_config* cfg, int32_t T) {
  if (check_norm(cfg, T) != MEP_OK) return 0;
  const size_t n = (size_t)mep::norm_backward_blocks(cfg->hidden_dim, T) * 4 *
                   (size_t)cfg->hidden_dim * sizeof(float);
  return n ? n : 16;
}

int mep_block_norm_backward(const mep_norm_config* cfg, const void* grad_s, const void* grad_n,
                            const void* s, const void* y, const void* gate,
                            const float* post_weight, const float* post_bias,
                            const float* pre_weight, int32_t T, void* grad_x, void* grad_y,
                            void* grad_gate, float* grad_post_weight, float* grad_post_bias,
                            float* grad_pre_weight, float* grad_pre_bias, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int rc = check_norm(cfg, T);
  if (rc != MEP_OK) return rc;
  const bool of_block = grad_y || grad_gate || grad_post_weight || grad_post_bias;
  const bool of_pre = grad_pre_weight || grad_pre_bias;
  if ((gate || grad_gate) && cfg->gate == MEP_BLOCK_GATE_NONE) return MEP_ERR_CONFIG;
  if (!workspace || (!grad_x && !of_block && !of_pre)) return MEP_ERR_NULL;
  if (T > 0) {
    if (!grad_s && !grad_n) return MEP_ERR_NULL;
    if (grad_n ? !s : of_pre) return MEP_ERR_NULL;
    if (of_block && (!y || (cfg->gate != MEP_BLOCK_GATE_NONE && !gate))) return MEP_ERR_NULL;
  }
  if (!all_aligned({grad_s, grad_n, s, y, gate, post_weight, post_bias, pre_weight, grad_x, grad_y,
                    grad_gate, grad_post_weight, grad_post_bias, grad_pre_weight, grad_pre_bias,
                    workspace}))
    return MEP_ERR_ALIGN;
  if (workspace_bytes < mep_block_norm_workspace_bytes(cfg, T)) return MEP_ERR_SHAPE;
  mep::NormBackwardArgs a{};
  a.grad_s = grad_s;
  a.grad_n = grad_n;
  a.s = s;
  a.y = of_block ? y : nullptr;
  a.gate = gate;
  a.post_weight = post_weight;
  a.post_bias = post_bias;
  a.pre_weight = grad_n ? pre_weight : nullptr;  // else it would meet gradients of 0
  a.grad_x = grad_x;
  a.grad_y = grad_y;
  a.grad_gate = grad_gate;
  a.columns[0] = grad_post_weight;
  a.columns[1] = grad_post_bias;
  a.columns[2] = grad_pre_weight;
  a.columns[3] = grad_pre_bias;
  a.part = (float*)workspace;
  a.T = T;
  a.H = cfg->hidden_dim;
  a.dtype = cfg->dtype;
  a.post = cfg->post;
  a.pre = cfg->pre;
  a.gate_kind = cfg->gate;
  a.sigmoid = cfg->gate_sigmoid != 0;
  a.eps = cfg->eps;
  a.offset = cfg->weight_offset;
  a.residual_scale = cfg->residual_scale;
  a.block_scale = cfg->block_scale;
  return hip_rc(mep::launch_block_norm_backward(a, (hipStream_t)stream));
}

size_t mep_grad_workspace_bytes(const mep_grad* grads, int32_t n) {
  if (check_grads(grads, n) != MEP_OK) return 0;
  size_t parts = 0;
  by_tables(grads, n, [&](const mep::GradTable& t) {
    parts += (size_t)mep::grad_norm_blocks(t);
    return MEP_OK;
  });
  return parts * sizeof(double);
}

int mep_grad_norm(const mep_grad* grads, int32_t n, float* norm, void* workspace,
                  size_t workspace_bytes, void* stream) {
  int rc = check_grads(grads, n);
  if (rc != MEP_OK) return rc;
  if (!norm || !workspace) return MEP_ERR_NULL;
  for (int32_t i = 0; i < n; ++i)
    if (grads[i].numel > 0 && !grads[i].data) return MEP_ERR_NULL;
  if (!all_aligned({norm, workspace})) return MEP_ERR_ALIGN;
  for (int32_t i = 0; i < n; ++i)
    if (!aligned(grads[i].data)) return MEP_ERR_ALIGN;
  if (workspace_bytes < mep_grad_workspace_bytes(grads, n)) return MEP_ERR_SHAPE;
  double* part = (double*)workspace;
  rc = by_tables(grads, n, [&](const mep::GradTable& t) {
    const hipError_t e = mep::launch_grad_norm(t, part, (hipStream_t)stream);
    part += mep::grad_norm_blocks(t);
    return hip_rc(e);
  });
  if (rc != MEP_OK) return rc;
  return hip_rc(mep::launch_grad_join((double*)workspace, (int32_t)(part - (double*)workspace), norm,
                                      (hipStream_t)stream));
}

int mep_grad_clip(const mep_grad* grads, int32_t n, const float* norm, float max_norm,
                  void* stream) {
  int rc = check_grads(grads, n);
  if (rc != MEP_OK) return rc;
  if (!(max_norm > 0.0f)) return MEP_ERR_CONFIG;
  if (!norm) return MEP_ERR_NULL;
  for (int32_t i = 0; i < n; ++i)
    if (grads[i].numel > 0 && (!grads[i].data || !grads[i].out)) return MEP_ERR_NULL;
  if (!aligned(norm)) return MEP_ERR_ALIGN;
  for (int32_t i = 0; i < n; ++i)
    if (!all_aligned({grads[i].data, grads[i].out})) return MEP_ERR_ALIGN;
  return by_tables(grads, n, [&](const mep::GradTable& t) {
    return hip_rc(mep::launch_grad_clip(t, norm, max_norm, (hipStream_t)stream));
  });
}

}  // extern "C"
