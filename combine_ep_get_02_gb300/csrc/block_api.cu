// C ABI of the norm, of activations kept in 8 bits and of the experts' layer of a few tokens: argument
// checks, workspace layout, launches. Every host-detectable problem is reported before anything
// is enqueued.
#include "block_internal.cuh"

namespace ep {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int check_workspace(void* ws, size_t bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || bytes < need ? EP_ERR_WORKSPACE : EP_OK;
}

int check_norm(const ep_norm_config_t* c) {
  if (c == nullptr) return EP_ERR_INVALID_ARG;
  if (c->rows < 0 || c->hidden < 8 || c->hidden % 8 != 0) return EP_ERR_INVALID_ARG;
  if (c->rows > INT32_MAX || c->hidden > kNormMaxHidden) return EP_ERR_UNSUPPORTED;
  if (c->x_dtype != EP_DTYPE_BF16 && c->x_dtype != EP_DTYPE_FP32) return EP_ERR_INVALID_ARG;
  if (c->sf_pack != 0 && c->sf_pack != 1) return EP_ERR_INVALID_ARG;
  if (!(c->eps >= kNormMinEps && c->eps <= kNormMaxEps)) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

size_t norm_workspace(const ep_norm_config_t* c) {
  return 256 + round256(sizeof(float) * kNormGradCtas * static_cast<size_t>(c->hidden));
}

int make_checkpoint(const ep_checkpoint_config_t* c, Groups* g) {
  if (c == nullptr) return EP_ERR_INVALID_ARG;
  if (c->num_ranks < 1 || c->num_experts < 1 || c->num_experts % c->num_ranks != 0) return EP_ERR_INVALID_ARG;
  if (c->num_experts > kMaxExperts) return EP_ERR_UNSUPPORTED;
  if (c->rows < 0 || c->features < 128 || c->features % 128 != 0) return EP_ERR_INVALID_ARG;
  if (c->rows > INT32_MAX - 256 || c->features > 1 << 21) return EP_ERR_UNSUPPORTED;
  if (c->activation < EP_ACT_NONE || c->activation > EP_ACT_SWIGLU) return EP_ERR_INVALID_ARG;
  if (c->sf_pack != 0 && c->sf_pack != 1) return EP_ERR_INVALID_ARG;
  *g = Groups{nullptr, nullptr, nullptr, c->num_experts, c->num_experts / c->num_ranks, static_cast<int>(c->rows)};
  return EP_OK;
}

size_t checkpoint_workspace(const ep_checkpoint_config_t* c) {
  const int64_t tiles = c->rows / kDzRows + c->num_experts;
  return 256 + round256(sizeof(float) * static_cast<size_t>(tiles) * c->features);
}

int set_blocks(Groups* g, const ep_layout_t* layout) {
  if (layout == nullptr) return g->E == 1 ? EP_OK : EP_ERR_INVALID_ARG;
  if (layout->exp_cnt == nullptr || layout->exp_base == nullptr || layout->exp_region == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned(layout->exp_cnt, 4) || !aligned(layout->exp_base, 4) || !aligned(layout->exp_region, 4))
    return EP_ERR_INVALID_ARG;
  g->count = layout->exp_cnt;
  g->base = layout->exp_base;
  g->region = layout->exp_region;
  return EP_OK;
}

int checkpoint(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const void* in, void* out, float* sf, bool back,
               void* workspace, size_t workspace_bytes, void* stream) {
  CheckpointArgs a;
  int st = make_checkpoint(cfg, &a.groups);
  if (st != EP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, checkpoint_workspace(cfg))) != EP_OK) return st;
  if ((st = set_blocks(&a.groups, layout)) != EP_OK) return st;
  if (cfg->rows == 0) return EP_OK;
  if (in == nullptr || out == nullptr || sf == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned(in, 16) || !aligned(out, 16) || !aligned(sf, 4)) return EP_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return EP_ERR_CUDA;
  a.F = cfg->features;
  a.sf_pack = cfg->sf_pack;
  a.in = in;
  a.out = out;
  a.sf = sf;
  a.err = at<uint32_t>(workspace, 0);
  return cuda_status(launch_checkpoint(a, back, sms, static_cast<cudaStream_t>(stream)));
}

int check_layer(const ep_layer_config_t* c) {
  if (c == nullptr) return EP_ERR_INVALID_ARG;
  if (c->num_tokens < 0 || c->num_experts < 1 || c->num_topk < 1 || c->num_sms < 0) return EP_ERR_INVALID_ARG;
  if (c->num_tokens > kLayerMaxTokens || c->num_experts > kMaxExperts || c->num_topk > kMaxTopk) return EP_ERR_UNSUPPORTED;
  if (c->activation < EP_ACT_NONE || c->activation > EP_ACT_SWIGLU) return EP_ERR_INVALID_ARG;
  if (c->weight_dtype != EP_DTYPE_BF16 && c->weight_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
  const int unit = c->weight_dtype == EP_DTYPE_FP8_E4M3 ? 128 : 8;
  if (c->hidden < unit || c->hidden % unit != 0 || c->inner < unit || c->inner % unit != 0) return EP_ERR_INVALID_ARG;
  if (c->hidden > 1 << 20 || c->inner > 1 << 20) return EP_ERR_UNSUPPORTED;
  return EP_OK;
}

struct LayerWorkspace {
  size_t done, h, part, total;
};

LayerWorkspace layer_workspace(const ep_layer_config_t* c) {
  LayerWorkspace w;
  const size_t T = static_cast<size_t>(c->num_tokens);
  w.done = 256;
  w.h = w.done + round256(sizeof(uint32_t) * ((c->hidden + 15) / 16));
  w.part = w.h + round256((c->num_tokens <= kLayerPairTokens ? 4 : 2) * T * c->num_topk * c->inner);
  w.total = w.part + round256(sizeof(float) * kLayerMaxSplit * T * c->hidden);
  return w;
}

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" {

size_t ep_norm_workspace_bytes(const ep_norm_config_t* cfg) { return check_norm(cfg) == EP_OK ? norm_workspace(cfg) : 0; }

int ep_norm(const ep_norm_config_t* cfg, const void* x, const void* residual, const uint16_t* weight, void* sum,
            uint16_t* y, uint8_t* codes, float* sf, void* stream) {
  const int st = check_norm(cfg);
  if (st != EP_OK) return st;
  if (codes != nullptr && cfg->hidden % 128 != 0) return EP_ERR_INVALID_ARG;
  if (cfg->rows == 0) return EP_OK;
  if ((codes != nullptr) != (sf != nullptr) || (y == nullptr && codes == nullptr)) return EP_ERR_INVALID_ARG;
  if (x == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(y, 16) ||
      !aligned(codes, 16) || !aligned(sf, 4))
    return EP_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return EP_ERR_CUDA;
  const NormArgs a = {x, residual, weight, sum, y, codes, sf, cfg->rows, cfg->hidden, cfg->sf_pack, cfg->eps};
  return cuda_status(launch_norm(a, cfg->x_dtype == EP_DTYPE_FP32, sms, static_cast<cudaStream_t>(stream)));
}

int ep_norm_grad(const ep_norm_config_t* cfg, const void* sum, const uint16_t* weight, const uint8_t* token_mask,
                 const uint16_t* d_y, const void* d_sum, void* d_x, float* d_weight, void* workspace,
                 size_t workspace_bytes, void* stream) {
  int st = check_norm(cfg);
  if (st != EP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, norm_workspace(cfg))) != EP_OK) return st;
  if (!aligned(sum, 16) || !aligned(weight, 16) || !aligned(d_y, 16) || !aligned(d_sum, 16) || !aligned(d_x, 16) ||
      !aligned(d_weight, 4))
    return EP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->rows == 0)  // the sum over no rows
    return d_weight == nullptr ? EP_OK : cuda_status(cudaMemsetAsync(d_weight, 0, sizeof(float) * cfg->hidden, s));
  if (d_x == nullptr && d_weight == nullptr) return EP_OK;
  if (sum == nullptr || d_y == nullptr) return EP_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return EP_ERR_CUDA;
  const NormGradArgs a = {sum, weight, token_mask, d_y, d_sum, d_x, d_weight,
                          d_weight == nullptr ? nullptr : at<float>(workspace, 256), at<uint32_t>(workspace, 0), cfg->rows, cfg->hidden, cfg->eps};
  return cuda_status(launch_norm_grad(a, cfg->x_dtype == EP_DTYPE_FP32, sms, s));
}

size_t ep_checkpoint_workspace_bytes(const ep_checkpoint_config_t* cfg) {
  Groups g;
  return make_checkpoint(cfg, &g) == EP_OK ? checkpoint_workspace(cfg) : 0;
}

int ep_checkpoint(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint16_t* x, uint8_t* codes, float* sf,
                  void* workspace, size_t workspace_bytes, void* stream) {
  return checkpoint(cfg, layout, x, codes, sf, false, workspace, workspace_bytes, stream);
}

int ep_checkpoint_rows(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const float* sf,
                       uint16_t* x, void* workspace, size_t workspace_bytes, void* stream) {
  return checkpoint(cfg, layout, codes, x, const_cast<float*>(sf), true, workspace, workspace_bytes, stream);
}

int ep_checkpoint_grad(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const float* sf,
                       const uint16_t* d_h, uint16_t* h, uint16_t* d_z, float* d_bias, void* workspace,
                       size_t workspace_bytes, void* stream) {
  CheckpointGradArgs a;
  int st = make_checkpoint(cfg, &a.groups);
  if (st != EP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, checkpoint_workspace(cfg))) != EP_OK) return st;
  if ((st = set_blocks(&a.groups, layout)) != EP_OK) return st;
  if (!aligned(codes, 16) || !aligned(sf, 4) || !aligned(d_h, 16) || !aligned(h, 16) || !aligned(d_z, 16) ||
      !aligned(d_bias, 4))
    return EP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->rows == 0)  // every sum over no rows is zero
    return d_bias == nullptr
               ? EP_OK
               : cuda_status(cudaMemsetAsync(d_bias, 0, sizeof(float) * static_cast<size_t>(cfg->num_experts) * cfg->features, s));
  if (h == nullptr && d_z == nullptr && d_bias == nullptr) return EP_OK;
  if (codes == nullptr || sf == nullptr || d_h == nullptr) return EP_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return EP_ERR_CUDA;
  a.Z = cfg->features;
  a.N = cfg->activation == EP_ACT_SWIGLU ? cfg->features / 2 : cfg->features;
  a.act = cfg->activation;
  a.sf_pack = cfg->sf_pack;
  a.codes = codes;
  a.sf = sf;
  a.d_h = d_h;
  a.h = h;
  a.d_z = d_z;
  a.part = d_bias == nullptr ? nullptr : at<float>(workspace, 256);
  a.done = at<uint32_t>(workspace, 64);
  a.d_bias = d_bias;
  a.err = at<uint32_t>(workspace, 0);
  return cuda_status(launch_checkpoint_grad(a, sms, s));
}

size_t ep_layer_workspace_bytes(const ep_layer_config_t* cfg) {
  return check_layer(cfg) == EP_OK ? layer_workspace(cfg).total : 0;
}

int ep_expert_layer(const ep_layer_config_t* cfg, const uint16_t* x, const int64_t* topk_idx, const float* topk_weights,
                    const void* up, const float* up_sf, const uint16_t* up_bias, const void* down, const float* down_sf,
                    const uint16_t* down_bias, const uint16_t* residual, uint16_t* out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_layer(cfg);
  if (st != EP_OK) return st;
  const LayerWorkspace w = layer_workspace(cfg);
  if ((st = check_workspace(workspace, workspace_bytes, w.total)) != EP_OK) return st;
  if (cfg->num_tokens == 0) return EP_OK;
  if (x == nullptr || topk_idx == nullptr || topk_weights == nullptr || up == nullptr || down == nullptr || out == nullptr)
    return EP_ERR_INVALID_ARG;
  const bool fp8 = cfg->weight_dtype == EP_DTYPE_FP8_E4M3;
  if (fp8 != (up_sf != nullptr) || fp8 != (down_sf != nullptr)) return EP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4) || !aligned(up, 16) || !aligned(up_sf, 4) ||
      !aligned(up_bias, 16) || !aligned(down, 16) || !aligned(down_sf, 4) || !aligned(down_bias, 16) ||
      !aligned(residual, 16) || !aligned(out, 16))
    return EP_ERR_INVALID_ARG;
  LayerArgs a;
  a.device_sms = device_sm_count();
  if (a.device_sms <= 0) return EP_ERR_CUDA;
  const int sms = cfg->num_sms > 0 && cfg->num_sms < a.device_sms ? cfg->num_sms : a.device_sms;
  a.x = x;
  a.idx = topk_idx;
  a.w = topk_weights;
  a.up = up;
  a.up_sf = up_sf;
  a.up_bias = up_bias;
  a.down = down;
  a.down_sf = down_sf;
  a.down_bias = down_bias;
  a.residual = residual;
  a.out = out;
  a.h = at<uint16_t>(workspace, w.h);
  a.part = at<float>(workspace, w.part);
  a.done = at<uint32_t>(workspace, w.done);
  a.err = at<uint32_t>(workspace, 0);
  a.T = cfg->num_tokens;
  a.E = cfg->num_experts;
  a.K = cfg->num_topk;
  a.H = cfg->hidden;
  a.I = cfg->inner;
  a.Z = cfg->activation == EP_ACT_SWIGLU ? 2 * cfg->inner : cfg->inner;
  a.act = cfg->activation;
  return cuda_status(launch_layer(a, fp8, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
