// C ABI of the router, the combine's gradient and the experts' products: argument
// checks, workspace layout, launches. Every host-detectable problem is reported
// before anything is enqueued.
#include <math.h>

#include "moe_internal.cuh"

namespace ep {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int sms_or_all(int requested) {
  const int n = device_sm_count();
  if (n <= 0) return -1;
  return (requested > 0 && requested < n) ? requested : n;
}

int check_workspace(void* ws, size_t bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || bytes < need ? EP_ERR_WORKSPACE : EP_OK;
}

int make_route(const ep_route_config_t* c, RouteGeometry* g) {
  if (c == nullptr) return EP_ERR_INVALID_ARG;
  if (c->num_segments < 1 || c->num_tokens < 0 || c->num_experts < 1) return EP_ERR_INVALID_ARG;
  if (c->num_experts > kMaxExperts) return EP_ERR_UNSUPPORTED;
  if (c->num_topk < 1 || c->num_topk > kMaxTopk || c->num_topk > c->num_experts) return EP_ERR_INVALID_ARG;
  if (c->logits_dtype != EP_DTYPE_FP32 && c->logits_dtype != EP_DTYPE_BF16) return EP_ERR_INVALID_ARG;
  if (c->score != EP_SCORE_SOFTMAX && c->score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
  if (c->normalize != 0 && c->normalize != 1) return EP_ERR_INVALID_ARG;
  if (!isfinite(c->scale)) return EP_ERR_INVALID_ARG;
  if (c->num_groups < 0) return EP_ERR_INVALID_ARG;
  const int G = c->num_groups > 1 ? c->num_groups : 1;
  if (G > 1) {
    if (c->num_experts % G != 0 || c->num_experts / G < 2) return EP_ERR_INVALID_ARG;
    if (G > kMaxGroups) return EP_ERR_UNSUPPORTED;
    if (c->topk_groups < 1 || c->topk_groups > G) return EP_ERR_INVALID_ARG;
    if (c->num_topk > c->topk_groups * (c->num_experts / G)) return EP_ERR_INVALID_ARG;
  }
  const int64_t tokens = static_cast<int64_t>(c->num_segments) * c->num_tokens;
  if (tokens > INT32_MAX / c->num_topk || c->num_segments > 1 << 20) return EP_ERR_UNSUPPORTED;
  g->B = c->num_segments;
  g->T = c->num_tokens;
  g->E = c->num_experts;
  g->K = c->num_topk;
  g->G = G;
  g->keep = G > 1 ? c->topk_groups : 1;
  g->bf16 = c->logits_dtype == EP_DTYPE_BF16;
  g->sigmoid = c->score == EP_SCORE_SIGMOID;
  g->normalize = c->normalize;
  g->scale = c->scale;
  // one token per warp at least, and no more CTAs in all than kRouteCtas (one per segment at least)
  int C = c->num_tokens / kRouteWarps + (c->num_tokens % kRouteWarps != 0);
  const int most = kRouteCtas / c->num_segments;
  if (C > most) C = most;
  g->C = C < 1 ? 1 : C;
  g->prob_shift = 62;
  while (g->prob_shift > 0 && (int64_t{1} << (62 - g->prob_shift)) <= c->num_tokens) --g->prob_shift;
  return EP_OK;
}

RouteWorkspace route_workspace(const RouteGeometry& g) {
  RouteWorkspace w;
  const size_t B = static_cast<size_t>(g.B);
  w.seg_done = 256;
  w.seg_valid = w.seg_done + round256(4 * B);
  w.seg_loss = w.seg_valid + round256(4 * B);
  w.count = w.seg_loss + round256(4 * B);
  w.prob = w.count + round256(4 * B * g.E);
  w.total = w.prob + round256(8 * B * g.E);
  return w;
}

int make_product(const ep_product_config_t* c, ProductGeometry* g) {
  if (c == nullptr) return EP_ERR_INVALID_ARG;
  if (c->num_ranks < 1 || c->num_experts < 1 || c->num_experts % c->num_ranks != 0) return EP_ERR_INVALID_ARG;
  if (c->num_experts > kMaxExperts) return EP_ERR_UNSUPPORTED;
  if (c->rows < 0 || c->num_sms < 0) return EP_ERR_INVALID_ARG;
  if (c->rows > INT32_MAX - 256) return EP_ERR_UNSUPPORTED;  // a tile past the last row still has a 32-bit index
  if (c->in_features < 8 || c->in_features % 8 != 0 || c->out_features < 8 || c->out_features % 8 != 0)
    return EP_ERR_INVALID_ARG;
  if (c->in_features > 1 << 20 || c->out_features > 1 << 20) return EP_ERR_UNSUPPORTED;
  if (c->activation < EP_ACT_NONE || c->activation > EP_ACT_SWIGLU) return EP_ERR_INVALID_ARG;
  if (c->x_dtype != EP_DTYPE_BF16 && c->x_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
  if (c->sf_pack != 0 && c->sf_pack != 1) return EP_ERR_INVALID_ARG;
  if (c->x_dtype == EP_DTYPE_FP8_E4M3 && c->in_features % 128 != 0) return EP_ERR_INVALID_ARG;
  if (c->sf_pack && c->x_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_UNSUPPORTED;
  // output tiles are numbered in 32 bits (more would not fit any GPU's memory)
  const int64_t width = 2ll * (c->in_features > c->out_features ? c->in_features : c->out_features) / 64 + 2;
  if ((c->rows / kDzRows + c->num_experts) * width > INT32_MAX ||
      (c->in_features / 256 + 1ll) * (c->out_features / 128 + 1ll) * c->num_experts > INT32_MAX)
    return EP_ERR_UNSUPPORTED;
  g->K = c->in_features;
  g->N = c->out_features;
  g->Z = c->activation == EP_ACT_SWIGLU ? 2 * c->out_features : c->out_features;
  g->act = c->activation;
  g->x_fp8 = c->x_dtype == EP_DTYPE_FP8_E4M3;
  g->sf_pack = c->sf_pack;
  g->groups = Groups{nullptr, nullptr, nullptr, c->num_experts, c->num_experts / c->num_ranks, static_cast<int>(c->rows)};
  return EP_OK;
}

struct ProductWorkspace {
  size_t done;  // uint32 [kDzCounters] in the header: tiles finished (return to 0)
  size_t rows;  // bf16 rows of FP8 x [rows][K], or dz [rows][Z]
  size_t part;  // float [tiles of kDzRows rows][Z]
  size_t total;
};

ProductWorkspace product_workspace(const ProductGeometry& g, bool grad) {
  ProductWorkspace w;
  w.done = 64;
  w.rows = 256;
  size_t bytes = 0;
  if (grad) bytes = g.act == EP_ACT_NONE ? 0 : 2 * static_cast<size_t>(g.groups.rows) * g.Z;
  else if (g.x_fp8) bytes = 2 * static_cast<size_t>(g.groups.rows) * g.K;
  w.part = w.rows + round256(bytes);
  const int64_t tiles = g.groups.rows / kDzRows + g.groups.E;
  w.total = w.part + (grad ? round256(4 * static_cast<size_t>(tiles) * g.Z) : 0);
  return w;
}

// The blocks of an expanded layout, or one group of all rows.
int set_groups(ProductGeometry* g, const ep_layout_t* layout) {
  if (layout == nullptr) return g->groups.E == 1 ? EP_OK : EP_ERR_INVALID_ARG;
  if (layout->exp_cnt == nullptr || layout->exp_base == nullptr || layout->exp_region == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned(layout->exp_cnt, 4) || !aligned(layout->exp_base, 4) || !aligned(layout->exp_region, 4))
    return EP_ERR_INVALID_ARG;
  g->groups.count = layout->exp_cnt;
  g->groups.base = layout->exp_base;
  g->groups.region = layout->exp_region;
  return EP_OK;
}

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" {

size_t ep_route_workspace_bytes(const ep_route_config_t* cfg) {
  RouteGeometry g;
  return make_route(cfg, &g) == EP_OK ? route_workspace(g).total : 0;
}

int ep_route(const ep_route_config_t* cfg, const void* logits, const float* choice_bias, const uint8_t* token_mask,
             const ep_route_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  RouteArgs a;
  int st = make_route(cfg, &a.g);
  if (st != EP_OK) return st;
  const RouteWorkspace w = route_workspace(a.g);
  if ((st = check_workspace(workspace, workspace_bytes, w.total)) != EP_OK) return st;
  if (out == nullptr) return EP_ERR_INVALID_ARG;
  const bool tokens = a.g.T > 0;
  if (tokens && (logits == nullptr || out->topk_idx == nullptr || out->topk_weights == nullptr)) return EP_ERR_INVALID_ARG;
  const int stats = (out->expert_count != nullptr) + (out->prob_sum != nullptr) + (out->num_valid != nullptr) +
                    (out->balance_loss != nullptr);
  if (stats != 0 && stats != 4) return EP_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(choice_bias, 4) || !aligned(out->topk_idx, 8) || !aligned(out->topk_weights, 4) ||
      !aligned(out->expert_count, 4) || !aligned(out->prob_sum, 4) || !aligned(out->num_valid, 4) ||
      !aligned(out->balance_loss, 4))
    return EP_ERR_INVALID_ARG;
  if (!tokens && stats == 0) return EP_OK;
  a.logits = logits;
  a.bias = choice_bias;
  a.mask = token_mask;
  a.idx = out->topk_idx;
  a.weights = out->topk_weights;
  a.count = out->expert_count;
  a.prob_sum = out->prob_sum;
  a.num_valid = out->num_valid;
  a.loss = out->balance_loss;
  a.err = at<uint32_t>(workspace, 0);
  a.done = at<uint32_t>(workspace, 4);
  a.seg_done = at<uint32_t>(workspace, w.seg_done);
  a.seg_valid = at<uint32_t>(workspace, w.seg_valid);
  a.seg_loss = at<float>(workspace, w.seg_loss);
  a.ws_count = at<uint32_t>(workspace, w.count);
  a.ws_prob = at<unsigned long long>(workspace, w.prob);
  return cuda_status(launch_route(a, static_cast<cudaStream_t>(stream)));
}

int ep_route_grad(const ep_route_config_t* cfg, const void* logits, const uint8_t* token_mask, const ep_route_t* route,
                  const float* d_weights, const float* d_loss, void* d_logits, void* workspace, size_t workspace_bytes,
                  void* stream) {
  RouteGradArgs a;
  int st = make_route(cfg, &a.g);
  if (st != EP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, route_workspace(a.g).total)) != EP_OK) return st;
  if (route == nullptr) return EP_ERR_INVALID_ARG;
  if (a.g.T == 0) return EP_OK;
  if (logits == nullptr || d_logits == nullptr || route->topk_idx == nullptr) return EP_ERR_INVALID_ARG;
  if (d_loss != nullptr && (route->expert_count == nullptr || route->num_valid == nullptr)) return EP_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(d_logits, 16) || !aligned(route->topk_idx, 8) || !aligned(d_weights, 4) ||
      !aligned(d_loss, 4) || !aligned(route->expert_count, 4) || !aligned(route->num_valid, 4))
    return EP_ERR_INVALID_ARG;
  a.logits = logits;
  a.mask = token_mask;
  a.idx = route->topk_idx;
  a.count = route->expert_count;
  a.num_valid = route->num_valid;
  a.d_weights = d_weights;
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.err = at<uint32_t>(workspace, 0);
  return cuda_status(launch_route_grad(a, static_cast<cudaStream_t>(stream)));
}

int ep_combine_grad(const ep_config_t* cfg, const ep_layout_t* layout, const uint16_t* y, const int64_t* topk_idx,
                    const float* topk_weights, const uint16_t* d_out, uint16_t* d_y, float* d_weights, void* workspace,
                    size_t workspace_bytes, void* stream) {
  Geometry g;
  int st = make_geometry(cfg, &g);
  if (st != EP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, workspace_layout(g).total)) != EP_OK) return st;
  if (layout == nullptr) return EP_ERR_INVALID_ARG;
  if (g.num_tokens == 0 || (d_y == nullptr && d_weights == nullptr)) return EP_OK;
  if (d_out == nullptr || topk_idx == nullptr || topk_weights == nullptr || (d_weights != nullptr && y == nullptr))
    return EP_ERR_INVALID_ARG;
  if (g.expand ? (layout->exp_pos == nullptr || layout->exp_region == nullptr) : layout->slot_map == nullptr)
    return EP_ERR_INVALID_ARG;
  if (g.compact && layout->recv_psum == nullptr) return EP_ERR_INVALID_ARG;
  if (g.compact == 2 && layout->recv_region == nullptr) return EP_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(d_out, 16) || !aligned(d_y, 16) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4) ||
      !aligned(d_weights, 4))
    return EP_ERR_INVALID_ARG;
  const int sms = sms_or_all(cfg->num_sms);
  if (sms < 0) return EP_ERR_CUDA;
  CombineGradArgs a = {};
  a.c.y = y;
  a.c.topk_idx = topk_idx;
  a.c.topk_w = topk_weights;
  a.c.slot_map = layout->slot_map;
  a.c.exp_pos = layout->exp_pos;
  a.c.exp_region = layout->exp_region;
  a.c.recv_psum = layout->recv_psum;
  a.c.recv_region = layout->recv_region;
  a.c.err = at<uint32_t>(workspace, workspace_layout(g).err);
  a.c.y_rows = ep_recv_rows(cfg);
  a.c.E = g.E;
  a.c.L = g.L;
  a.c.K = g.K;
  a.c.T = g.T;
  a.c.H = g.H;
  a.c.R = g.R;
  a.c.M = g.M;
  a.c.compact = g.compact;
  a.c.region_rows = g.region_rows;
  a.c.num_tokens = g.num_tokens;
  a.d_out = d_out;
  a.d_y = d_y;
  a.d_w = d_weights;
  return cuda_status(launch_combine_grad(g, a, sms, static_cast<cudaStream_t>(stream)));
}

size_t ep_product_workspace_bytes(const ep_product_config_t* cfg, int32_t grad) {
  ProductGeometry g;
  return make_product(cfg, &g) == EP_OK ? product_workspace(g, grad != 0).total : 0;
}

int ep_expert_product(const ep_product_config_t* cfg, const ep_layout_t* layout, const void* x, const float* x_sf,
                      const uint16_t* weight, const uint16_t* bias, const uint16_t* residual, uint16_t* z, uint16_t* out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  ProductArgs a;
  int st = make_product(cfg, &a.g);
  if (st != EP_OK) return st;
  const ProductWorkspace w = product_workspace(a.g, false);
  if ((st = check_workspace(workspace, workspace_bytes, w.total)) != EP_OK) return st;
  if ((st = set_groups(&a.g, layout)) != EP_OK) return st;
  if (a.g.groups.rows == 0) return EP_OK;
  if (x == nullptr || weight == nullptr || out == nullptr) return EP_ERR_INVALID_ARG;
  if ((a.g.x_fp8 != 0) != (x_sf != nullptr)) return EP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_sf, 4) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(residual, 16) ||
      !aligned(z, 16) || !aligned(out, 16))
    return EP_ERR_INVALID_ARG;
  const int sms = sms_or_all(cfg->num_sms);
  if (sms < 0) return EP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.x = static_cast<const uint16_t*>(x);
  a.x_sf = nullptr;
  if (a.g.x_fp8) {
    // a code times a power of two is exact in bf16; other scales are applied to the fp32 sums
    if (!a.g.sf_pack) a.x_sf = x_sf;
    uint16_t* rows = at<uint16_t>(workspace, w.rows);
    const cudaError_t e =
        launch_dequant(a.g, static_cast<const uint8_t*>(x), a.g.sf_pack ? x_sf : nullptr, rows, sms, s);
    if (e != cudaSuccess) return EP_ERR_CUDA;
    a.x = rows;
  }
  a.weight = weight;
  a.bias = bias;
  a.residual = residual;
  a.z = z;
  a.out = out;
  a.err = at<uint32_t>(workspace, 0);
  return cuda_status(launch_product(a, sms, s));
}

int ep_expert_product_grad(const ep_product_config_t* cfg, const ep_layout_t* layout, const uint16_t* x,
                           const uint16_t* weight, const uint16_t* z, const uint16_t* d_out, uint16_t* d_x,
                           uint16_t* d_weight, float* d_bias, void* workspace, size_t workspace_bytes, void* stream) {
  ProductGradArgs a;
  int st = make_product(cfg, &a.g);
  if (st != EP_OK) return st;
  if (a.g.x_fp8) return EP_ERR_UNSUPPORTED;
  const ProductWorkspace w = product_workspace(a.g, true);
  if ((st = check_workspace(workspace, workspace_bytes, w.total)) != EP_OK) return st;
  if ((st = set_groups(&a.g, layout)) != EP_OK) return st;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(z, 16) || !aligned(d_out, 16) || !aligned(d_x, 16) ||
      !aligned(d_weight, 16) || !aligned(d_bias, 4))
    return EP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.groups.rows == 0) {  // every sum over no rows is zero
    const size_t mats = static_cast<size_t>(a.g.groups.E) * a.g.Z;
    if (d_weight != nullptr && cudaMemsetAsync(d_weight, 0, 2 * mats * a.g.K, s) != cudaSuccess) return EP_ERR_CUDA;
    if (d_bias != nullptr && cudaMemsetAsync(d_bias, 0, 4 * mats, s) != cudaSuccess) return EP_ERR_CUDA;
    return EP_OK;
  }
  if (d_out == nullptr || (z == nullptr && a.g.act != EP_ACT_NONE) || (d_weight != nullptr && x == nullptr) ||
      (d_x != nullptr && weight == nullptr))
    return EP_ERR_INVALID_ARG;
  const int sms = sms_or_all(cfg->num_sms);
  if (sms < 0) return EP_ERR_CUDA;
  a.x = x;
  a.weight = weight;
  a.z = z;
  a.d_out = d_out;
  const bool products = d_x != nullptr || d_weight != nullptr;
  a.dz = a.g.act == EP_ACT_NONE || !products ? nullptr : at<uint16_t>(workspace, w.rows);
  a.part = d_bias != nullptr ? at<float>(workspace, w.part) : nullptr;
  a.done = at<uint32_t>(workspace, w.done);
  a.d_x = d_x;
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.err = at<uint32_t>(workspace, 0);
  if (a.dz != nullptr || a.part != nullptr) {
    const cudaError_t e = launch_product_dz(a, sms, s);
    if (e != cudaSuccess) return EP_ERR_CUDA;
  }
  if (d_x != nullptr) {
    const cudaError_t e = launch_product_dx(a, sms, s);
    if (e != cudaSuccess) return EP_ERR_CUDA;
  }
  if (d_weight != nullptr) return cuda_status(launch_product_dw(a, sms, s));
  return EP_OK;
}

}  // extern "C"
