// Internal declarations of the router, the combine's gradient and the experts'
// products: what stands beside the dispatch and combine of ep_internal.cuh.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ep_get.h"
#include "ep_internal.cuh"

namespace ep {

constexpr uint32_t kErrNonfinite = 16u;  // a NaN or +inf logit or choice bias

// ---- router -------------------------------------------------------------------

constexpr int kRouteThreads = 256;  // 8 warps, a token each
constexpr int kRouteWarps = kRouteThreads / 32;
// CTAs of a router launch, shared evenly by the segments (at least one each): four
// per SM on 152 SMs. A constant, so that the order in which the probabilities are
// summed, and with it every result, does not depend on the device.
constexpr int kRouteCtas = 608;
constexpr int kMaxGroups = 32;

struct RouteGeometry {
  int B, T, E, K, G, keep;
  int bf16, sigmoid, normalize;
  float scale;
  int C;           // CTAs per segment
  int prob_shift;  // 62 bits hold a segment's sum of probabilities in units of 2^-prob_shift
};

// Byte offsets of the router's workspace: the 256-byte header (error word at 0,
// counter of finished segments at 4), then the pieces below, all of which return to 0, so that
// a workspace serves calls of other sizes too.
struct RouteWorkspace {
  size_t seg_done;   // uint32 [B]: CTAs of each segment that have delivered
  size_t seg_valid;  // uint32 [B]: valid tokens
  size_t seg_loss;   // float [B]
  size_t count;      // uint32 [B][E]: lanes
  size_t prob;       // uint64 [B][E]: probabilities in units of 2^-prob_shift
  size_t total;
};

struct RouteArgs {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int64_t* idx;
  float* weights;
  int32_t* count;     // null: no statistics
  float* prob_sum;
  int32_t* num_valid;
  float* loss;
  uint32_t* err;
  uint32_t* done;
  uint32_t* seg_done;
  uint32_t* seg_valid;
  float* seg_loss;
  uint32_t* ws_count;
  unsigned long long* ws_prob;
  RouteGeometry g;
};

struct RouteGradArgs {
  const void* logits;
  const uint8_t* mask;
  const int64_t* idx;
  const int32_t* count;
  const int32_t* num_valid;
  const float* d_weights;  // may be null
  const float* d_loss;     // may be null
  void* d_logits;
  uint32_t* err;
  RouteGeometry g;
};

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t stream);

// ---- gradient of the combine -----------------------------------------------------

struct CombineGradArgs {
  CombineArgs c;          // y, routing and layout as the combine reads them (out unused)
  const uint16_t* d_out;  // [R][T][H]
  uint16_t* d_y;          // rows of y; may be null
  float* d_w;             // [R][T][K]; may be null
};

cudaError_t launch_combine_grad(const Geometry& g, const CombineGradArgs& a, int num_sms, cudaStream_t stream);

// ---- experts' products ------------------------------------------------------------

// Groups of rows: group g's rows are [begin(g), begin(g) + count(g)) of a tensor of
// `rows` rows. From an expanded layout (count != null), or one group of all rows.
struct Groups {
  const int32_t* count;   // [R][L]
  const int32_t* base;    // [R][L+1]
  const int32_t* region;  // [R+1]
  int E, L;
  int rows;
};

struct GroupRows {
  int begin, count;
};

// A block that leaves the tensor (a layout of another configuration) is cut to it.
__device__ __forceinline__ GroupRows clip_rows(const Groups& q, int64_t begin, int n, bool* cut) {
  if (n >= 0 && begin >= 0 && begin + n <= q.rows) return GroupRows{static_cast<int>(begin), n};
  *cut = true;
  if (n <= 0 || begin < 0 || begin >= q.rows) return GroupRows{0, 0};
  return GroupRows{static_cast<int>(begin), static_cast<int>(q.rows - begin)};
}
__device__ __forceinline__ GroupRows group_rows(const Groups& q, int g, bool* cut = nullptr) {
  if (q.count == nullptr) return GroupRows{0, q.rows};
  const int d = g / q.L;  // block g starts at entry g + d of the [R][L+1] block starts
  bool over = false;
  const GroupRows r = clip_rows(q, static_cast<int64_t>(__ldg(q.region + d)) + __ldg(q.base + g + d), __ldg(q.count + g), &over);
  if (over && cut != nullptr) *cut = true;
  return r;
}

struct ProductGeometry {
  Groups groups;
  int K, N, Z;  // columns of x, of out, and of z (Z = 2 N when gated)
  int act, x_fp8, sf_pack;
};

struct ProductArgs {
  ProductGeometry g;
  const uint16_t* x;        // bf16 rows (of an FP8 dispatch: its values, or its codes if x_sf is set)
  const float* x_sf;        // [rows][K / 128] scales of the codes' sums; null: none
  const uint16_t* weight;   // [E][Z][K]
  const uint16_t* bias;     // [E][Z] or null
  const uint16_t* residual; // [rows][N] or null
  uint16_t* z;              // [rows][Z] or null
  uint16_t* out;            // [rows][N]
  uint32_t* err;
};

struct ProductGradArgs {
  ProductGeometry g;
  const uint16_t* x;
  const uint16_t* weight;
  const uint16_t* z;
  const uint16_t* d_out;
  uint16_t* dz;       // workspace [rows][Z]; null when the activation is none (dz = d_out)
  float* part;        // workspace [tiles of kDzRows rows][Z]: column sums of dz; null without d_bias
  uint32_t* done;     // workspace [kDzCounters]: tiles whose sums are in part (return to 0)
  uint16_t* d_x;      // may be null
  uint16_t* d_weight; // may be null
  float* d_bias;      // may be null
  uint32_t* err;
};

constexpr int kTileRows = 128;  // rows a CTA's products take at once
constexpr int kDzRows = 64;     // rows whose dz is summed to one partial bias gradient
constexpr int kDzColumns = 128; // output columns a CTA takes there
constexpr int kDzCounters = 48; // of finished tiles, in the last 192 bytes of the workspace's header
// Row tiles of all groups together, at most: whole ones and one part of every group that
// has a row.
__host__ __device__ inline int64_t max_row_tiles(const Groups& q, int tile_rows = kTileRows) {
  const int64_t groups = q.count == nullptr ? 1 : q.E < q.rows ? q.E : q.rows;
  return q.rows / tile_rows + groups;
}

// x_sf: packed powers of two; null: the codes alone
cudaError_t launch_dequant(const ProductGeometry& g, const uint8_t* x, const float* x_sf, uint16_t* out, int num_sms,
                           cudaStream_t stream);
cudaError_t launch_product(const ProductArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_product_dz(const ProductGradArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_product_dx(const ProductGradArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_product_dw(const ProductGradArgs& a, int num_sms, cudaStream_t stream);

}  // namespace ep
