// Gradient of the combine: out[t] = sum_k w_k y[row_k] gives, for the gradient g of out[t],
//   dw_k = <g, y[row_k]>  and  dy[row] = (sum of w_k over the lanes of t on that row) g.
//
// A row belongs to one token (in the row form the lanes of a token to one rank share
// it), so every row of dy is written once, by the token's unit, and nothing is added
// across units. Reading g and the rows of y and writing the rows of dy is what it
// cannot do without, and memory bounds it; the multiply-adds are 3 per column and row.
// Measured: 16 x 1024 tokens of 7168, shared rows, 513 us (3.2 GB, 6.3 TB/s); per-expert
// rows of 64 x 512 tokens of 2048, 360 us (2.3 GB, 6.4 TB/s); one token of 7168 6 us.
//
// `ways` warps take a token (one, when there are tokens for every warp of the GPU; up to the
// eight of a CTA when there are few, so that a token's columns load at once); lane k finds
// the row of top-k lane k, and the lowest lane of those that share a row stands for it.
// Each lane holds 8 columns of g per step and streams the distinct rows past them; the K
// dot products stay in registers in 32 bits to the end of the token and are summed across
// the warp once, then over the token's warps in their order. Up to 16 top-k lanes the rows in
// flight fit the registers; with 17 to 32 a thread takes 255 of them and spills 240 bytes.
#include "ep_device.cuh"
#include "moe_internal.cuh"

namespace ep {

namespace {

constexpr int kWarps = kCopyThreads / 32;

template <bool kExpand, int kMaxK>
__global__ void __launch_bounds__(kCopyThreads) combine_grad_kernel(CombineGradArgs ga, int ways) {
  const CombineArgs& a = ga.c;
  __shared__ int64_t s_row[kWarps][kMaxK];
  __shared__ float s_w[kWarps][kMaxK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float s_dot[kWarps][kMaxK];
  const int nchunk = a.H >> 3;  // 8 bf16 per chunk
  const int per_cta = kWarps / ways, way = warp % ways;
  pdl_launch_dependents();
  pdl_wait();

  // the CTA's warps go round together: they meet where a token's dot products are joined
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * per_cta; base < a.num_tokens;
       base += static_cast<int64_t>(gridDim.x) * per_cta) {
    const int64_t tok = base + warp / ways;
    int64_t row = -1;
    float w = 0.f;
    if (lane < a.K && tok < a.num_tokens) {
      const int64_t i = tok * a.K + lane;
      const int64_t e = __ldg(a.topk_idx + i);
      const int r = __ldg((kExpand ? a.exp_pos : a.slot_map) + i);
      w = __ldg(a.topk_w + i);
      if (e >= 0 && e < a.E && r >= 0) {
        const int d = static_cast<int>(e) / a.L;
        row = kExpand ? static_cast<int64_t>(a.exp_region[d]) + r : entry_row(a, d, r, a.err);
        if (!row_usable(row, a.y_rows, a.compact == 2, a.err)) row = -1;
      }
    }
    // lanes on the same row: the lowest stands for all, with the sum of their weights in lane order
    const unsigned same = __match_any_sync(kFullMask, row);
    const int leader = __ffs(same) - 1;
    float w_sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const float wk = __shfl_sync(kFullMask, w, k);
      if (same >> k & 1u) w_sum += wk;
    }
    if (lane < kMaxK) {
      s_row[warp][lane] = leader == lane ? row : -1;
      s_w[warp][lane] = w_sum;
    }
    __syncwarp();
    int64_t at[kMaxK];
    float wk[kMaxK], dot[kMaxK];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
      at[k] = s_row[warp][k];
      wk[k] = s_w[warp][k];
      dot[k] = 0.f;
    }
    const uint16_t* grow = ga.d_out + tok * a.H;
    for (int c = way * 32 + lane; tok < a.num_tokens && c < nchunk; c += 32 * ways) {
      const size_t col = static_cast<size_t>(c) << 3;
      const uint4 gv = ld_stream16(grow + col);
      uint4 yv[kMaxK];
      if (ga.d_w != nullptr) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
          if (at[k] >= 0) yv[k] = ld_stream16(a.y + at[k] * a.H + col);
      }
      const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
      float g[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_f32x2(gw[i]);
        g[2 * i] = f.x;
        g[2 * i + 1] = f.y;
      }
#pragma unroll
      for (int k = 0; k < kMaxK; ++k) {
        if (at[k] < 0) continue;
        if (ga.d_w != nullptr) {
          const uint32_t v[4] = {yv[k].x, yv[k].y, yv[k].z, yv[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f32x2(v[i]);
            dot[k] = fmaf(f.x, g[2 * i], dot[k]);
            dot[k] = fmaf(f.y, g[2 * i + 1], dot[k]);
          }
        }
        if (ga.d_y != nullptr) {
          uint4 o;
          o.x = f32x2_to_bf16x2(wk[k] * g[0], wk[k] * g[1]);
          o.y = f32x2_to_bf16x2(wk[k] * g[2], wk[k] * g[3]);
          o.z = f32x2_to_bf16x2(wk[k] * g[4], wk[k] * g[5]);
          o.w = f32x2_to_bf16x2(wk[k] * g[6], wk[k] * g[7]);
          st16(ga.d_y + at[k] * a.H + col, o);
        }
      }
    }
    if (ga.d_w != nullptr) {
      float mine = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxK; ++k) {
#pragma unroll
        for (int o = 16; o; o >>= 1) dot[k] += __shfl_xor_sync(kFullMask, dot[k], o);
        if (lane == k) mine = dot[k];
      }
      if (ways > 1) {
        if (lane < kMaxK) s_dot[warp][lane] = mine;
        __syncthreads();
        mine = 0.f;
        if (lane < kMaxK)
          for (int i = 0; i < ways; ++i) mine += s_dot[warp - way + i][lane];
        __syncthreads();
      }
      mine = __shfl_sync(kFullMask, mine, leader);
      if (way == 0 && lane < a.K && tok < a.num_tokens) ga.d_w[tok * a.K + lane] = row >= 0 ? mine : 0.f;
    }
    __syncwarp();  // s_row / s_w are rewritten by the next token
  }
}

template <bool kExpand, int kMaxK>
cudaError_t launch_one(const CombineGradArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = combine_grad_kernel<kExpand, kMaxK>;
  int per_sm = resident_ctas(reinterpret_cast<const void*>(kern), kCopyThreads, 0);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  // warps a token: enough for the warps of 152 SMs at two CTAs each (a constant, so that results
  // do not depend on the device), and no more than sweeps of 32 chunks in a row
  int ways = 1;
  while (ways < kWarps && a.c.num_tokens * ways * 2 <= 152 * 2 * kWarps && a.c.H / 8 >= ways * 32 * 2) ways *= 2;
  const int64_t per_cta = kWarps / ways;
  int64_t ctas = static_cast<int64_t>(num_sms) * per_sm;
  const int64_t need = (a.c.num_tokens + per_cta - 1) / per_cta;
  if (ctas > need) ctas = need;
  if (ctas < 1) return cudaSuccess;
  return launch_chained(kern, dim3(static_cast<unsigned>(ctas)), dim3(kCopyThreads), 0, stream, a, ways);
}

}  // namespace

cudaError_t launch_combine_grad(const Geometry& g, const CombineGradArgs& a, int num_sms, cudaStream_t stream) {
  if (g.K <= 8) return g.expand ? launch_one<true, 8>(a, num_sms, stream) : launch_one<false, 8>(a, num_sms, stream);
  if (g.K <= 16) return g.expand ? launch_one<true, 16>(a, num_sms, stream) : launch_one<false, 16>(a, num_sms, stream);
  return g.expand ? launch_one<true, 32>(a, num_sms, stream) : launch_one<false, 32>(a, num_sms, stream);
}

}  // namespace ep
