// Shared by the products' kernels: the groups' row tiles, and the activations.
#pragma once

#include "moe_internal.cuh"
#include "tensor_core.cuh"

namespace ep {

// prefix[g] = row tiles of the groups before g, prefix[E] = of all. Called by every
// thread of the CTA (a multiple of 32, at most 1024); ends with a CTA barrier. Cut
// groups latch kErrOverflow.
template <int kThreads>
__device__ __forceinline__ void build_prefix(const Groups& q, int tile_rows, int* prefix, uint32_t* err) {
  __shared__ int s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (q.E + kThreads - 1) / kThreads;
  const int g0 = min(q.E, static_cast<int>(threadIdx.x) * per), g1 = min(q.E, g0 + per);
  bool cut = false;
  int sum = 0;
  for (int g = g0; g < g1; ++g) sum += (group_rows(q, g, &cut).count + tile_rows - 1) / tile_rows;
  if (cut && err != nullptr) atomicOr(err, kErrOverflow);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  for (int g = g0; g < g1; ++g) {
    prefix[g] = before;
    before += (group_rows(q, g).count + tile_rows - 1) / tile_rows;
    if (g == q.E - 1) prefix[q.E] = before;
  }
  __syncthreads();
}

// The group that row tile `t` (< prefix[E]) belongs to.
__device__ __forceinline__ int group_of_tile(const int* prefix, int E, int t) {
  int lo = 0, hi = E;  // prefix[lo] <= t < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float sigmoid_fast(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// act(z)
template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == EP_ACT_RELU) return fmaxf(z, 0.f);
  if constexpr (kAct == EP_ACT_SILU || kAct == EP_ACT_SWIGLU) return z * sigmoid_fast(z);
  if constexpr (kAct == EP_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}

// act'(z)
template <int kAct>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (kAct == EP_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (kAct == EP_ACT_SILU || kAct == EP_ACT_SWIGLU) {
    const float s = sigmoid_fast(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if constexpr (kAct == EP_ACT_GELU)
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * (1.f + erff(z * 0.70710678118654752f)));
  return 1.f;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = bf16x2_to_f32x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                    f32x2_to_bf16x2(f[6], f[7]));
}

}  // namespace ep
