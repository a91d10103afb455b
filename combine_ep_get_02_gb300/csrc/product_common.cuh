// Shared by the products' kernels: the groups' row tiles, and the activations.
#pragma once

#include "moe_internal.cuh"
#include "tensor_core.cuh"

namespace ep {

// prefix[g] = row tiles of the groups before g, prefix[E] = of all. Called by every
// thread of the CTA (a multiple of 32, at most 1024); ends with a CTA barrier. Cut
// groups latch kErrOverflow. Blocks that lie apart never need more than max_row_tiles, which
// the workspace and the tiles' numbering count on; of blocks that overlap (a layout of
// another configuration) the tiles past that are left out and latch it too.
template <int kThreads>
__device__ __forceinline__ void build_prefix(const Groups& q, int tile_rows, int* prefix, uint32_t* err) {
  __shared__ int s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (q.E + kThreads - 1) / kThreads;
  const int g0 = min(q.E, static_cast<int>(threadIdx.x) * per), g1 = min(q.E, g0 + per);
  const int most = static_cast<int>(max_row_tiles(q, tile_rows));  // below 2^26, as tiles have 64 rows at least
  bool cut = false;
  auto add = [&](int a, int b) {
    cut = cut || a + b > most;
    return min(a + b, most);
  };
  int sum = 0;
  for (int g = g0; g < g1; ++g) sum = add(sum, (group_rows(q, g, &cut).count + tile_rows - 1) / tile_rows);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl = add(incl, v);
  }
  if (lane == 31) s_warp[warp] = incl;
  int before = __shfl_up_sync(kFullMask, incl, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = add(before, s_warp[w]);
  for (int g = g0; g < g1; ++g) {
    prefix[g] = before;
    before = add(before, (group_rows(q, g).count + tile_rows - 1) / tile_rows);
    if (g == q.E - 1) prefix[q.E] = before;
  }
  if (cut && err != nullptr) atomicOr(err, kErrOverflow);
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

// the larger; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// act(z); a NaN stays one
template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == EP_ACT_RELU) return max_nan(z, 0.f);
  if constexpr (kAct == EP_ACT_SILU || kAct == EP_ACT_SWIGLU) return z * sigmoid_fast(z);
  if constexpr (kAct == EP_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}

// act'(z); NaN of a NaN
template <int kAct>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (kAct == EP_ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
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

// ---- rows between registers and memory ------------------------------------------------
//
// An accumulator row lives in one thread, 32 columns at a time; a warp holds 32 rows. To
// touch memory in whole 64-byte pieces of rows they pass through 2 KB of shared memory per
// warp (16-byte chunks, XOR-permuted so that neither side has bank conflicts); a store
// straight from the registers writes 16 bytes to each of 32 rows at once and took about
// twice as long on the shortest sums.

constexpr int kPatchBytes = 32 * 64;

__device__ __forceinline__ uint32_t patch_at(uint32_t patch, int row, int chunk) {
  return patch + row * 64 + ((chunk ^ (row >> 1 & 3)) << 4);
}
__device__ __forceinline__ void st_shared16(uint32_t p, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}

// The warp's 32 x 32 values to `dst` (its row 0, column 0; rows `stride` apart), rounded to
// bf16: the first `rows` rows, the first `cols` (a multiple of 8) columns.
__device__ __forceinline__ void store_rows(uint32_t patch, const float (&v)[32], uint16_t* dst, int64_t stride, int rows,
                                           int cols, int lane) {
#pragma unroll
  for (int c = 0; c < 4; ++c) st_shared16(patch_at(patch, lane, c), pack8(v + 8 * c));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), c = lane & 3;
    const uint4 w = ld_shared16(patch_at(patch, r, c));
    if (r < rows && c * 8 < cols) st16(dst + r * stride + c * 8, w);
  }
  __syncwarp();
}

// The same rows and columns of a tensor, in flight in the order they are read ...
struct RowsInFlight {
  uint4 v[4];
};
__device__ __forceinline__ RowsInFlight fetch_rows(const uint16_t* src, int64_t stride, int rows, int cols, int lane) {
  RowsInFlight f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), c = lane & 3;
    f.v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && c * 8 < cols) f.v[i] = *reinterpret_cast<const uint4*>(src + r * stride + c * 8);
  }
  return f;
}
// ... and added to the thread's row.
__device__ __forceinline__ void add_rows(uint32_t patch, const RowsInFlight& f, float (&v)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) st_shared16(patch_at(patch, i * 8 + (lane >> 2), lane & 3), f.v[i]);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[8];
    unpack8(ld_shared16(patch_at(patch, lane, c)), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * c + j] += x[j];
  }
  __syncwarp();
}

// What a product does with its sums.
struct Epilogue {
  const uint16_t* bias;      // [E][z_cols] or null
  const uint16_t* residual;  // [rows][cols] or null
  uint16_t* z;               // [rows][z_cols] or null
  uint16_t* out;             // [rows][cols]
  int cols, z_cols;
};

// 32 columns n0.. of a warp's 32 rows row0.. of group g, `rows` of which count: v the sums
// (gated: u those of the other half), n0 < cols; fewer than 32 with `width` (a multiple of 8).
template <int kAct>
__device__ __forceinline__ void finish_rows(const Epilogue& e, uint32_t patch, float (&v)[32],
                                            float (&u)[kAct == EP_ACT_SWIGLU ? 32 : 1], int g, int64_t row0, int rows,
                                            int n0, int lane, int width = 32) {
  constexpr bool kGated = kAct == EP_ACT_SWIGLU;
  const int cols = min(width, e.cols - n0);
  RowsInFlight res;
  if (e.residual != nullptr) res = fetch_rows(e.residual + row0 * e.cols + n0, e.cols, rows, cols, lane);
  if (e.bias != nullptr) {
    const uint16_t* b = e.bias + static_cast<int64_t>(g) * e.z_cols + n0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c * 8 >= cols) break;
      float f[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(b + c * 8)), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * c + j] += f[j];
      if constexpr (kGated) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(b + e.cols + c * 8)), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[8 * c + j] += f[j];
      }
    }
  }
  if (e.z != nullptr) {
    store_rows(patch, v, e.z + row0 * e.z_cols + n0, e.z_cols, rows, cols, lane);
    if constexpr (kGated) store_rows(patch, u, e.z + row0 * e.z_cols + e.cols + n0, e.z_cols, rows, cols, lane);
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = activate<kAct>(v[j]);
    if constexpr (kGated) v[j] *= u[j];
  }
  if (e.residual != nullptr) add_rows(patch, res, v, lane);
  store_rows(patch, v, e.out + row0 * e.cols + n0, e.cols, rows, cols, lane);
}

}  // namespace ep
