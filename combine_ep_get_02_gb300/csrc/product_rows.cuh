// What the kernels of the rows' products share: arguments, tiles, tensor maps.
#pragma once

#include "product_common.cuh"

namespace ep {

// Warps of the epilogue, two to each quarter of the TMEM lanes, each with half of the columns. With
// scaled sums (below) four, so that a thread's 64 sums stay in registers.
constexpr int epilogue_warps(bool scaled) { return scaled ? 16 : 8; }
constexpr int rows_threads(bool scaled) { return 64 + 32 * epilogue_warps(scaled); }
constexpr int kBK = 64;       // summed index per stage: 128 bytes of bf16, one swizzle row
constexpr int kScaledBlocks = 2;  // blocks of kBK that one scale of the rows covers
constexpr int kAccColumns = 256;  // TMEM columns of each of the two accumulators
constexpr int kRaster = 16;   // row tiles that share a sweep over the columns

struct RowsArgs {
  Groups groups;
  int sum;  // length of the summed index
  Epilogue epi;
  uint32_t* err;
  const float* a_sf;  // [rows][sum / 128]: scales of A, applied to the sums; null: none
};

struct Tile {
  int g, begin, rows;  // group, first row of the tile, rows of the group from there on
  int n0;
};

// Output tiles of kRows rows x `width` columns, numbered in 32 bits.
template <int kRows>
struct Tiles {
  const Groups& q;
  const int* prefix;  // row tiles (of kRows) before each group
  int width, nt, total;
  __device__ Tiles(const Groups& groups, const int* p, int cols, int w)
      : q(groups), prefix(p), width(w), nt((cols + w - 1) / w), total(p[groups.E] * nt) {}
  // Within a group: bands of kRaster row tiles, columns in turn inside a band, so that the
  // CTAs at work share rows of A and columns of B in L2.
  __device__ Tile at(int i) const {
    const int g = group_of_tile(prefix, q.E, i / nt);
    const GroupRows rows = group_rows(q, g);
    const int mt = prefix[g + 1] - prefix[g];
    int r = i - prefix[g] * nt;
    const int band = r / (kRaster * nt);
    r -= band * kRaster * nt;
    const int height = min(kRaster, mt - band * kRaster);
    const int n = r / height;
    const int m = band * kRaster + r - n * height;
    return Tile{g, rows.begin + m * kRows, rows.count - m * kRows, n * width};
  }
};

// ---- scaled sums -----------------------------------------------------------------------
//
// FP8 rows with fp32 scales: the codes are exact in bf16, their products with 128 columns of B are
// summed in TMEM, and that sum times the row's scale is added to the thread's sums in
// registers, out = sum_g sf[r][g] * (sum over the 128 columns of g), so that nothing is
// rounded to bf16 before the end (1.7e-3 of the result's norm, its own rounding; 2.8e-3 with rows
// rounded after scaling). A warp holds 32 rows and two chunks of 32 columns of the tile:
// chunk h = its place among the four of its quarter, and chunk h + 4 (gated: h of the other half).

__device__ __forceinline__ void add_scaled(uint32_t at, float scale, float (&sum)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    float t[16];
    tmem_ld16(at + i, t);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[i + j] = fmaf(scale, t[j], sum[i + j]);
  }
}

// Takes `n` accumulators in turn, the first being number `acc`: v += scale * columns c0 on, u those
// from c1 on (negative: none). `lanes`: TMEM address of column 0 in the warp's lanes; `sf`: the
// row's first scale (null: the row does not count). arrive(b) hands accumulator b back.
// False if a wait gave up.
template <class Arrive>
__device__ __forceinline__ bool sum_scaled(uint64_t* full, uint32_t lanes, int c0, int c1, const float* sf, int n,
                                           uint32_t& acc, float (&v)[32], float (&u)[32], const volatile int* abort,
                                           Arrive arrive) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = u[j] = 0.f;
  const bool live = __any_sync(kFullMask, sf != nullptr);
  float next = sf != nullptr && n > 0 ? __ldg(sf) : 0.f;
  for (int g = 0; g < n; ++g, ++acc) {
    const float scale = next;
    if (sf != nullptr && g + 1 < n) next = __ldg(sf + g + 1);
    const uint32_t b = acc & 1u;
    const bool ok = *abort == 0 && mbar_wait_timed<false>(smem_addr(&full[b]), acc >> 1 & 1u);
    if (!__all_sync(kFullMask, ok)) return false;
    tc_fence_after();
    const uint32_t d = lanes + b * kAccColumns;
    if (live) {
      if (c0 >= 0) add_scaled(d + c0, scale, v);
      if (c1 >= 0) add_scaled(d + c1, scale, u);
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(b);
  }
  return true;
}

// Tensor maps of A (boxes of `a_rows` rows) and B: K-major boxes of `b_rows` of the output
// index, or MN-major panels of 64.
template <bool kBMn>
cudaError_t make_rows_maps(CUtensorMap* map_a, CUtensorMap* map_b, const uint16_t* A, const uint16_t* B, const RowsArgs& a,
                           int a_rows, int b_rows) {
  const uint64_t size_a[2] = {static_cast<uint64_t>(a.sum), static_cast<uint64_t>(a.groups.rows)};
  const uint32_t box_a[2] = {kBK, static_cast<uint32_t>(a_rows)};
  const cudaError_t st = make_tensor_map(map_a, A, 2, size_a, box_a);
  if (st != cudaSuccess) return st;
  const uint64_t E = static_cast<uint64_t>(a.groups.E), sum = static_cast<uint64_t>(a.sum);
  if (kBMn) {
    const uint64_t size[3] = {static_cast<uint64_t>(a.epi.cols), sum, E};
    const uint32_t box[3] = {64, kBK, 1};
    return make_tensor_map(map_b, B, 3, size, box);
  }
  const uint64_t size[3] = {sum, static_cast<uint64_t>(a.epi.z_cols), E};
  const uint32_t box[3] = {kBK, static_cast<uint32_t>(b_rows), 1};
  return make_tensor_map(map_b, B, 3, size, box);
}

// How a call with few tiles is shared out (product_split.cu), from its sizes alone: S CTAs to a
// tile, each `part` blocks of the summed index; S = 1: not at all. The parts are summed apart
// and added in their order, whatever runs them, so that results do not depend on the SMs.
struct SplitPlan {
  int S, part;
  bool narrow;  // tiles of 128 rows of B instead of 256
  int64_t tiles;
};
SplitPlan plan_rows_split(const RowsArgs& a, bool gated);  // with scales, parts are whole scales

// The three kernels: a CTA per tile of 128 rows, CTA pairs on tiles of 256 rows (both with
// tiles of `bn` rows of B), and clusters that split the summed index of a few tiles.
// The first also sums by parts of `part` blocks (0: all at once), on tiles of 128 rows of B at most.
template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_single(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int part, int num_sms,
                               cudaStream_t stream);
template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_pair(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int num_sms, cudaStream_t stream);
template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_split(const uint16_t* A, const uint16_t* B, const RowsArgs& a, const SplitPlan& plan, cudaStream_t stream);

#define EP_ROWS_INSTANCES(X)                                                                                      \
  X(EP_ACT_NONE, false, false) X(EP_ACT_RELU, false, false) X(EP_ACT_SILU, false, false) X(EP_ACT_GELU, false, false) \
  X(EP_ACT_SWIGLU, false, false) X(EP_ACT_NONE, true, false) X(EP_ACT_NONE, false, true) X(EP_ACT_RELU, false, true) \
  X(EP_ACT_SILU, false, true) X(EP_ACT_GELU, false, true) X(EP_ACT_SWIGLU, false, true)

}  // namespace ep
