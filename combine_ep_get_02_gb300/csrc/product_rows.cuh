// What the kernels of the rows' products share: arguments, tiles, tensor maps.
#pragma once

#include "product_common.cuh"

namespace ep {

constexpr int kEpilogueWarps = 8;  // two to each quarter of the TMEM lanes, each with half of the columns
constexpr int kRowsThreadsTc = 64 + 32 * kEpilogueWarps;
constexpr int kBK = 64;       // summed index per stage: 128 bytes of bf16, one swizzle row
constexpr int kRaster = 16;   // row tiles that share a sweep over the columns

struct RowsArgs {
  Groups groups;
  int sum;  // length of the summed index
  Epilogue epi;
  uint32_t* err;
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
SplitPlan plan_rows_split(const RowsArgs& a, bool gated);

// The three kernels: a CTA per tile of 128 rows, CTA pairs on tiles of 256 rows (both with
// tiles of `bn` rows of B), and clusters that split the summed index of a few tiles.
// The first also sums by parts of `part` blocks (0: all at once), on tiles of 128 rows of B at most.
template <int kAct, bool kBMn>
cudaError_t launch_rows_single(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int part, int num_sms,
                               cudaStream_t stream);
template <int kAct, bool kBMn>
cudaError_t launch_rows_pair(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int num_sms, cudaStream_t stream);
template <int kAct, bool kBMn>
cudaError_t launch_rows_split(const uint16_t* A, const uint16_t* B, const RowsArgs& a, const SplitPlan& plan, cudaStream_t stream);

#define EP_ROWS_INSTANCES(X) \
  X(EP_ACT_NONE, false) X(EP_ACT_RELU, false) X(EP_ACT_SILU, false) X(EP_ACT_GELU, false) X(EP_ACT_SWIGLU, false) X(EP_ACT_NONE, true)

}  // namespace ep
