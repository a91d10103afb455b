// The experts' products on the tensor cores: every group's rows times its matrix,
//   acc[r][n] = sum_k A[r][k] B_g[n][k],   r in group g,
// with bias, activation and residual applied to the fp32 sums before the one rounding
// (forward: A = x, B = W), or plain (gradient of the rows: A = dz, B = W transposed, read
// in place as an MN-major operand).
//
// A CTA per SM walks over output tiles of 128 rows x 256 columns (128 or 64 when there are few). Warp 0 brings tiles
// of A and B (64 of the summed index at a time) into a ring of shared-memory stages by
// TMA, one thread of warp 1 issues tcgen05.mma into one of two TMEM accumulators, and
// warps 2-9 take the other accumulator through the epilogue meanwhile. Row tiles start
// at each group's first row, so a tile's last rows may belong to the next group: they are
// computed and not stored (an output row depends on its own row of A alone). Columns past
// the tensors read as zero.
//
// It serves groups too short for pairs of CTAs (product_pair.cu); there reading B bounds it.
// Measured: 64 experts with 8 rows on average, 4096 -> 2 x 2048, 305-316 us (2.15 GB of
// matrices, 6.8-7.0 TB/s); 48 experts with a few rows, 4376 -> 256, 31 us.
//
// Every wait is bounded; one that gives up latches kErrTimeout, lets the CTA's copies
// and products finish and returns.
#include "product_rows.cuh"

namespace ep {

namespace {

constexpr int kBM = kTileRows, kMaxBN = kAccColumns;
constexpr int kLowRows = 32;  // tiles with no more rows read that many of A
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxStages = 8;
constexpr int ring_bytes(bool scaled) { return scaled ? 180224 : 196608; }  // the more warps, the more patches

__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn * kBK * 2; }
__host__ __device__ constexpr int stage_count(int ring, int bn) {
  return ring / stage_bytes(bn) < kMaxStages ? ring / stage_bytes(bn) : kMaxStages;
}

// kParts: a tile's sum is taken `part` blocks at a time, as the clusters of product_split.cu do
// it. The epilogue warps add each part to the sum of those before, which lies in the half of TMEM
// that accumulators of 128 columns leave, and finish the tile after the last. It runs
// the calls that are allowed fewer SMs than those clusters take.
constexpr int kSumColumn = 128;
// v += the sum kept at `at` (0 before the first part), which goes back there unless v is the last
__device__ __forceinline__ void add_part(uint32_t at, float (&v)[32], bool first, bool last) {
  float sum[32];
  if (!first) {
    tmem_ld32(at, sum);
    tmem_ld_wait();
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = (first ? 0.f : sum[j]) + v[j];
  if (!last) {
    tmem_st32(at, v);
    tmem_st_wait();
  }
}

// kScaled: scaled sums (product_rows.cuh), an accumulator per scale.
template <int kAct, bool kBMn, bool kParts, bool kScaled>
__global__ void __launch_bounds__(rows_threads(kScaled), 1)
    rows_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_low,
                const __grid_constant__ CUtensorMap map_b, RowsArgs a, int bn, int part) {
  constexpr bool kGated = kAct == EP_ACT_SWIGLU;
  constexpr int kThreads = rows_threads(kScaled), kEpilogueWarps = epilogue_warps(kScaled), kRingBytes = ring_bytes(kScaled);
  const int cols = kGated ? bn / 2 : bn;  // output columns of a tile
  const int b_bytes = bn * kBK * 2;
  const uint32_t kStages = static_cast<uint32_t>(stage_count(kRingBytes, bn)), kStageBytes = static_cast<uint32_t>(stage_bytes(bn));
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_acc_full[2], s_acc_empty[2], s_drained;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage0 = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t patch0 = stage0 + kRingBytes;
  int* prefix = reinterpret_cast<int*>(s_raw + (patch0 - smem_addr(s_raw)) + kEpilogueWarps * kPatchBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init_count(smem_addr(&s_full[s]), 1);
      mbar_init_count(smem_addr(&s_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_count(smem_addr(&s_acc_full[i]), 1);
      mbar_init_count(smem_addr(&s_acc_empty[i]), kEpilogueWarps);
    }
    mbar_init_count(smem_addr(&s_drained), 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_low);
    tma_prefetch_map(&map_b);
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  build_prefix<kThreads>(a.groups, kBM, prefix, blockIdx.x == 0 ? a.err : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Tiles<kBM> tiles(a.groups, prefix, a.epi.cols, cols);
  const int blocks = (a.sum + kBK - 1) / kBK;
  const int parts = kParts ? (blocks + part - 1) / part : 1;
  auto give_up = [&] {
    s_abort = 1;
    atomicOr(a.err, kErrTimeout);
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t n = 0;  // stages filled so far
      bool ok = true;
      for (int i = blockIdx.x; ok && i < tiles.total; i += gridDim.x) {
        const Tile t = tiles.at(i);
        const bool low = t.rows <= kLowRows;
        const uint32_t bytes = static_cast<uint32_t>(b_bytes + (low ? kLowRows * kBK * 2 : kABytes));
        for (int kb = 0; kb < blocks; ++kb, ++n) {
          const uint32_t s = n % kStages, bar = smem_addr(&s_full[s]);
          if (s_abort || !mbar_wait_timed(smem_addr(&s_empty[s]), (n / kStages & 1u) ^ 1u)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          mbar_expect(bar, bytes);
          const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
          tma_load_2d(sa, low ? &map_low : &map_a, kb * kBK, t.begin, bar);
          if constexpr (kBMn) {
            for (int p = 0; p < bn / 64; ++p)
              tma_load_3d(sb + p * (kBK * 128), &map_b, t.n0 + p * 64, kb * kBK, t.g, bar);
          } else {
            tma_load_3d(sb, &map_b, kb * kBK, t.n0, t.g, bar);
            tma_load_3d(sb + b_bytes / 2, &map_b, kb * kBK, kGated ? a.epi.cols + t.n0 : t.n0 + bn / 2, t.g, bar);
          }
        }
      }
      if (!ok)  // the copies in flight land before the CTA's memory goes
        for (uint32_t back = n < kStages ? n : kStages; back > 0; --back) {
          const uint32_t m = n - back;
          mbar_wait_timed(smem_addr(&s_full[m % kStages]), m / kStages & 1u);
        }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16(kBM, bn, false, kBMn);
      uint32_t n = 0, acc = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < tiles.total; i += gridDim.x) {
        for (int p = 0; ok && p < (kScaled ? blocks / kScaledBlocks : parts); ++p, ++acc) {
          const uint32_t b = acc & 1u;
          if (s_abort || !mbar_wait_timed(smem_addr(&s_acc_empty[b]), (acc >> 1 & 1u) ^ 1u)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * kMaxBN;
          const int each = kScaled ? kScaledBlocks : part;  // blocks of an accumulator
          const int k0 = kScaled || kParts ? p * each : 0, k1 = kScaled || kParts ? min(blocks, k0 + each) : blocks;
          for (int kb = k0; kb < k1; ++kb, ++n) {
            const uint32_t s = n % kStages;
            if (s_abort || !mbar_wait_timed(smem_addr(&s_full[s]), n / kStages & 1u)) {
              if (!s_abort) give_up();
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
            const uint64_t da = desc_k_major(sa);
            const uint64_t db = kBMn ? desc_mn_major(sb, kBK * 128) : desc_k_major(sb);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              mma_bf16(d, da + k * kStepK, db + k * (kBMn ? kStepMN : kStepK), idesc, kb > k0 || k > 0);
            mma_commit(smem_addr(&s_empty[s]));
          }
          if (ok) mma_commit(smem_addr(&s_acc_full[b]));
        }
      }
      if (!ok) {  // the products in flight finish before the CTA's memory goes
        mma_commit(smem_addr(&s_drained));
        mbar_wait_timed(smem_addr(&s_drained), 0);
      }
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;
    const uint32_t patch = patch0 + (warp - 2) * kPatchBytes;
    uint32_t acc = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < tiles.total; i += gridDim.x) {
      const Tile t = tiles.at(i);
      const int m = quarter * 32;
      const int64_t row = static_cast<int64_t>(t.begin) + m;
      const int rows = t.rows - m;
      if constexpr (kScaled) {
        const bool valid = lane < rows;
        const int h = (warp - 2) >> 2, c0 = h * 32 < cols ? h * 32 : -1;
        const int c1 = kGated ? (c0 >= 0 ? cols + c0 : -1) : (h + 4) * 32 < cols ? (h + 4) * 32 : -1;
        const int each = part / kScaledBlocks, all = blocks / kScaledBlocks;  // scales
        const float* sf = valid ? a.a_sf + (row + lane) * all : nullptr;
        for (int p = 0; p < parts; ++p) {
          float v[32], u[32];
          const int g0 = kParts ? p * each : 0, n = kParts ? min(each, all - g0) : all;
          ok = sum_scaled(s_acc_full, tmem + (static_cast<uint32_t>(m) << 16), c0, c1, valid ? sf + g0 : nullptr, n, acc, v, u,
                          &s_abort, [&](uint32_t b) { mbar_arrive(smem_addr(&s_acc_empty[b])); });
          if (!ok) {
            if (lane == 0 && !s_abort) give_up();
            break;
          }
          if (rows <= 0) continue;
          if constexpr (kParts) {
            const bool last = p + 1 == parts;
            const uint32_t sum = tmem + (static_cast<uint32_t>(m) << 16) + kSumColumn;
            if (c0 >= 0) add_part(sum + c0, v, p == 0, last);
            if (c1 >= 0) add_part(sum + c1, u, p == 0, last);
            if (!last) continue;
          }
          if constexpr (kGated) {
            if (c0 >= 0 && t.n0 + c0 < a.epi.cols) finish_rows<kAct>(a.epi, patch, v, u, t.g, row, rows, t.n0 + c0, lane);
          } else {
            float none[1];
            if (c0 >= 0 && t.n0 + c0 < a.epi.cols) finish_rows<kAct>(a.epi, patch, v, none, t.g, row, rows, t.n0 + c0, lane);
            if (c1 >= 0 && t.n0 + c1 < a.epi.cols) finish_rows<kAct>(a.epi, patch, u, none, t.g, row, rows, t.n0 + c1, lane);
          }
        }
      } else {
        for (int p = 0; p < parts; ++p, ++acc) {
          const uint32_t b = acc & 1u;
          ok = s_abort == 0 && mbar_wait_timed(smem_addr(&s_acc_full[b]), acc >> 1 & 1u);
          ok = __all_sync(kFullMask, ok);
          if (!ok) {
            if (lane == 0 && !s_abort) give_up();
            break;
          }
          tc_fence_after();
          const uint32_t lanes = tmem + (static_cast<uint32_t>(m) << 16), d = lanes + b * kMaxBN;
          for (int c = half * 32; c < cols; c += 64) {
            if (rows <= 0 || t.n0 + c >= a.epi.cols) break;
            float v[32], u[kGated ? 32 : 1];
            tmem_ld32(d + c, v);
            if constexpr (kGated) tmem_ld32(d + cols + c, u);
            tmem_ld_wait();
            if constexpr (kParts) {
              const bool last = p + 1 == parts;
              add_part(lanes + kSumColumn + c, v, p == 0, last);
              if constexpr (kGated) add_part(lanes + kSumColumn + cols + c, u, p == 0, last);
              if (!last) continue;
            }
            finish_rows<kAct>(a.epi, patch, v, u, t.g, row, rows, t.n0 + c, lane);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&s_acc_empty[b]));
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

}  // namespace

template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_single(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int part, int num_sms,
                               cudaStream_t stream) {
  const int halves = kAct == EP_ACT_SWIGLU ? 2 : 1;
  CUtensorMap map_a, map_low, map_b;
  cudaError_t st = make_rows_maps<kBMn>(&map_a, &map_b, A, B, a, kBM, bn / 2);
  if (st != cudaSuccess) return st;
  const uint64_t size[2] = {static_cast<uint64_t>(a.sum), static_cast<uint64_t>(a.groups.rows)};
  const uint32_t box[2] = {kBK, kLowRows};
  st = make_tensor_map(&map_low, A, 2, size, box);
  if (st != cudaSuccess) return st;
  auto kern = part > 0 ? rows_kernel<kAct, kBMn, true, kScaled> : rows_kernel<kAct, kBMn, false, kScaled>;
  constexpr int kThreads = rows_threads(kScaled);
  const size_t smem = 1024 + ring_bytes(kScaled) + epilogue_warps(kScaled) * kPatchBytes + sizeof(int) * (static_cast<size_t>(a.groups.E) + 1);
  if (resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem) < 1) return cudaErrorInvalidConfiguration;
  const int64_t tiles = max_row_tiles(a.groups) * ((a.epi.cols + bn / halves - 1) / (bn / halves));
  const unsigned grid = static_cast<unsigned>(tiles < num_sms ? tiles : num_sms);
  return launch_chained(kern, dim3(grid), dim3(kThreads), smem, stream, map_a, map_low, map_b, a, bn, part);
}
#define X(act, mn, scaled) \
  template cudaError_t launch_rows_single<act, mn, scaled>(const uint16_t*, const uint16_t*, const RowsArgs&, int, int, int, cudaStream_t);
EP_ROWS_INSTANCES(X)
#undef X

namespace {

// Which kernel and tile width. A split of the summed index when the tiles would leave most
// SMs idle; if its clusters want more SMs than are allowed, single CTAs sum the same parts.
// Pairs when their tiles of 256 rows are mostly full: groups of 384 rows on average
// (8 groups of about 350 rows, 3336 -> 2408: pairs 77 us, single CTAs 66). The width is
// the one with the least rounds of tiles x cycles of a 64-block of the summed index,
// which are 2 a column of the tile (the tensor cores) or the tile's bytes at the 64 a
// cycle that L2 gives an SM, whichever is more. How the rows lie in the groups is not known
// here: half a tile of every group is taken to be empty. So narrow tiles come where wide
// ones leave SMs idle or a last round short:
//   1613 rows 1152 -> 3064 (pairs): 256 columns 21.7 us, the 192 taken 18.2;
//   48 experts with a few rows, 4376 -> 256: 256 columns 50 us, the 128 taken 32.
// (MN-major tiles load whole panels of 64 columns, so the widths between gain nothing there.)
template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int num_sms, cudaStream_t stream) {
  const SplitPlan split = plan_rows_split(a, kAct == EP_ACT_SWIGLU);
  if (split.S > 1 && split.tiles * split.S <= num_sms) return launch_rows_split<kAct, kBMn, kScaled>(A, B, a, split, stream);
  const int halves = kAct == EP_ACT_SWIGLU ? 2 : 1;
  const int64_t rows = a.groups.rows, groups = a.groups.count == nullptr ? 1 : a.groups.E < rows ? a.groups.E : rows;
  auto cost = [&](int tile_rows, int bn, int at_once) {
    int64_t row_tiles = a.groups.count == nullptr ? (rows + tile_rows - 1) / tile_rows : rows / tile_rows + groups / 2;
    if (row_tiles < groups) row_tiles = groups;
    const int64_t tiles = row_tiles * ((a.epi.cols + bn / halves - 1) / (bn / halves));
    const bool pair = tile_rows > kBM;
    const int b_rows = pair ? bn / 2 : bn;  // of B, loaded by a CTA
    const int64_t bytes = kABytes + 128 * (kBMn ? (b_rows + 63) / 64 * 64 : b_rows);
    return (tiles + at_once - 1) / at_once * (2 * bn > bytes / 64 ? 2 * bn : bytes / 64);
  };
  const bool by_parts = split.S > 1;
  const bool pair = !by_parts && rows >= 384 * groups && num_sms >= 2;
  int bn = kMaxBN;
  int64_t least = INT64_MAX;
  for (int w = by_parts ? kMaxBN / 2 : kMaxBN; w >= (pair ? 128 : 64); w = pair ? w - 32 : w / 2) {
    const int64_t c = pair ? cost(2 * kBM, w, num_sms / 2) : cost(kBM, w, num_sms);
    if (c < least) least = c, bn = w;
  }
  return pair ? launch_rows_pair<kAct, kBMn, kScaled>(A, B, a, bn, num_sms, stream)
              : launch_rows_single<kAct, kBMn, kScaled>(A, B, a, bn, by_parts ? split.part : 0, num_sms, stream);
}

template <int kAct>
cudaError_t launch_forward(const ProductArgs& p, const RowsArgs& a, int num_sms, cudaStream_t stream) {
  return a.a_sf != nullptr ? launch_rows<kAct, false, true>(p.x, p.weight, a, num_sms, stream)
                           : launch_rows<kAct, false, false>(p.x, p.weight, a, num_sms, stream);
}

}  // namespace

cudaError_t launch_product(const ProductArgs& p, int num_sms, cudaStream_t stream) {
  RowsArgs a = {p.g.groups, p.g.K, {p.bias, p.residual, p.z, p.out, p.g.N, p.g.Z}, p.err, p.x_sf};
  switch (p.g.act) {
    case EP_ACT_RELU: return launch_forward<EP_ACT_RELU>(p, a, num_sms, stream);
    case EP_ACT_SILU: return launch_forward<EP_ACT_SILU>(p, a, num_sms, stream);
    case EP_ACT_GELU: return launch_forward<EP_ACT_GELU>(p, a, num_sms, stream);
    case EP_ACT_SWIGLU: return launch_forward<EP_ACT_SWIGLU>(p, a, num_sms, stream);
    default: return launch_forward<EP_ACT_NONE>(p, a, num_sms, stream);
  }
}

cudaError_t launch_product_dx(const ProductGradArgs& p, int num_sms, cudaStream_t stream) {
  RowsArgs a = {p.g.groups, p.g.Z, {nullptr, nullptr, nullptr, p.d_x, p.g.K, p.g.K}, p.err, nullptr};
  const uint16_t* dz = p.dz != nullptr ? p.dz : p.d_out;
  return launch_rows<EP_ACT_NONE, true, false>(dz, p.weight, a, num_sms, stream);
}

}  // namespace ep
