// The rows' products when there are few tiles (a token or a handful through a matrix):
// reading the matrix is what counts, and too few CTAs could not read it at full rate. A
// cluster of S CTAs takes one tile of 128 rows, each CTA 1/S of the summed index. Then
// each CTA gets 1/S of the tile's columns: every CTA writes its partial sums of those
// columns into that CTA's shared memory, which adds them in the order of the CTAs and
// does the epilogue.
//
// Measured: one row, 7168 -> 2 x 2048: 15.6 us (58.7 MB; 16 CTAs without the split 42 us, and
// 29 us with 16 clusters of 8, of which 15 fit at once). 9 us of it are the matrix at 6.5 TB/s;
// the rest is start-up, the first loads and the exchange, which bound the smaller calls.
//
// The split depends on the sizes alone, not on the device, and the order of the additions
// is fixed, so results repeat bit for bit.
#include "product_rows.cuh"

namespace ep {

namespace {

constexpr int kBM = kTileRows;
// Clusters of S CTAs that fit on the GPU this is written for at one CTA per SM (152 SMs in
// processing clusters of unequal size); one more would run after the others.
constexpr int resident_clusters(int S) { return S == 8 ? 15 : S == 4 ? 36 : 76; }

template <int kBN, bool kScaled>
struct Shape {
  static constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2, kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (kScaled ? 180224 : 196608) / kStageBytes;  // the more warps, the more patches
  // the exchanged sums of 8 CTAs fit where the stages were
  static_assert(8 * kBM * (kBN / 8 + 4) * 4 <= kStages * kStageBytes, "");
};

// kScaled: scaled sums (product_rows.cuh), an accumulator per scale; a CTA's sums stay in its
// threads' registers until they are exchanged.
template <int kAct, bool kBMn, bool kScaled, int kBN>
__global__ void __launch_bounds__(rows_threads(kScaled), 1)
    rows_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, RowsArgs a,
                      int S, int per, int a_rows) {
  constexpr bool kGated = kAct == EP_ACT_SWIGLU;
  constexpr int kThreads = rows_threads(kScaled), kEpilogueWarps = epilogue_warps(kScaled);
  constexpr int kCols = kGated ? kBN / 2 : kBN;
  constexpr int kHalves = kGated ? 2 : 1;
  using Sizes = Shape<kBN, kScaled>;
  constexpr int kStages = Sizes::kStages, kStageBytes = Sizes::kStageBytes, kABytes = Sizes::kABytes;
  constexpr int kTmem = kScaled ? 2 * kAccColumns : kBN;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full, s_sum_full[2], s_sum_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const uint32_t stage0 = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t patch0 = stage0 + kStages * kStageBytes;
  int* prefix = reinterpret_cast<int*>(s_raw + (patch0 - smem_addr(s_raw)) + kEpilogueWarps * kPatchBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init_count(smem_addr(&s_full[s]), 1);
      mbar_init_count(smem_addr(&s_empty[s]), 1);
    }
    mbar_init_count(smem_addr(&s_acc_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init_count(smem_addr(&s_sum_full[i]), 1);
      mbar_init_count(smem_addr(&s_sum_empty[i]), kEpilogueWarps);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(&s_tmem), kTmem);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  build_prefix<kThreads>(a.groups, kBM, prefix, blockIdx.x == 0 ? a.err : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Tiles<kBM> tiles(a.groups, prefix, a.epi.cols, kCols);
  const int tile = blockIdx.x / S;
  const bool work = tile < tiles.total;  // the same for the whole cluster
  const Tile t = work ? tiles.at(tile) : Tile{0, 0, 0, 0};
  const int blocks = (a.sum + kBK - 1) / kBK;
  const int kb0 = work ? min(blocks, rank * per) : 0, kb1 = work ? min(blocks, kb0 + per) : 0;
  auto give_up = [&] {
    s_abort = 1;
    atomicOr(a.err, kErrTimeout);
  };

  if (warp == 0) {
    if (elect_one()) {
      const uint32_t bytes = static_cast<uint32_t>(a_rows) * (kBK * 2) + kBN * (kBK * 2);
      uint32_t n = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const uint32_t s = n % kStages, bar = smem_addr(&s_full[s]);
        if (s_abort || !mbar_wait_timed(smem_addr(&s_empty[s]), (n / kStages & 1u) ^ 1u)) {
          if (!s_abort) give_up();
          ok = false;
          break;
        }
        mbar_expect(bar, bytes);
        const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
        tma_load_2d(sa, &map_a, kb * kBK, t.begin, bar);
        if constexpr (kBMn) {
#pragma unroll
          for (int p = 0; p < kBN / 64; ++p)
            tma_load_3d(sb + p * (kBK * 128), &map_b, t.n0 + p * 64, kb * kBK, t.g, bar);
        } else {
          tma_load_3d(sb, &map_b, kb * kBK, t.n0, t.g, bar);
          tma_load_3d(sb + kBN / 2 * kBK * 2, &map_b, kb * kBK, kGated ? a.epi.cols + t.n0 : t.n0 + kBN / 2, t.g, bar);
        }
      }
      if (!ok)
        for (uint32_t back = n < kStages ? n : kStages; back > 0; --back) {
          const uint32_t m = n - back;
          mbar_wait_timed(smem_addr(&s_full[m % kStages]), m / kStages & 1u);
        }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16(kBM, kBN, false, kBMn);
      uint32_t n = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const uint32_t s = n % kStages;
        if (s_abort || !mbar_wait_timed(smem_addr(&s_full[s]), n / kStages & 1u)) {
          if (!s_abort) give_up();
          break;
        }
        tc_fence_after();
        uint32_t d = tmem;
        bool first = n == 0;
        const uint32_t acc = n / kScaledBlocks, b = acc & 1u;  // scaled: the accumulator
        if constexpr (kScaled) {
          first = n % kScaledBlocks == 0;
          d += b * kAccColumns;
          if (first && (s_abort || !mbar_wait_timed(smem_addr(&s_sum_empty[b]), (acc >> 1 & 1u) ^ 1u))) {
            if (!s_abort) give_up();
            break;
          }
          tc_fence_after();
        }
        const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
        const uint64_t da = desc_k_major(sa);
        const uint64_t db = kBMn ? desc_mn_major(sb, kBK * 128) : desc_k_major(sb);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          mma_bf16(d, da + k * kStepK, db + k * (kBMn ? kStepMN : kStepK), idesc, !first || k > 0);
        mma_commit(smem_addr(&s_empty[s]));
        if constexpr (kScaled)
          if (n % kScaledBlocks == kScaledBlocks - 1) mma_commit(smem_addr(&s_sum_full[b]));
      }
      mma_commit(smem_addr(&s_acc_full));  // also when it gave up: what was issued has finished
    }
  }
  const int quarter = warp & 3, rows = min(kBM, t.rows);
  const int row = quarter * 32 + lane;
  // scaled sums of this thread's row: 32 columns each from column c0 and c0 + 128 of the tile on
  float own[kScaled ? 2 : 1][32];
  const int c0 = (warp - 2) / 4 * 32;
  if constexpr (kScaled) {
    if (warp >= 2) {
      const int all = blocks / kScaledBlocks;
      const float* sf = row < rows ? a.a_sf + (static_cast<int64_t>(t.begin) + row) * all + kb0 / kScaledBlocks : nullptr;
      uint32_t acc = 0;
      if (!sum_scaled(s_sum_full, tmem + (static_cast<uint32_t>(quarter * 32) << 16), c0, kBN > 128 ? c0 + 128 : -1, sf,
                      (kb1 - kb0) / kScaledBlocks, acc, own[0], own[1], &s_abort,
                      [&](uint32_t b) { mbar_arrive(smem_addr(&s_sum_empty[b])); }) &&
          lane == 0 && !s_abort)
        give_up();
    }
  }
  __syncwarp();
  // every thread: the CTA's products are done, and with them its stages are free
  if (!mbar_wait_timed(smem_addr(&s_acc_full), 0) && lane == 0 && !s_abort) give_up();
  __syncwarp();
  tc_fence_after();
  cluster_sync_all();  // all stages of the cluster are free

  // partial sums [S][rows][width + 4] floats over the stages; CTA r holds columns r * slice on
  const int slice = kCols / S, width = slice * kHalves, stride = width + 4;
  auto give_out = [&](int c, const float (&v)[32]) {
    if (row >= rows) return;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const int n = c + j, h = n / kCols, col = n - h * kCols, r = col / slice;
      const uint32_t at = stage0 + 4u * static_cast<uint32_t>((rank * kBM + row) * stride + h * slice + col - r * slice);
      st_cluster16(cluster_addr(at, static_cast<uint32_t>(r)), v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  };
  if (warp >= 2 && quarter * 32 < rows) {
    if constexpr (kScaled) {
      give_out(c0, own[0]);
      if constexpr (kBN > 128) give_out(c0 + 128, own[1]);
    } else {
      const int half = (warp - 2) >> 2;
      const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2); c += 32) {
        float v[32];
        if (kb1 > kb0) {
          tmem_ld32(d + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        give_out(c, v);
      }
    }
  }
  cluster_sync_all();  // the partial sums have arrived
  if (warp >= 2 && quarter * 32 < rows) {
    const uint32_t patch = patch0 + (warp - 2) * kPatchBytes;
    for (int c = (warp - 2) / 4 * 32; c < slice; c += kEpilogueWarps * 8) {
      const int n0 = t.n0 + rank * slice + c, cols = min(32, slice - c);
      if (n0 >= a.epi.cols) break;
      float v[32], u[kGated ? 32 : 1];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = 0.f;
        if constexpr (kGated) u[j] = 0.f;
      }
      for (int q = 0; q < S; ++q) {
        const uint32_t at = stage0 + 4u * static_cast<uint32_t>((q * kBM + row) * stride + c);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          if (j >= cols) break;
          const uint4 x = ld_shared16(at + 4u * j);
          v[j] += __uint_as_float(x.x), v[j + 1] += __uint_as_float(x.y);
          v[j + 2] += __uint_as_float(x.z), v[j + 3] += __uint_as_float(x.w);
          if constexpr (kGated) {
            const uint4 y = ld_shared16(at + 4u * static_cast<uint32_t>(slice + j));
            u[j] += __uint_as_float(y.x), u[j + 1] += __uint_as_float(y.y);
            u[j + 2] += __uint_as_float(y.z), u[j + 3] += __uint_as_float(y.w);
          }
        }
      }
      finish_rows<kAct>(a.epi, patch, v, u, t.g, static_cast<int64_t>(t.begin) + quarter * 32, rows - quarter * 32, n0, lane,
                        cols);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, kTmem);
}

template <int kAct, bool kBMn, bool kScaled, int kBN>
cudaError_t launch(const uint16_t* A, const uint16_t* B, const RowsArgs& a, const SplitPlan& plan, cudaStream_t stream) {
  using Sizes = Shape<kBN, kScaled>;
  constexpr int kThreads = rows_threads(kScaled);
  const int S = plan.S;
  // boxes of A no higher than the rows there are
  const int a_rows = a.groups.rows < kBM ? (a.groups.rows + 7) / 8 * 8 : kBM;
  CUtensorMap map_a, map_b;
  const cudaError_t st = make_rows_maps<kBMn>(&map_a, &map_b, A, B, a, a_rows, kBN / 2);
  if (st != cudaSuccess) return st;
  auto kern = rows_split_kernel<kAct, kBMn, kScaled, kBN>;
  const size_t smem = 1024 + Sizes::kStages * Sizes::kStageBytes + epilogue_warps(kScaled) * kPatchBytes +
                      sizeof(int) * (static_cast<size_t>(a.groups.E) + 1);
  if (resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem) < 1) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.tiles * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, map_a, map_b, a, S, plan.part, a_rows);
}

}  // namespace

// The split is taken when at least two CTAs can share a tile and all clusters run at once;
// of tiles of 256 and of 128 columns and the ways to split them, the one with the most
// CTAs at work (the wider tile when equal). A single tile of a few rows takes 3.4 us and 0.27
// a block of 64 of the summed index, the exchange 2.5 us (5 with 100 rows): one row, 512 ->
// 2048, 6.6 us split and 5.7 not, 1024 -> 2048 7.0 and 7.7; 100 rows, 1024 -> 2048 9.6 and
// 8.0, 2048 -> 2048 10.5 and 12.3. So it needs 16 blocks, or 32 with more than 32 rows.
SplitPlan plan_rows_split(const RowsArgs& a, bool gated) {
  const int64_t rows = a.groups.rows;
  const int64_t row_tiles = a.groups.count == nullptr ? (rows + kBM - 1) / kBM : max_row_tiles(a.groups);
  const int halves = gated ? 2 : 1;
  const int blocks = (a.sum + kBK - 1) / kBK;
  const int64_t wide = row_tiles * ((a.epi.cols + 256 / halves - 1) / (256 / halves));
  const int64_t narrow = row_tiles * ((a.epi.cols + 128 / halves - 1) / (128 / halves));
  SplitPlan plan = {1, blocks, false, 0};
  if (blocks < (rows <= 32 ? 16 : 32)) return plan;
  int64_t ctas = 0;
  for (int s = 2; s <= 8 && blocks >= s * 2; s *= 2) {
    int part = (blocks + s - 1) / s;
    if (a.a_sf != nullptr) part = (part + kScaledBlocks - 1) / kScaledBlocks * kScaledBlocks;
    if (wide <= resident_clusters(s) && wide * s > ctas) plan = {s, part, false, wide}, ctas = wide * s;
    if (narrow <= resident_clusters(s) && narrow * s > ctas) plan = {s, part, true, narrow}, ctas = narrow * s;
  }
  return plan;
}

template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_split(const uint16_t* A, const uint16_t* B, const RowsArgs& a, const SplitPlan& plan, cudaStream_t stream) {
  return plan.narrow ? launch<kAct, kBMn, kScaled, 128>(A, B, a, plan, stream)
                     : launch<kAct, kBMn, kScaled, 256>(A, B, a, plan, stream);
}
#define X(act, mn, scaled) \
  template cudaError_t launch_rows_split<act, mn, scaled>(const uint16_t*, const uint16_t*, const RowsArgs&, const SplitPlan&, cudaStream_t);
EP_ROWS_INSTANCES(X)
#undef X

}  // namespace ep
