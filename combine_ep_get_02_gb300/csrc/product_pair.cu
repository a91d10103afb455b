// The rows' products with pairs of CTAs: tiles of 256 rows x up to 256 columns, one tcgen05.mma
// over both SMs of a cluster of two. Each CTA brings its 128 rows of A and its half of B's
// columns, so B crosses from L2 once for 256 rows instead of once for 128, and a
// stage is 32 KB instead of 48, which makes room for six. (L2 gives an SM about 64 bytes a
// cycle; a 128 x 256 tile of its own wants 96 at the tensor cores' full rate, a pair's tile 64.)
//
// The tensor cores bound it (70 to 90% of their time busy; the rest is the first loads, the last
// epilogue and the last round of tiles). Measured: 4096 x 2048 -> 7168 with bias and residual
// 70-82 us (1.5-1.7 PFLOP/s, by the clock that the power limit leaves; single CTAs 94 us);
// 65536 x 7168 -> 2 x 2048 over 64 experts 2.26 ms (1.70 PFLOP/s), 2.7 ms on FP8 codes with scaled
// sums (an accumulator changes hands every 0.6 us of products; arriving on the first CTA's
// barriers with release at cluster scope took 5.0).
//
// The pair's first CTA issues the products for both. Its "full" barriers count the bytes
// that land in both CTAs; the commits arrive on both CTAs' "empty" and "accumulator full"
// barriers; the epilogue warps of both arrive on its "accumulator empty" ones.
#include "product_rows.cuh"

namespace ep {

namespace {

constexpr int kBM = kTileRows, kBN = kAccColumns;  // rows a CTA, columns a pair at most
constexpr int stages(bool scaled) { return scaled ? 5 : 6; }  // the more warps, the more patches
constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN / 2 * kBK * 2, kStageBytes = kABytes + kBBytes;

// kScaled: scaled sums (product_rows.cuh), an accumulator per scale.
template <int kAct, bool kBMn, bool kScaled>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(rows_threads(kScaled), 1)
    rows_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, RowsArgs a, int bn) {
  constexpr bool kGated = kAct == EP_ACT_SWIGLU;
  constexpr int kThreads = rows_threads(kScaled), kEpilogueWarps = epilogue_warps(kScaled), kStages = stages(kScaled);
  const int cols = kGated ? bn / 2 : bn;  // output columns of a tile
  const int panels = (bn / 2 + 63) / 64;  // of B's half, MN-major
  const uint32_t bytes = static_cast<uint32_t>(kABytes + (kBMn ? panels * (kBK * 128) : bn / 2 * kBK * 2));
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_acc_full[2], s_acc_empty[2], s_drained;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t stage0 = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t patch0 = stage0 + kStages * kStageBytes;
  int* prefix = reinterpret_cast<int*>(s_raw + (patch0 - smem_addr(s_raw)) + kEpilogueWarps * kPatchBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init_count(smem_addr(&s_full[s]), 1);
      mbar_init_count(smem_addr(&s_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_count(smem_addr(&s_acc_full[i]), 1);
      mbar_init_count(smem_addr(&s_acc_empty[i]), 2 * kEpilogueWarps);
    }
    mbar_init_count(smem_addr(&s_drained), 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(&s_tmem), 512);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();
  build_prefix<kThreads>(a.groups, 2 * kBM, prefix, blockIdx.x == 0 ? a.err : nullptr);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers and accumulators exist
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Tiles<2 * kBM> tiles(a.groups, prefix, a.epi.cols, cols);
  // an accumulator per scale makes many waits; none of them is for memory that a CTA wrote
  constexpr bool kClusterWaits = !kScaled;
  const int blocks = (a.sum + kBK - 1) / kBK;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto give_up = [&] {
    s_abort = 1;
    atomicOr(a.err, kErrTimeout);
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t n = 0;  // stages filled so far
      bool ok = true;
      for (int i = first; ok && i < tiles.total; i += step) {
        const Tile t = tiles.at(i);
        for (int kb = 0; kb < blocks; ++kb, ++n) {
          const uint32_t s = n % kStages, bar = cluster_addr(smem_addr(&s_full[s]), 0);
          if (s_abort || !mbar_wait_timed<kClusterWaits>(smem_addr(&s_empty[s]), (n / kStages & 1u) ^ 1u)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect(smem_addr(&s_full[s]), 2 * bytes);
          const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
          tma_load_2d_pair(sa, &map_a, kb * kBK, t.begin + static_cast<int>(rank) * kBM, bar);
          if constexpr (kBMn) {
            for (int p = 0; p < panels; ++p)
              tma_load_3d_pair(sb + p * (kBK * 128), &map_b, t.n0 + static_cast<int>(rank) * (bn / 2) + p * 64, kb * kBK,
                               t.g, bar);
          } else {
            const int second = kGated ? a.epi.cols : bn / 2;
            tma_load_3d_pair(sb, &map_b, kb * kBK, t.n0 + (rank ? second : 0), t.g, bar);
          }
        }
      }
      if (!ok && rank == 0)  // the copies in flight land before the CTAs' memory goes
        for (uint32_t back = n < kStages ? n : kStages; back > 0; --back) {
          const uint32_t m = n - back;
          mbar_wait_timed<kClusterWaits>(smem_addr(&s_full[m % kStages]), m / kStages & 1u);
        }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_bf16(2 * kBM, bn, false, kBMn);
      uint32_t n = 0, acc = 0;
      bool ok = true;
      for (int i = first; ok && i < tiles.total; i += step) {
        const int each = kScaled ? kScaledBlocks : blocks;  // blocks of an accumulator
        for (int k0 = 0; ok && k0 < blocks; k0 += each, ++acc) {
          const uint32_t b = acc & 1u;
          if (s_abort || !mbar_wait_timed<kClusterWaits>(smem_addr(&s_acc_empty[b]), (acc >> 1 & 1u) ^ 1u)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * kBN;
          for (int kb = k0; kb < k0 + each; ++kb, ++n) {
            const uint32_t s = n % kStages;
            if (s_abort || !mbar_wait_timed<kClusterWaits>(smem_addr(&s_full[s]), n / kStages & 1u)) {
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
              mma_bf16_pair(d, da + k * kStepK, db + k * (kBMn ? kStepMN : kStepK), idesc, kb > k0 || k > 0);
            mma_commit_pair(smem_addr(&s_empty[s]));
          }
          if (ok) mma_commit_pair(smem_addr(&s_acc_full[b]));
        }
      }
      if (!ok) {  // the products in flight finish before the CTAs' memory goes
        mma_commit_pair(smem_addr(&s_drained));
        mbar_wait_timed<kClusterWaits>(smem_addr(&s_drained), 0);
      }
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;
    const uint32_t patch = patch0 + (warp - 2) * kPatchBytes;
    uint32_t acc = 0;
    if constexpr (kScaled) {
      const int c0 = half * 32 < cols ? half * 32 : -1, all = blocks / kScaledBlocks;
      const int c1 = kGated ? (c0 >= 0 ? cols + c0 : -1) : (half + 4) * 32 < cols ? (half + 4) * 32 : -1;
      for (int i = first; i < tiles.total; i += step) {
        const Tile t = tiles.at(i);
        const int m = quarter * 32;
        const int rows = t.rows - static_cast<int>(rank) * kBM - m;
        const int64_t row = static_cast<int64_t>(t.begin) + static_cast<int>(rank) * kBM + m;
        const float* sf = lane < rows ? a.a_sf + (row + lane) * all : nullptr;
        float v[32], u[32];
        if (!sum_scaled(s_acc_full, tmem + (static_cast<uint32_t>(m) << 16), c0, c1, sf, all, acc, v, u, &s_abort,
                        [&](uint32_t b) { mbar_arrive_read(cluster_addr(smem_addr(&s_acc_empty[b]), 0)); })) {
          if (lane == 0 && !s_abort) give_up();
          break;
        }
        if (rows <= 0) continue;
        if constexpr (kGated) {
          if (c0 >= 0 && t.n0 + c0 < a.epi.cols)
            finish_rows<kAct>(a.epi, patch, v, u, t.g, row, rows, t.n0 + c0, lane, min(32, cols - c0));
        } else {
          float none[1];
          if (c0 >= 0 && t.n0 + c0 < a.epi.cols)
            finish_rows<kAct>(a.epi, patch, v, none, t.g, row, rows, t.n0 + c0, lane, min(32, cols - c0));
          if (c1 >= 0 && t.n0 + c1 < a.epi.cols)
            finish_rows<kAct>(a.epi, patch, u, none, t.g, row, rows, t.n0 + c1, lane, min(32, cols - c1));
        }
      }
    } else {
      for (int i = first; i < tiles.total; i += step, ++acc) {
        const uint32_t b = acc & 1u;
        const Tile t = tiles.at(i);
        bool ok = s_abort == 0 && mbar_wait_timed(smem_addr(&s_acc_full[b]), acc >> 1 & 1u);
        ok = __all_sync(kFullMask, ok);
        if (!ok) {
          if (lane == 0 && !s_abort) give_up();
          break;
        }
        tc_fence_after();
        const int m = quarter * 32;
        const int rows = t.rows - static_cast<int>(rank) * kBM - m;
        const int64_t row = static_cast<int64_t>(t.begin) + static_cast<int>(rank) * kBM + m;
        const uint32_t d = tmem + b * kBN + (static_cast<uint32_t>(m) << 16);
        for (int c = half * 32; c < cols; c += 64) {
          if (rows <= 0 || t.n0 + c >= a.epi.cols) break;
          float v[32], u[kGated ? 32 : 1];
          tmem_ld32(d + c, v);
          if constexpr (kGated) tmem_ld32(d + cols + c, u);
          tmem_ld_wait();
          finish_rows<kAct>(a.epi, patch, v, u, t.g, row, rows, t.n0 + c, lane, min(32, cols - c));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_acc_empty[b]), 0));
      }
    }
  }
  __syncwarp();
  __syncthreads();
  cluster_sync_all();  // neither CTA's memory goes while the other may still use it
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

}  // namespace

template <int kAct, bool kBMn, bool kScaled>
cudaError_t launch_rows_pair(const uint16_t* A, const uint16_t* B, const RowsArgs& a, int bn, int num_sms, cudaStream_t stream) {
  const int halves = kAct == EP_ACT_SWIGLU ? 2 : 1;
  CUtensorMap map_a, map_b;
  const cudaError_t st = make_rows_maps<kBMn>(&map_a, &map_b, A, B, a, kBM, bn / 2);
  if (st != cudaSuccess) return st;
  auto kern = rows_pair_kernel<kAct, kBMn, kScaled>;
  constexpr int kThreads = rows_threads(kScaled);
  const size_t smem = 1024 + stages(kScaled) * kStageBytes + epilogue_warps(kScaled) * kPatchBytes + sizeof(int) * (static_cast<size_t>(a.groups.E) + 1);
  if (resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem) < 1) return cudaErrorInvalidConfiguration;
  const int cols = bn / halves;
  const int64_t most = max_row_tiles(a.groups, 2 * kBM) * ((a.epi.cols + cols - 1) / cols);
  const int64_t pairs = most < num_sms / 2 ? most : num_sms / 2;  // num_sms >= 2
  return launch_chained(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), smem, stream, map_a, map_b, a, bn);
}
#define X(act, mn, scaled) \
  template cudaError_t launch_rows_pair<act, mn, scaled>(const uint16_t*, const uint16_t*, const RowsArgs&, int, int, cudaStream_t);
EP_ROWS_INSTANCES(X)
#undef X

}  // namespace ep
