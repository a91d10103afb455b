// Gradient of the experts' matrices: dW_g[z][k] = sum over the group's rows r of
// dz[r][z] x[r][k], for every group (zeros for an empty one).
//
// Tiles of 256 x 256 of dW, one to a pair of CTAs (a cluster of two) with one tcgen05.mma
// over both SMs, as in the rows' products; roles as there (a warp for TMA, one for the
// products, eight for the epilogue), and one that mends the tiles below. Both operands are MN-major: the summed index is the
// row, so tiles of 64 rows are used as they lie in the tensors, without a transposition.
//
// A group's last tile ends inside the next group's rows (or padding). The rows past the
// group, up to the next multiple of 16 (one instruction's share), are zeroed in shared memory
// in both operands, so that not even a NaN there reaches the sum; the rest is left out by
// issuing fewer instructions. Since each CTA must have mended its own half before the
// pair's product reads it, the loads of such a tile count on the CTA's own barrier; a warp of
// each CTA waits for that, mends, and arrives on a barrier of the first CTA, which its
// product thread waits for. (All tiles' loads taking that way more than doubled the
// kernel's time; the product warp mending itself, all its lanes waiting for every tile, cost
// a fifth: 97 us against 80 at 4096 x 4096 x 4096.)
// Measured: 4096 x 4096 x 4096 80 us (1.7 PFLOP/s; 4 rounds of tiles, the last a third
// full); 32 experts of about 512 rows, 2048 x 2048, 125 us (1.1 PFLOP/s): there the writing
// of 268 MB of dW weighs as much as the products (100 us without the stores).
// (Single CTAs with tiles of 128 x 256 reached 48% of the tensor cores' time: they want
// 96 bytes a cycle from L2 where an SM gets about 64.)
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + 32 * kEpilogueWarps + 32;
constexpr int kBM = 128, kBN = 256, kBK = 64;  // rows of dW a CTA, columns a pair, rows of x and dz a stage
constexpr int kStages = 6;
constexpr int kPanel = kBK * 128;  // bytes of 64 columns x 64 rows
constexpr int kABytes = kBM * kBK * 2, kBBytes = kBN / 2 * kBK * 2, kStageBytes = kABytes + kBBytes;

struct WeightArgs {
  Groups groups;
  int Z, K;
  uint32_t* err;
};

// Rows of a stage that count, and whether the tile ends inside an instruction's 16.
__device__ __forceinline__ bool to_mend(int left) { return left < kBK && (left & 15) != 0; }

struct Tile {
  int g, begin, rows, z0, k0;
};

// A tile whose group's place is still on its way from memory: the next one is looked up
// (and nothing computed from it) while the current one is worked on.
struct Ahead {
  int g, r, region, base, count;
};
__device__ __forceinline__ Ahead look_up(const WeightArgs& a, int i, int total, int mt, int nt) {
  Ahead t{0, 0, 0, 0, 0};
  if (i >= total) return t;
  t.g = i / (mt * nt);
  t.r = i - t.g * (mt * nt);
  const Groups& q = a.groups;
  if (q.count == nullptr) {
    t.count = q.rows;
  } else {
    const int d = t.g / q.L;
    t.region = __ldg(q.region + d);
    t.base = __ldg(q.base + t.g + d);
    t.count = __ldg(q.count + t.g);
  }
  return t;
}
__device__ __forceinline__ Tile resolve(const WeightArgs& a, const Ahead& t, int mt) {
  bool cut = false;
  const GroupRows rows = clip_rows(a.groups, static_cast<int64_t>(t.region) + t.base, t.count, &cut);
  const int n = t.r / mt;
  return Tile{t.g, rows.begin, rows.count, (t.r - n * mt) * 2 * kBM, n * kBN};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    weight_grad_kernel(const __grid_constant__ CUtensorMap map_dz, const __grid_constant__ CUtensorMap map_x,
                       const __grid_constant__ CUtensorMap map_out, WeightArgs a) {
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_part[kStages], s_mended[kStages], s_acc_full[2], s_acc_empty[2], s_drained;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const uint32_t stage0 = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t patch0 = stage0 + kStages * kStageBytes;
  uint8_t* stage_mem = s_raw + (stage0 - smem_addr(s_raw));
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init_count(smem_addr(&s_full[s]), 1);
      mbar_init_count(smem_addr(&s_empty[s]), 1);
      mbar_init_count(smem_addr(&s_part[s]), 1);
      mbar_init_count(smem_addr(&s_mended[s]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_count(smem_addr(&s_acc_full[i]), 1);
      mbar_init_count(smem_addr(&s_acc_empty[i]), 2 * kEpilogueWarps);
    }
    mbar_init_count(smem_addr(&s_drained), 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_dz);
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_out);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(&s_tmem), 512);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0) {  // blocks that leave the tensors are reported once
    bool cut = false;
    for (int g = threadIdx.x; g < a.groups.E; g += kThreads) group_rows(a.groups, g, &cut);
    if (cut) atomicOr(a.err, kErrOverflow);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers and accumulators exist
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int mt = (a.Z + 2 * kBM - 1) / (2 * kBM), nt = (a.K + kBN - 1) / kBN;
  const int total = a.groups.E * mt * nt;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  Ahead ahead = look_up(a, first, total, mt, nt);
  auto give_up = [&] {
    s_abort = 1;
    atomicOr(a.err, kErrTimeout);
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t n = 0;
      uint32_t part = 0, full_phase = 0, part_phase = 0;  // bit s: stage s's last use, phases of its barriers
      bool ok = true;
      for (int i = first; ok && i < total; i += step) {
        const Tile t = resolve(a, ahead, mt);
        ahead = look_up(a, i + step, total, mt, nt);
        for (int r = 0; r < t.rows; r += kBK, ++n) {
          const uint32_t s = n % kStages, bit = 1u << s;
          if (s_abort || !mbar_wait_timed(smem_addr(&s_empty[s]), (n / kStages & 1u) ^ 1u)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
          const int z = t.z0 + rank * kBM, k = t.k0 + rank * (kBN / 2);
          uint32_t bar;
          if (to_mend(t.rows - r)) {
            bar = smem_addr(&s_part[s]);
            mbar_expect(bar, kStageBytes);
            part |= bit;
            part_phase ^= bit;
          } else {
            bar = cluster_addr(smem_addr(&s_full[s]), 0);
            if (rank == 0) mbar_expect(smem_addr(&s_full[s]), 2 * kStageBytes);
            part &= ~bit;
            full_phase ^= bit;
          }
#pragma unroll
          for (int p = 0; p < kBM / 64; ++p) tma_load_2d_pair(sa + p * kPanel, &map_dz, z + p * 64, t.begin + r, bar);
#pragma unroll
          for (int p = 0; p < kBN / 128; ++p) tma_load_2d_pair(sb + p * kPanel, &map_x, k + p * 64, t.begin + r, bar);
        }
      }
      if (!ok)  // the copies in flight land before the CTAs' memory goes
        for (uint32_t s = 0; s < kStages && s < n; ++s) {
          if (part >> s & 1u) mbar_wait_timed(smem_addr(&s_part[s]), (part_phase >> s & 1u) ^ 1u);
          else if (rank == 0) mbar_wait_timed(smem_addr(&s_full[s]), (full_phase >> s & 1u) ^ 1u);
        }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_bf16(2 * kBM, kBN, true, true);
      uint32_t n = 0, acc = 0;
      uint32_t full_phase = 0, mended_phase = 0;  // bit s: phase of stage s's barriers
      bool ok = true;
      for (int i = first; ok && i < total; i += step) {
        const Tile t = resolve(a, ahead, mt);
        ahead = look_up(a, i + step, total, mt, nt);
        if (t.rows == 0) continue;
        const uint32_t b = acc & 1u;
        if (s_abort || !mbar_wait_timed(smem_addr(&s_acc_empty[b]), (acc >> 1 & 1u) ^ 1u)) {
          if (!s_abort) give_up();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + b * kBN;
        for (int r = 0; r < t.rows; r += kBK, ++n) {
          const uint32_t s = n % kStages, bit = 1u << s;
          uint32_t bar, phase;
          if (to_mend(t.rows - r)) {
            bar = smem_addr(&s_mended[s]);
            phase = mended_phase >> s & 1u;
            mended_phase ^= bit;
          } else {
            bar = smem_addr(&s_full[s]);
            phase = full_phase >> s & 1u;
            full_phase ^= bit;
          }
          if (s_abort || !mbar_wait_timed(bar, phase)) {
            if (!s_abort) give_up();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = stage0 + s * kStageBytes, sb = sa + kABytes;
          const uint64_t da = desc_mn_major(sa, kPanel), db = desc_mn_major(sb, kPanel);
          const int left = t.rows - r;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            if (k * 16 < left) mma_bf16_pair(d, da + k * kStepMN, db + k * kStepMN, idesc, r > 0 || k > 0);
          mma_commit_pair(smem_addr(&s_empty[s]));
        }
        if (ok) mma_commit_pair(smem_addr(&s_acc_full[b]));
        ++acc;
      }
      if (!ok) {  // the products in flight finish before the CTAs' memory goes
        mma_commit_pair(smem_addr(&s_drained));
        mbar_wait_timed(smem_addr(&s_drained), 0);
      }
    }
  } else if (warp == 2 + kEpilogueWarps) {
    uint32_t n = 0, part_phase = 0, waited = 0;  // waited: stages up to the last tile that was mended
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
      const Tile t = resolve(a, ahead, mt);
      ahead = look_up(a, i + step, total, mt, nt);
      const int stages = (t.rows + kBK - 1) / kBK;
      n += static_cast<uint32_t>(stages);
      const int left = t.rows - (stages - 1) * kBK;  // rows of the last stage that count
      if (stages == 0 || !to_mend(left)) continue;
      const uint32_t s = (n - 1) % kStages;
      ok = __all_sync(kFullMask, s_abort == 0 && mbar_wait_stages(smem_addr(&s_part[s]), part_phase >> s & 1u, n - waited, &s_abort));
      waited = n;
      if (!ok) {
        if (lane == 0 && !s_abort) give_up();
        break;
      }
      part_phase ^= 1u << s;
      // a 128-byte row of a panel holds one row's 64 columns, in whatever order
      const int chunks = (((left + 15) & ~15) - left) * 8;
      uint8_t* base = stage_mem + s * kStageBytes + left * 128;
      for (int p = 0; p < kStageBytes / kPanel; ++p)
        for (int c = lane; c < chunks; c += 32)
          *reinterpret_cast<uint4*>(base + p * kPanel + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_mended[s]), 0));
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t patch = patch0 + (warp - 2) * 2 * kPatchBytes;
    uint32_t stored = 0;  // chunks handed to TMA; two patches in turn
    uint32_t acc = 0;
    for (int i = first; i < total; i += step) {
      const Tile t = resolve(a, ahead, mt);
      ahead = look_up(a, i + step, total, mt, nt);
      const uint32_t b = acc & 1u;
      const int z0 = t.z0 + rank * kBM + quarter * 32;
      if (t.rows > 0) {
        bool ok = s_abort == 0 && mbar_wait_stages(smem_addr(&s_acc_full[b]), acc >> 1 & 1u,
                                                   static_cast<uint32_t>(t.rows) / kBK, &s_abort);
        ok = __all_sync(kFullMask, ok);
        if (!ok) {
          if (lane == 0 && !s_abort) give_up();
          break;
        }
        tc_fence_after();
      }
      const uint32_t d = tmem + b * kBN + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2); c += 32) {
        if (z0 >= a.Z || t.k0 + c >= a.K) break;
        float v[32];
        if (t.rows > 0) {
          tmem_ld32(d + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        // the last but one store from this patch has been read by now, or is waited for
        if (lane == 0) tma_store_wait_reads<1>();
        __syncwarp();
        const uint32_t at = patch + (stored++ & 1u) * kPatchBytes;
#pragma unroll
        for (int j = 0; j < 4; ++j) st_shared16(patch_at(at, lane, j), pack8(v + 8 * j));
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {  // what lies past Z or K is not written
          tma_store_3d(&map_out, t.k0 + c, z0, t.g, at);
          bulk_commit();
        }
      }
      if (t.rows > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_acc_empty[b]), 0));
        ++acc;
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  __syncthreads();
  cluster_sync_all();  // neither CTA's memory goes while the other may still use it
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

}  // namespace

cudaError_t launch_product_dw(const ProductGradArgs& p, int num_sms, cudaStream_t stream) {
  const uint16_t* dz = p.dz != nullptr ? p.dz : p.d_out;
  WeightArgs a = {p.g.groups, p.g.Z, p.g.K, p.err};
  CUtensorMap map_dz, map_x, map_out;
  const uint32_t box[2] = {64, kBK};
  const uint64_t size_dz[2] = {static_cast<uint64_t>(a.Z), static_cast<uint64_t>(a.groups.rows)};
  const uint64_t size_x[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.groups.rows)};
  cudaError_t st = make_tensor_map(&map_dz, dz, 2, size_dz, box);
  if (st == cudaSuccess) st = make_tensor_map(&map_x, p.x, 2, size_x, box);
  const uint64_t size_out[3] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.Z), static_cast<uint64_t>(a.groups.E)};
  const uint32_t box_out[3] = {32, 32, 1};
  if (st == cudaSuccess) st = make_tensor_map(&map_out, p.d_weight, 3, size_out, box_out);
  if (st != cudaSuccess) return st;
  const size_t smem = 1024 + kStages * kStageBytes + 2 * kEpilogueWarps * kPatchBytes;
  if (resident_ctas(reinterpret_cast<const void*>(weight_grad_kernel), kThreads, smem) < 1)
    return cudaErrorInvalidConfiguration;
  const int64_t total =
      static_cast<int64_t>(a.groups.E) * ((a.Z + 2 * kBM - 1) / (2 * kBM)) * ((a.K + kBN - 1) / kBN);
  const int64_t pairs = num_sms < 4 ? 1 : num_sms / 2;
  const unsigned grid = static_cast<unsigned>(2 * (total < pairs ? total : pairs));
  return launch_chained(weight_grad_kernel, dim3(grid), dim3(kThreads), smem, stream, map_dz, map_x,
                        map_out, a);
}

}  // namespace ep
