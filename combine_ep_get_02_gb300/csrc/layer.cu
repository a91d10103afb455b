// The experts' layer of a few tokens in two kernels, straight from the router's choice:
//
//   up    h_l = act(x_t W_up[e]^T + b_up[e])                      for every lane l = (t, k), e its expert
//   down  out_t = sum_k w_tk (h_l W_down[e]^T + b_down[e]) + residual_t
//
// Reading the chosen experts' matrices once is what it costs, so both kernels are one stream of
// matrix rows through shared memory: a producer warp keeps a ring of stages full with bulk copies, eight
// warps multiply. A work item is a strip of 16 or 32 matrix rows times all tokens of that expert
// (a group; tokens past kTokens are another group): the matrix rows are the 16 rows of mma.sync's
// A operand, the tokens its 8 columns, and the eight warps share the summed index. With at most
// 32 tokens to a matrix the tensor cores are far from being the limit, so the products go where their
// operands need least preparation: the fragments are read straight from rows as they lie in
// memory (the summed index is permuted alike for both), and FP8 codes become bf16 on the way.
#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kWarps = 8;                        // that multiply
constexpr int kThreads = (kWarps + 1) * 32;      // and the producer's
constexpr int kMaxStages = 16;
constexpr int kMaxLanes = kLayerMaxTokens * kMaxTopk;

// A group: the tokens (at most kTokens) that go to one expert, `n` of them at `start` in the lists.
struct Group {
  int expert, start, n;
};
__device__ __forceinline__ uint32_t pack_group(int expert, int start, int n) {
  return static_cast<uint32_t>(expert) | static_cast<uint32_t>(start) << 12 | static_cast<uint32_t>(n) << 23;
}
__device__ __forceinline__ Group unpack_group(uint32_t v) {
  return Group{static_cast<int>(v & 0xFFFu), static_cast<int>(v >> 12 & 0x7FFu), static_cast<int>(v >> 23)};
}
static_assert(kMaxExperts <= 4096 && kMaxLanes <= 2048, "a group fits one word");

// The chosen lanes ordered by expert, then token: both kernels make the same lists of the same choice.
struct Lists {
  uint16_t* token;   // [lanes]
  float* weight;     // [lanes]
  uint32_t* groups;  // [lanes]
};

// Builds the lists; returns the number of groups. An expert that a token chose twice is one lane with
// both weights. `scratch`: (2 lanes + 2 E) words. Called by all threads; ends with a barrier.
__device__ int build_lists(const LayerArgs& a, int tokens_a_group, const Lists& q, uint32_t* scratch, uint32_t* err) {
  __shared__ uint32_t s_warp[kThreads / 32];
  __shared__ int s_groups;
  const int lanes = a.T * a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto expert_at = [&](int i) {
    const int64_t e = __ldg(a.idx + i);
    if (e >= 0 && e < a.E) return static_cast<int>(e);
    if (e != -1 && err != nullptr) atomicOr(err, kErrBadTopk);
    return -1;
  };
  if (lanes <= 32) {  // one warp, in registers
    if (warp == 0) {
      int e = lane < lanes ? expert_at(lane) : -1;
      float w = lane < lanes ? __ldg(a.w + lane) : 0.f;
      const int t = lane / a.K;
      const unsigned same = __match_any_sync(kFullMask, e >= 0 ? e * 64 + t : -1 - lane);
      unsigned more = same & ~lanemask_lt() & ~(1u << lane);
      const float own = w;
      while (__any_sync(kFullMask, more != 0)) {
        const float v = __shfl_sync(kFullMask, own, more ? __ffs(more) - 1 : lane);
        if (more) w += v;
        more &= more - 1;
      }
      if (same & lanemask_lt()) e = -1;
      const unsigned mates = __match_any_sync(kFullMask, e >= 0 ? e : -1 - lane);
      const int rank = __popc(mates & lanemask_lt()), n = __popc(mates);
      int before = e >= 0 && rank == 0 ? n : 0;
      const int mine = before;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFullMask, before, o);
        if (lane >= o) before += v;
      }
      const int start = __shfl_sync(kFullMask, before - mine, __ffs(mates) - 1);
      const bool first = e >= 0 && rank % tokens_a_group == 0;
      const unsigned firsts = __ballot_sync(kFullMask, first);
      if (e >= 0) {
        q.token[start + rank] = static_cast<uint16_t>(t);
        q.weight[start + rank] = w;
      }
      if (first) q.groups[__popc(firsts & lanemask_lt())] = pack_group(e, start + rank, min(tokens_a_group, n - rank));
      if (lane == 0) s_groups = __popc(firsts);
    }
    __syncthreads();
    return s_groups;
  }
  int* raw = reinterpret_cast<int*>(scratch);
  float* weight = reinterpret_cast<float*>(scratch + lanes);
  uint32_t* count = scratch + 2 * lanes;
  uint32_t* run = count + a.E;  // where an expert's next lane goes
  for (int e = threadIdx.x; e < a.E; e += kThreads) count[e] = 0;
  for (int i = threadIdx.x; i < lanes; i += kThreads) {
    raw[i] = expert_at(i);
    weight[i] = __ldg(a.w + i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < lanes; i += kThreads) {
    const int e = raw[i], k = i % a.K;
    bool again = false;
    for (int j = 1; j <= k; ++j) again = again || raw[i - j] == e;
    if (e >= 0 && !again) atomicAdd(count + e, 1u);
  }
  __syncthreads();
  // lanes (low half) and groups (high half) of the experts before each
  const int per = (a.E + kThreads - 1) / kThreads;
  const int e0 = min(a.E, static_cast<int>(threadIdx.x) * per), e1 = min(a.E, e0 + per);
  auto both = [&](uint32_t n) { return n | (n + tokens_a_group - 1) / tokens_a_group << 16; };
  uint32_t sum = 0;
  for (int e = e0; e < e1; ++e) sum += both(count[e]);
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  uint32_t before = incl - sum;
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  for (int e = e0; e < e1; ++e) {
    const uint32_t n = count[e];
    run[e] = before & 0xFFFFu;
    for (uint32_t c = 0; c < n; c += tokens_a_group)
      q.groups[(before >> 16) + c / tokens_a_group] =
          pack_group(e, (before & 0xFFFFu) + c, min(static_cast<uint32_t>(tokens_a_group), n - c));
    before += both(n);
  }
  if (threadIdx.x == kThreads - 1) s_groups = before >> 16;
  __syncthreads();
  if (warp == 0) {  // lanes to their places, in their order
    for (int i0 = 0; i0 < lanes; i0 += 32) {
      const int i = i0 + lane;
      int e = i < lanes ? raw[i] : -1;
      const int t = i / a.K, k = i - t * a.K;
      float w = 0.f;
      if (e >= 0) {
        bool again = false;
        for (int j = 0; j < a.K; ++j)
          if (raw[i - k + j] == e) {
            again = again || j < k;
            w += weight[i - k + j];
          }
        if (again) e = -1;
      }
      const unsigned mates = __match_any_sync(kFullMask, e >= 0 ? e : -1 - lane);
      const int rank = __popc(mates & lanemask_lt());
      const uint32_t at = e >= 0 ? run[e] + rank : 0;
      __syncwarp();
      if (e >= 0) {
        if (rank == 0) run[e] += __popc(mates);
        q.token[at] = static_cast<uint16_t>(t);
        q.weight[at] = w;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  return s_groups;
}

__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes -> two pairs of bf16, exactly.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  float f[4];
  e4m3x4_to_f32(w, f);
  lo = f32x2_to_bf16x2(f[0], f[1]);
  hi = f32x2_to_bf16x2(f[2], f[3]);
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

__device__ __forceinline__ void bulk_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float act_any(float z, int act) {
  switch (act) {
    case EP_ACT_RELU: return activate<EP_ACT_RELU>(z);
    case EP_ACT_SILU:
    case EP_ACT_SWIGLU: return activate<EP_ACT_SILU>(z);
    case EP_ACT_GELU: return activate<EP_ACT_GELU>(z);
    default: return z;
  }
}

// Shared memory of a kernel, in bytes from the start of its dynamic part.
struct Plan {
  uint32_t token, weight, groups, sums, acc, ring, stage, stages, total;
};

// A stage: kRowBytes of each matrix row of the strip and as many values of each token's row, at pitches that put
// the 16-byte pieces which eight threads read at once in different banks; with FP8 the
// scales of 8 rows x 128 columns each.
template <bool kFp8, int kRows, int kTokens>
struct Stage {
  static constexpr int kRowBytes = kFp8 || kTokens == 32 ? 512 : 1024;
  static constexpr int kPitch = kRowBytes + 64;
  static constexpr int kColumns = kFp8 ? kRowBytes : kRowBytes / 2;  // of the summed index
  static constexpr int kXPitch = kFp8 ? 2 * kRowBytes + 16 : kPitch;
  static constexpr int kXAt = kRows * kPitch;
  static constexpr int kScaleAt = kXAt + kTokens * kXPitch;
  static constexpr int kGroups = kColumns / 128;  // of columns with a scale
  static constexpr int kBytes = (kScaleAt + (kFp8 ? kRows / 8 * kGroups * 4 : 0) + 127) / 128 * 128;
};

template <bool kFp8, int kRows, int kTokens>
Plan plan_of(int T, int K, int E) {
  const uint32_t lanes = static_cast<uint32_t>(T) * K;
  auto up = [](uint32_t n) { return (n + 127u) & ~127u; };
  Plan p;
  p.token = 0;
  p.weight = up(lanes * 2);
  p.groups = p.weight + up(lanes * 4);
  p.sums = p.groups + up(lanes * 4);
  p.acc = p.sums + kWarps * kRows * kTokens * 4;
  p.ring = p.acc + up(static_cast<uint32_t>(T) * kRows * 4);
  p.stage = Stage<kFp8, kRows, kTokens>::kBytes;
  const uint32_t room = 220u * 1024u;
  p.stages = (room - p.ring) / p.stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  uint32_t ring = p.stages * p.stage;
  const uint32_t scratch = (2 * lanes + 2 * static_cast<uint32_t>(E)) * 4;  // of the lists, before the ring is used
  if (ring < scratch) ring = scratch;
  p.total = p.ring + ring;
  return p;
}

// kDown: the second kernel. kRows: matrix rows of a strip, kTokens: of a group at most.
template <bool kFp8, bool kDown, int kRows, int kTokens>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(LayerArgs a, Plan p) {
  constexpr int kM = kRows / 16, kN = kTokens / 8;
  using S = Stage<kFp8, kRows, kTokens>;
  constexpr int kColumns = S::kColumns, kPitch = S::kPitch, kXPitch = S::kXPitch, kXAt = S::kXAt, kScaleAt = S::kScaleAt;
  constexpr int kPiece = kFp8 ? 64 : 32;  // columns that a warp takes at once: 64 bytes of a matrix row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  __shared__ volatile int s_abort;
  __shared__ bool s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = static_cast<int>(p.stages);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init_count(smem_addr(&s_full[i]), kFp8 ? 33 : 1);  // with scales, every lane of the producer
      mbar_init_count(smem_addr(&s_empty[i]), kWarps);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if constexpr (!kDown) pdl_wait();
  // The second kernel may be placed as soon as what ran before the first is done: only h, which
  // its producer waits for, comes from the first.
  pdl_launch_dependents();
  const Lists lists = {reinterpret_cast<uint16_t*>(smem + p.token), reinterpret_cast<float*>(smem + p.weight),
                       reinterpret_cast<uint32_t*>(smem + p.groups)};
  float* acc_out = reinterpret_cast<float*>(smem + p.acc);  // [T][kRows]
  if constexpr (kDown)
    for (int i = threadIdx.x; i < a.T * kRows; i += kThreads) acc_out[i] = 0.f;
  const int groups = build_lists(a, kTokens, lists, reinterpret_cast<uint32_t*>(smem + p.ring),
                                 !kDown && blockIdx.x == 0 ? a.err : nullptr);
  fence_async_shared();  // the lists' scratch was where the ring is
  __syncthreads();

  const int sum = kDown ? a.I : a.H;                            // summed index
  const int z_rows = kDown ? a.H : a.Z;                         // rows of a matrix
  const bool gated = !kDown && a.act == EP_ACT_SWIGLU;
  const int out_rows = kDown ? a.H : a.I;                       // results a token
  const int strip = gated ? kRows / 2 : kRows;                  // results of a strip a token
  const int tiles = (out_rows + strip - 1) / strip;
  const int steps = (sum + kColumns - 1) / kColumns;
  // Down: a tile's groups are split in `split` parts where that evens the SMs' work out; the parts'
  // sums are added by the last to finish. By the device's SMs, so that results do not depend on num_sms.
  int split = 1;
  if constexpr (kDown) {
    int best = (tiles + a.device_sms - 1) / a.device_sms * groups;
    for (int s = 2; s <= min(kLayerMaxSplit, groups); ++s) {
      const int cost = (tiles * s + a.device_sms - 1) / a.device_sms * ((groups + s - 1) / s);
      if (cost < best) best = cost, split = s;
    }
  }
  const int64_t units = static_cast<int64_t>(tiles) * (kDown ? split : groups);

  // Every strip of this CTA in order: f(group, tile, part) until it says false.
  auto walk = [&](auto f) {
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
      const int part = static_cast<int>(u / tiles), tile = static_cast<int>(u - static_cast<int64_t>(part) * tiles);
      const int g0 = kDown ? groups * part / split : part, g1 = kDown ? groups * (part + 1) / split : part + 1;
      for (int g = g0; g < g1; ++g)
        if (!f(g, tile)) return;
    }
  };

  if (warp == kWarps) {
    const uint32_t ring = smem_addr(smem + p.ring);
    const uint8_t* matrices = static_cast<const uint8_t*>(kDown ? a.down : a.up);
    const float* scales = kDown ? a.down_sf : a.up_sf;
    const uint16_t* x = kDown ? a.h : a.x;
    const int bytes_a = kFp8 ? 1 : 2;
    const int scale_rows = (z_rows + 127) >> 7, scale_columns = sum >> 7;
    // matrix rows (and their scales) and token rows of one stage
    auto issue = [&](uint32_t n, int g, int tile, int step, bool rows, bool tokens) {
      const Group q = unpack_group(lists.groups[g]);
      const uint32_t s = n % stages, bar = smem_addr(&s_full[s]), at = ring + s * p.stage;
      const int c0 = step * kColumns, columns = min(kColumns, sum - c0);
      const uint32_t row_bytes = columns * bytes_a, x_bytes = columns * 2;
      // row i of the strip: gated, 8 rows of the gate, then the same 8 of the other half
      const int first = gated ? tile * strip : tile * kRows;
      auto row_of = [&](int i) { return gated ? (i & 8 ? a.I : 0) + first + (i >> 4) * 8 + (i & 7) : first + i; };
      auto there = [&](int i) { return gated ? first + (i >> 4) * 8 + (i & 7) < a.I : first + i < z_rows; };
      if (rows) {
        const bool mine = lane < kRows && there(lane);
        const unsigned all = __ballot_sync(kFullMask, mine);
        if (lane == 0) mbar_expect(bar, __popc(all) * row_bytes + q.n * x_bytes);
        __syncwarp();
        if (mine)
          bulk_row(at + lane * kPitch, matrices + ((static_cast<int64_t>(q.expert) * z_rows + row_of(lane)) * sum + c0) * bytes_a,
                   row_bytes, bar);
        if constexpr (kFp8) {  // scale [i / 8][column / 128] of the strip's rows
          constexpr int kGroups = S::kGroups;
          static_assert(kRows / 8 * kGroups <= 32, "a lane a scale");
          const int i = lane / kGroups * 8, c = (c0 >> 7) + lane % kGroups;
          if (i < kRows && there(i) && c < scale_columns) {
            const float* src = scales + (static_cast<int64_t>(q.expert) * scale_rows + (row_of(i) >> 7)) * scale_columns + c;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + kScaleAt + lane * 4), "l"(src) : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
      }
      if (tokens && lane < q.n) {
        const int64_t row = kDown ? q.start + lane : lists.token[q.start + lane];
        bulk_row(at + kXAt + lane * kXPitch, x + row * sum + c0, x_bytes, bar);
      }
    };
    uint32_t early = 0;
    if constexpr (kDown) {  // the first stages' matrix rows do not wait for h
      walk([&](int g, int tile) {
        for (int step = 0; step < steps; ++step) {
          if (early == static_cast<uint32_t>(stages)) return false;
          issue(early++, g, tile, step, true, false);
        }
        return true;
      });
      pdl_wait();
    }
    uint32_t n = 0;
    bool ok = true;
    walk([&](int g, int tile) {
      for (int step = 0; step < steps; ++step, ++n) {
        bool free = true;
        if (lane == 0) {
          free = s_abort == 0 && mbar_wait_timed<false>(smem_addr(&s_empty[n % stages]), (n / stages & 1u) ^ 1u);
          if (!free && s_abort == 0) atomicOr(a.err, kErrTimeout);
        }
        if (!__shfl_sync(kFullMask, free, 0)) {
          s_abort = 1;
          ok = false;
          return false;
        }
        issue(n, g, tile, step, n >= early, true);
      }
      return true;
    });
    if (!ok) {  // the copies in flight end before the CTA does
      if (n < early) {  // matrix rows whose tokens' rows were not asked for: their barriers do not complete
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) __nanosleep(1000);
      }
      for (uint32_t back = min(n, static_cast<uint32_t>(stages)); back > 0; --back) {
        const uint32_t m = n - back;
        mbar_wait_timed<false>(smem_addr(&s_full[m % stages]), m / stages & 1u);
      }
    }
    return;
  }

  // ---- the eight warps that multiply
  const int t = lane & 3, r8 = lane >> 2;
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  float4* sums = reinterpret_cast<float4*>(smem + p.sums);  // [warp][kM * kN][lane]
  uint32_t n = 0;
  int64_t u = blockIdx.x;
  for (; u < units; u += gridDim.x) {
    const int part = static_cast<int>(u / tiles), tile = static_cast<int>(u - static_cast<int64_t>(part) * tiles);
    const int g0 = kDown ? groups * part / split : part, g1 = kDown ? groups * (part + 1) / split : part + 1;
    for (int g = g0; g < g1; ++g) {
      const Group q = unpack_group(lists.groups[g]);
      const int used = (q.n + 7) >> 3;  // tiles of 8 tokens
      float d[kM][kN][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[m][j][i] = 0.f;
      for (int step = 0; step < steps; ++step, ++n) {
        const uint32_t s = n % stages;
        if (!s_abort && !mbar_wait_timed<false>(smem_addr(&s_full[s]), n / stages & 1u)) {
          if (!s_abort && lane == 0) atomicOr(a.err, kErrTimeout);
          s_abort = 1;  // what follows is not waited for: outputs are incomplete
        }
        __syncwarp();
        const uint8_t* stage = smem + p.ring + s * p.stage;
        const int columns = min(kColumns, sum - step * kColumns);
#pragma unroll
        for (int b = 0; b < S::kRowBytes / 64 / kWarps; ++b) {
          const int piece = b * kWarps + warp, c = piece * kPiece;
          if (c >= columns) break;
          const bool in = kFp8 || c + t * 8 < columns;  // 16 bytes of a row are all there, or none is
          const uint8_t* rows = stage + r8 * kPitch + piece * 64 + t * 16;
          const uint8_t* xs = stage + kXAt + r8 * kXPitch + c * 2 + t * (kFp8 ? 32 : 16);
          uint4 xv[kN][kFp8 ? 2 : 1];
#pragma unroll
          for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int h = 0; h < (kFp8 ? 2 : 1); ++h) {
              xv[j][h] = make_uint4(0u, 0u, 0u, 0u);
              if (j < used && in) xv[j][h] = *reinterpret_cast<const uint4*>(xs + j * 8 * kXPitch + h * 16);
            }
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
            if (in) {
              lo = *reinterpret_cast<const uint4*>(rows + m * 16 * kPitch);
              hi = *reinterpret_cast<const uint4*>(rows + (m * 16 + 8) * kPitch);
            }
            if constexpr (kFp8) {
              const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u4[4] = {hi.x, hi.y, hi.z, hi.w};
              const float* sf = reinterpret_cast<const float*>(stage + kScaleAt) + m * 2 * S::kGroups + (c >> 7);
              const float s0 = sf[0], s1 = sf[S::kGroups];
              float e[kN][4];
#pragma unroll
              for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) e[j][i] = 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t a0, a1, a2, a3;
                codes_to_bf16(l[k], a0, a2);
                codes_to_bf16(u4[k], a1, a3);
#pragma unroll
                for (int j = 0; j < kN; ++j)
                  if (j < used) {
                    const uint4 v = xv[j][k >> 1];
                    mma_16x8(e[j], a0, a1, a2, a3, k & 1 ? v.z : v.x, k & 1 ? v.w : v.y);
                  }
              }
#pragma unroll
              for (int j = 0; j < kN; ++j) {
                d[m][j][0] = fmaf(s0, e[j][0], d[m][j][0]);
                d[m][j][1] = fmaf(s0, e[j][1], d[m][j][1]);
                d[m][j][2] = fmaf(s1, e[j][2], d[m][j][2]);
                d[m][j][3] = fmaf(s1, e[j][3], d[m][j][3]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < kN; ++j)
                if (j < used) {
                  mma_16x8(d[m][j], lo.x, hi.x, lo.y, hi.y, xv[j][0].x, xv[j][0].y);
                  mma_16x8(d[m][j], lo.z, hi.z, lo.w, hi.w, xv[j][0].z, xv[j][0].w);
                }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_empty[s]));
      }
      // the eight warps' sums, in their order: a warp takes a tile of 16 x 8 of them
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (j < used) sums[(warp * kM * kN + m * kN + j) * 32 + lane] = make_float4(d[m][j][0], d[m][j][1], d[m][j][2], d[m][j][3]);
      consumers_sync();
#pragma unroll
      for (int i = warp; i < kM * kN; i += kWarps) {
        const int m = i / kN, j = i - m * kN;
        if (j >= used) continue;
        float4 v = none;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 o = sums[(w * kM * kN + i) * 32 + lane];
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        // v: results of rows r8 and r8 + 8 for tokens 2 t and 2 t + 1 of the tile
        const float got[2][2] = {{v.x, v.y}, {v.z, v.w}};
        if (gated) {
          const int c = tile * strip + m * 8 + r8;
          if (c < a.I) {
            float b0 = 0.f, b1 = 0.f;
            if (a.up_bias != nullptr) {
              const uint16_t* bias = a.up_bias + static_cast<int64_t>(q.expert) * a.Z + c;
              b0 = __uint_as_float(static_cast<uint32_t>(__ldg(bias)) << 16);
              b1 = __uint_as_float(static_cast<uint32_t>(__ldg(bias + a.I)) << 16);
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int token = j * 8 + 2 * t + o;
              const float h = activate<EP_ACT_SWIGLU>(got[0][o] + b0) * (got[1][o] + b1);
              if (token < q.n) a.h[static_cast<int64_t>(q.start + token) * a.I + c] = static_cast<uint16_t>(f32x2_to_bf16x2(h, 0.f));
            }
          }
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int in_strip = m * 16 + half * 8 + r8, c = tile * kRows + in_strip;
            if (c >= out_rows) continue;
            const uint16_t* bias = kDown ? a.down_bias : a.up_bias;
            float b = 0.f;
            if (bias != nullptr) b = __uint_as_float(static_cast<uint32_t>(__ldg(bias + static_cast<int64_t>(q.expert) * z_rows + c)) << 16);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int token = j * 8 + 2 * t + o;
              if (token >= q.n) continue;
              if constexpr (kDown) {
                float& to = acc_out[lists.token[q.start + token] * kRows + in_strip];
                to = fmaf(lists.weight[q.start + token], got[half][o] + b, to);
              } else {
                a.h[static_cast<int64_t>(q.start + token) * a.I + c] =
                    static_cast<uint16_t>(f32x2_to_bf16x2(act_any(got[half][o] + b, a.act), 0.f));
              }
            }
          }
        }
      }
      consumers_sync();
    }
    if constexpr (kDown) {  // the tile's tokens: 8 results a thread
      constexpr int kEights = kRows / 8;
      bool finish = split == 1;
      if (split > 1) {
        for (int i = threadIdx.x; i < a.T * kEights; i += kWarps * 32) {
          const int token = i / kEights, c = (i - token * kEights) * 8;
          if (tile * kRows + c >= a.H) continue;
          const float* v = acc_out + token * kRows + c;
          float* to = a.part + (static_cast<int64_t>(part) * a.T + token) * a.H + tile * kRows + c;
          *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(v);
          *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<const float4*>(v + 4);
        }
        __threadfence();
        consumers_sync();
        if (threadIdx.x == 0) {
          s_last = atomicAdd(a.done + tile, 1u) == static_cast<uint32_t>(split) - 1u;
          if (s_last) a.done[tile] = 0u;
        }
        consumers_sync();
        finish = s_last;
        __threadfence();
      }
      if (finish) {
        for (int i = threadIdx.x; i < a.T * kEights; i += kWarps * 32) {
          const int token = i / kEights, c = (i - token * kEights) * 8;
          if (tile * kRows + c >= a.H) continue;
          float v[8];
          if (split == 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = acc_out[token * kRows + c + k];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
            for (int s = 0; s < split; ++s) {
              const float* from = a.part + (static_cast<int64_t>(s) * a.T + token) * a.H + tile * kRows + c;
              const float4 l = __ldcg(reinterpret_cast<const float4*>(from)), h = __ldcg(reinterpret_cast<const float4*>(from + 4));
              v[0] += l.x, v[1] += l.y, v[2] += l.z, v[3] += l.w, v[4] += h.x, v[5] += h.y, v[6] += h.z, v[7] += h.w;
            }
          }
          const int64_t at = static_cast<int64_t>(token) * a.H + tile * kRows + c;
          if (a.residual != nullptr) {
            float r[8];
            unpack8(*reinterpret_cast<const uint4*>(a.residual + at), r);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += r[k];
          }
          st16(a.out + at, pack8(v));
        }
      }
      consumers_sync();
      for (int i = threadIdx.x; i < a.T * kRows; i += kWarps * 32) acc_out[i] = 0.f;
      consumers_sync();
    }
  }
}

template <bool kFp8, bool kDown, int kRows, int kTokens>
cudaError_t launch_one(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = layer_kernel<kFp8, kDown, kRows, kTokens>;
  const Plan p = plan_of<kFp8, kRows, kTokens>(a.T, a.K, a.E);
  if (p.stages < 2 || resident_ctas(reinterpret_cast<const void*>(kern), kThreads, p.total) < 1) return cudaErrorInvalidConfiguration;
  return launch_chained(kern, dim3(num_sms), dim3(kThreads), p.total, stream, a, p);
}

template <bool kFp8, int kRows, int kTokens>
cudaError_t launch_both(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t st = launch_one<kFp8, false, kRows, kTokens>(a, num_sms, stream);
  return st != cudaSuccess ? st : launch_one<kFp8, true, kRows, kTokens>(a, num_sms, stream);
}

template <bool kFp8>
cudaError_t launch_typed(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  if (a.T <= 4) return launch_both<kFp8, 16, 8>(a, num_sms, stream);
  if (a.T <= 8) return launch_both<kFp8, 32, 8>(a, num_sms, stream);
  // tokens to a group: most experts' tokens are one group
  return 2 * a.T * a.K <= 21 * a.E ? launch_both<kFp8, 32, 16>(a, num_sms, stream) : launch_both<kFp8, 32, 32>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_layer(const LayerArgs& a, bool fp8, int num_sms, cudaStream_t stream) {
  return fp8 ? launch_typed<true>(a, num_sms, stream) : launch_typed<false>(a, num_sms, stream);
}

}  // namespace ep
