// The experts' layer of a few tokens in two kernels, straight from the router's choice:
//
//   up    h_l = act(x_t W_up[e]^T + b_up[e])                      for every lane l = (t, k), e its expert
//   down  out_t = sum_k w_tk (h_l W_down[e]^T + b_down[e]) + residual_t
//
// Reading the chosen experts' matrices is what it costs (once for every 16 tokens of an expert), so both kernels are one stream of
// matrix rows through shared memory: loader warps keep a ring of stages full of them (TMA), eight or twelve
// worker warps take a stage each in turn and multiply it, and epilogue warps add their sums up. A strip is 16 or
// 32 matrix rows times all tokens of that expert (a group; tokens past kTokens are another group): the
// matrix rows are the 16 rows of mma.sync's A operand, the tokens its 8 columns, and a stage
// is a part of the summed index, so the strip's stages go to different workers.
// Up to 4 tokens h goes from one kernel to the other as two bf16 terms, the second kernel's products have
// columns for both, and the layer's error is that of its last rounding (1.6e-3 of its norm; with one term 2.4e-3).
// With more tokens the columns are taken, and h is rounded once, as ep_expert_product rounds it between the products: a
// second term would be a product of its own, and as many bytes of h again for every matrix row.
// With at most 16 tokens to a matrix the tensor cores are far from being the limit, so the products go
// where their operands need least preparation: the fragments are read straight from rows as they
// lie in memory (the summed index is permuted alike for both), and FP8 codes become bf16 on the way.
// (Sharing each stage among the workers took 165 us where this takes 136: a stage's bookkeeping then
// comes eight times, and every stage waits for its slowest warp.)
// Memory bounds it with bf16 matrices: 16 tokens on 16 experts of 4096 x 2048 136 us (805 MB, 5.9 TB/s), one token on 8
// experts of 7168 x 2048 106 us (705 MB, 6.6 TB/s); with FP8 ones the codes' way to bf16, two instructions a code
// and thread: 70 us (5.0 TB/s; 60 without the products).
#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kMaxStages = 48;
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
template <int kThreads>
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

// A place in the ring: the stage, and the parity of its barriers' phase.
struct Place {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) stage = 0, phase ^= 1u;
  }
};

// As mbar_wait_timed, which looks at the clock after its first try; here most waits end within a few. kBehind: the kernel
// in front, which may take its time, comes first: the wait is timed from its end.
template <bool kBehind = false>
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try<false>(bar, parity)) return true;
  if constexpr (kBehind) pdl_wait();
  return mbar_wait_timed<false>(bar, parity);
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
  uint32_t token, weight, groups, sums, acc, ring, stages, total;
};

// A kernel's shape. kSmall: for little work, with both kernels' CTAs on an SM together, so that the second has its
// lists and first stages ready when the first ends (one token on 4 experts of 1024 x 512: 11.3 instead
// of 13.1 us, of 2048 x 1024: 16.6 and 17.3); with more work the ring gets the whole SM (on 8 of 4096 x 1024: 41
// instead of 44 us, of 7168 x 2048: 110 instead of 125).
// A stage is matrix rows in columns of 128 bytes a row, as TMA writes them with the 128-byte swizzle. Its size
// bounds the tokens' values that a worker's threads hold beside it; a loader takes about 330 cycles for
// a copy, most of them for its wait, so that 4 KB ones would take four loaders (one: 207 us instead of 127).
template <bool kFp8_, int kRows_, int kTokens_, bool kSmall>
struct Shape {
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kRows = kRows_, kTokens = kTokens_;     // of a strip, of a group at most
  static constexpr int kWorkers = kFp8 && kTokens == 8 && !kSmall ? 12 : 8;
  static constexpr int kLoaders = kFp8 && kTokens == 8 && !kSmall ? 3 : 2;  // that take the stages in turn
  static constexpr int kEpilogue = kSmall || (kFp8 && kTokens == 8) ? 1 : 2;  // warps that take the units in turn
  static constexpr int kBytes = kFp8 && kSmall ? 4096 : 8192;
  static constexpr int kBoxes = kBytes / (kRows * 128);        // columns of 128 bytes
  static constexpr int kColumns = kBoxes * (kFp8 ? 128 : 64);  // of the summed index
  static constexpr int kPieces = 2 * kBoxes;                   // of 64 bytes a row
  static constexpr int kM = kRows / 16, kN = kTokens / 8;
  static constexpr int kCtas = kSmall ? 2 : 1;
  static constexpr int kSlots = kRows == 32 ? 2 : 4;           // strips whose sums may wait for each of them
  static constexpr int kThreads = (kWorkers + kLoaders + kEpilogue) * 32;
  // stages are as many to each worker, so with this a stage is always the same loader's too
  static_assert(kWorkers % kLoaders == 0, "a loader that waits for a stage has itself sent for it before");
};

template <class S>
Plan plan_of(int T, int K, int E) {
  const uint32_t lanes = static_cast<uint32_t>(T) * K;
  auto up = [](uint32_t n) { return (n + 127u) & ~127u; };
  Plan p;
  p.token = 0;
  p.weight = up(lanes * 2);
  p.groups = p.weight + up(lanes * 4);
  p.sums = p.groups + up(lanes * 4);
  p.acc = p.sums + S::kEpilogue * S::kSlots * S::kWorkers * S::kM * S::kN * 512;
  p.ring = (p.acc + static_cast<uint32_t>(T) * S::kRows * S::kEpilogue * 4 + 1023u) & ~1023u;
  const uint32_t room = (S::kCtas == 2 ? 111u : 224u) * 1024u;  // of 113 or 227 KB, static memory among it
  // As many to each worker, so that it is always the same one's: a worker that waits for a stage has then
  // itself emptied it before, and a barrier is never two phases behind what is waited for.
  p.stages = room > p.ring ? (room - p.ring) / S::kBytes / S::kWorkers * S::kWorkers : 0;
  if (p.stages > kMaxStages) p.stages = kMaxStages / S::kWorkers * S::kWorkers;
  uint32_t ring = p.stages * S::kBytes;
  const uint32_t scratch = (2 * lanes + 2 * static_cast<uint32_t>(E)) * 4;  // of the lists, before the ring is used
  if (ring < scratch) ring = scratch;
  p.total = p.ring + ring;
  return p;
}

// kDown: the second kernel.
template <class S, bool kDown>
__global__ void __launch_bounds__(S::kThreads, S::kCtas)
    layer_kernel(const __grid_constant__ CUtensorMap matrices, LayerArgs a, Plan p, int whole) {
  constexpr bool kFp8 = S::kFp8;
  constexpr int kRows = S::kRows, kTokens = S::kTokens;
  constexpr int kM = S::kM, kN = S::kN, kHalves = kFp8 ? 2 : 1;
  constexpr int kColumns = S::kColumns, kPieces = S::kPieces, kStageBytes = S::kBytes, kSlots = S::kSlots;
  constexpr int kPiece = kFp8 ? 64 : 32;  // columns of 64 bytes of a matrix row
  constexpr int kThreads = S::kThreads, kWorkers = S::kWorkers, kLoaders = S::kLoaders;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages];     // of the stages
  // of the strips' sums: every epilogue warp has its own, so that each barrier has one that waits for it, in order
  constexpr int kEpilogue = S::kEpilogue;
  __shared__ __align__(8) uint64_t s_strip_full[kEpilogue * kSlots], s_strip_empty[kEpilogue * kSlots];
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = static_cast<int>(p.stages);

  const int sum = kDown ? a.I : a.H;                            // summed index
  const int z_rows = kDown ? a.H : a.Z;                         // rows of a matrix
  const bool gated = !kDown && a.act == EP_ACT_SWIGLU;
  const int out_rows = kDown ? a.H : a.I;                       // results a token
  const int strip = gated ? kRows / 2 : kRows;                  // results of a strip a token
  const int tiles = (out_rows + strip - 1) / strip;
  const int steps = (sum + kColumns - 1) / kColumns;            // stages of a strip
  const int parts = min(steps, kWorkers);                       // workers that share it
  const int lanes = a.T * a.K;
  static_assert(kN == 1 || kTokens > 2 * kLayerPairTokens, "two terms for each token fit 8 columns");
  const bool pairs = kDown && kN == 1 && a.T <= kLayerPairTokens;  // columns 0 to 3 are the first terms of h, 4 to 7 the second

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init_count(smem_addr(&s_full[i]), 1);
      mbar_init_count(smem_addr(&s_empty[i]), 1);
    }
    for (int i = 0; i < kEpilogue * kSlots; ++i) {
      mbar_init_count(smem_addr(&s_strip_full[i]), kWorkers);
      mbar_init_count(smem_addr(&s_strip_empty[i]), 1);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&matrices);
  }
  if constexpr (!kDown) {
    pdl_wait();
    // What another size's call, or another operator, left in the workspace is no count of the second kernel's tiles.
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < (a.H + 15) / 16; i += gridDim.x * kThreads) a.done[i] = 0u;
  }
  // The second kernel may be placed as soon as what ran before the first is done: only h, which its
  // workers wait for, comes from the first. On a part of the SMs its CTAs would wait on those that are not the
  // call's, so they (and what comes behind the second) are placed once every CTA has sent for its last rows.
  if (static_cast<int>(gridDim.x) >= a.device_sms) pdl_launch_dependents();
  const Lists lists = {reinterpret_cast<uint16_t*>(smem + p.token), reinterpret_cast<float*>(smem + p.weight),
                       reinterpret_cast<uint32_t*>(smem + p.groups)};
  if constexpr (kDown)
    for (int i = threadIdx.x; i < a.T * kRows * S::kEpilogue; i += kThreads) reinterpret_cast<float*>(smem + p.acc)[i] = 0.f;
  const int groups = build_lists<kThreads>(a, kTokens, lists, reinterpret_cast<uint32_t*>(smem + p.ring),
                                           !kDown && blockIdx.x == 0 ? a.err : nullptr);
  fence_async_shared();  // the lists' scratch was where the ring is
  __syncthreads();

  // Down: a tile's groups are split in `split` parts where that evens the SMs' work out; the parts'
  // sums are added by the last to finish. In bytes of matrices, with what a unit's end costs beside them: a
  // part's, with its fence and atomic, about 20 KB and 32 bytes for each of its sums (without the latter 64 tokens,
  // top 4 of 16 experts, were 8 parts: 217 instead of 180 us); by the device's SMs, so that results do not depend
  // on num_sms.
  int split = 1;
  if constexpr (kDown) {
    const int64_t bytes = static_cast<int64_t>(kRows) * sum * (kFp8 ? 1 : 2);
    int64_t best = (tiles + a.device_sms - 1) / a.device_sms * (groups * bytes + 4096 + a.T * kRows * 8);
    for (int s = 2; s <= min(kLayerMaxSplit, groups); ++s) {
      const int64_t rounds = (static_cast<int64_t>(tiles) * s + a.device_sms - 1) / a.device_sms;
      const int64_t cost = rounds * ((groups + s - 1) / s * bytes + 20480 + a.T * kRows * 32);
      if (cost < best) best = cost, split = s;
    }
  }
  const int64_t units = static_cast<int64_t>(tiles) * (kDown ? split : groups);

  // The strips of this CTA in order: a tile's groups, then the next tile (up: one group each).
  struct Cursor {
    int64_t u;
    int tile, part, g, end;
    int turn = 0;  // the unit's epilogue warp
  };
  auto enter = [&](Cursor& c) {
    if (c.u >= units) return;
    c.part = static_cast<int>(c.u / tiles);
    c.tile = static_cast<int>(c.u - static_cast<int64_t>(c.part) * tiles);
    c.g = kDown ? groups * c.part / split : c.part;
    c.end = kDown ? groups * (c.part + 1) / split : c.part + 1;
  };
  auto advance = [&](Cursor& c) {
    if (++c.g < c.end) return;
    c.u += gridDim.x;
    if (kEpilogue > 1) c.turn ^= 1;
    enter(c);
  };
  static_assert(kEpilogue <= 2, "turns");
  auto give_up = [&] {
    if (s_abort == 0) atomicOr(a.err, kErrTimeout);
    s_abort = 1;
  };
  // A wait that gives up is the CTA's last one: what follows is computed without, and reported. Returns whether what it is
  // for is there.
  auto wait_for = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try<false>(smem_addr(bar), parity)) return true;
    if (s_abort != 0) return false;
    if (wait_stage(smem_addr(bar), parity)) return true;
    give_up();
    return false;
  };
  Cursor cur = {static_cast<int64_t>(blockIdx.x), 0, 0, 0, 0};
  enter(cur);
  const uint8_t* const ring = smem + p.ring;
  float4* const all_sums = reinterpret_cast<float4*>(smem + p.sums);  // [slot][part][kM * kN][lane]
  // The matrix rows of threads r8 = 2 i and 2 i + 1 are 4 apart, so that with the swizzle the eight 16-byte
  // pieces that 8 threads read at once lie in different banks.
  const int t = lane & 3, r8 = lane >> 2, row8 = r8 >> 1 | (r8 & 1) << 2;

  // Matrix rows: one thread of a loader warp, one copy a stage (of every kLoaders-th stage); what lies outside
  // a matrix reads as zero. A copy takes this thread about 330 cycles, most of them for the wait.
  if (warp >= kWorkers && warp < kWorkers + kLoaders) {
    if (elect_one() && groups > 0) {
      Place at;
      uint32_t n = 0;
      bool ok = true;
      for (; ok && cur.u < units; advance(cur)) {
        const Group q = unpack_group(lists.groups[cur.g]);
        const int plane = gated ? 2 * q.expert : q.expert, row = cur.tile * strip;
        for (int step = 0; step < steps; ++step, at.next(stages), ++n) {
          if (kLoaders > 1 && n % kLoaders != static_cast<uint32_t>(warp - kWorkers)) continue;
          // down: a full ring is emptied only behind the first kernel
          if (!wait_stage<kDown>(smem_addr(&s_empty[at.stage]), at.phase ^ 1u)) {
            give_up();
            ok = false;
            break;
          }
          const uint32_t bar = smem_addr(&s_full[at.stage]), to = smem_addr(ring + at.stage * kStageBytes);
          if (whole) {
            mbar_expect(bar, kStageBytes);
            tma_load_4d(to, &matrices, 0, row, plane, step * S::kBoxes, bar);
          } else {  // columns that are no multiple of 128 bytes: box by box
            const int boxes = min(S::kBoxes, (sum - step * kColumns + 63) / 64);
            mbar_expect(bar, boxes * kRows * 128);
            for (int i = 0; i < boxes; ++i) tma_load_3d(to + i * kRows * 128, &matrices, step * kColumns + i * 64, row, plane, bar);
          }
        }
      }
      pdl_launch_dependents();
      // the last copies end before the CTA does, also when a wait gave up, here or in a worker
      for (uint32_t m = n - min(n, p.stages); m < n; ++m)
        if (kLoaders == 1 || m % kLoaders == static_cast<uint32_t>(warp - kWorkers))
          mbar_wait_timed<false>(smem_addr(&s_full[m % p.stages]), m / p.stages & 1u);
    }
    if constexpr (kDown) pdl_wait();  // no CTA of this kernel ends before the first kernel
    return;
  }

  if (warp < kWorkers) {
    if constexpr (kDown) pdl_wait();
    if (groups == 0) return;
    const uint16_t* const x = kDown ? a.h : a.x;
    const float* const scales = kDown ? a.down_sf : a.up_sf;
    const int scale_rows = (z_rows + 127) >> 7, scale_columns = sum >> 7;
    const int lo_step = gated ? 8 : 16, hi_at = gated ? kRows / 2 : 8;  // rows of the strip: lo_step m + (0 or hi_at) + row8
    // What a stage's pieces meet: this thread's tokens' values (zeros behind the last column), and the scales.
    struct Beside {
      uint4 x[kPieces][kN][kHalves];
      float scale[kFp8 ? kPieces / 2 : 1][kFp8 ? kM : 1][2];
    };
    const uint16_t* from[kN];  // of the strip that is fetched: this thread's tokens' rows (past the last token: the last's)
    auto enter_strip = [&](const Cursor& c) {
      const Group q = unpack_group(lists.groups[c.g]);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int i = q.start + min(pairs ? r8 & 3 : j * 8 + r8, q.n - 1);
        const int64_t row = kDown ? i + (pairs && r8 > 3 ? lanes : 0) : lists.token[i];
        from[j] = x + row * sum + t * (kFp8 ? 16 : 8);
      }
    };
    auto fetch = [&](const Cursor& c, int step, Beside& b) {
      const int c0 = step * kColumns;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int column = c0 + i * kPiece;
        const bool in = kFp8 ? column < sum : column + t * 8 < sum;
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            b.x[i][j][h] = make_uint4(0u, 0u, 0u, 0u);
            if (in) b.x[i][j][h] = __ldcg(reinterpret_cast<const uint4*>(from[j] + column + h * 8));
          }
      }
      if constexpr (kFp8) {
        const int expert = unpack_group(lists.groups[c.g]).expert;
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = c.tile * strip + (gated ? m * 8 + h * a.I : m * 16 + h * 8);
            const float* sf = scales + (static_cast<int64_t>(expert) * scale_rows + (row >> 7)) * scale_columns;
#pragma unroll
            for (int i = 0; i < kPieces / 2; ++i) {
              const int k = (c0 >> 7) + i;
              b.scale[i][m][h] = k < scale_columns ? __ldg(sf + k) : 0.f;
            }
          }
      }
    };
    int step = warp, stage = warp;
    uint32_t phase = 0, strips[2] = {0, 0};  // for each epilogue warp
    // This worker's share of a strip's sums, if it has one; every worker keeps pace with the strips' barriers.
    auto leave_strip = [&](int turn, auto put) {
      const uint32_t count = turn ? strips[1] : strips[0], slot = turn * kSlots + count % kSlots;
      wait_for(&s_strip_empty[slot], (count / kSlots & 1u) ^ 1u);
      put(all_sums + slot * kWorkers * (kM * kN * 32) + lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_strip_full[slot]));
      if (turn) ++strips[1];
      else ++strips[0];
    };
    const auto nothing = [](float4*) {};
    for (; cur.u < units && step >= steps; step -= steps, advance(cur)) leave_strip(cur.turn, nothing);
    if (cur.u >= units) return;
    int first = step;
    float d[kM][kN][4];
    auto clear = [&] {
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[m][j][i] = 0.f;
    };
    clear();
    enter_strip(cur);
    while (cur.u < units) {
      const int c0 = step * kColumns;
      Beside b;
      fetch(cur, step, b);  // while the matrix rows are on their way
      Cursor then = cur;
      int passed = 0;
      for (step += kWorkers; step >= steps && then.u < units; step -= steps, ++passed) advance(then);
      const bool landed = wait_for(&s_full[stage], phase);
      __syncwarp();
      const uint8_t* rows = ring + stage * kStageBytes + row8 * 128;
      // Sums before their scale: of its 128 columns (two pieces) where the registers hold them, else of a piece.
      constexpr bool kPair = kM * kN <= 2;
      float e[kFp8 ? (kPair ? kM : 1) : 1][kFp8 ? kN : 1][4];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        if (c0 + i * kPiece >= sum) break;
        const uint8_t* piece = rows + (i >> 1) * (kRows * 128) + ((((i & 1) << 2) + t) ^ row8) * 16;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const uint4 lo = *reinterpret_cast<const uint4*>(piece + m * lo_step * 128);
          const uint4 hi = *reinterpret_cast<const uint4*>(piece + (m * lo_step + hi_at) * 128);
          if constexpr (kFp8) {
            const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u4[4] = {hi.x, hi.y, hi.z, hi.w};
            if (!kPair || (i & 1) == 0) {
#pragma unroll
              for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) e[kPair ? m : 0][j][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a0, a1, a2, a3;
              codes_to_bf16(l[k], a0, a2);
              codes_to_bf16(u4[k], a1, a3);
#pragma unroll
              for (int j = 0; j < kN; ++j) {  // both tiles of 8 tokens: that costs less than asking
                const uint4 v = b.x[i][j][k >> 1];
                mma_16x8(e[kPair ? m : 0][j], a0, a1, a2, a3, k & 1 ? v.z : v.x, k & 1 ? v.w : v.y);
              }
            }
            if (!kPair || (i & 1)) {  // columns come in whole 128s
              const float s0 = b.scale[i >> 1][m][0], s1 = b.scale[i >> 1][m][1];
#pragma unroll
              for (int j = 0; j < kN; ++j) {
                d[m][j][0] = fmaf(s0, e[kPair ? m : 0][j][0], d[m][j][0]);
                d[m][j][1] = fmaf(s0, e[kPair ? m : 0][j][1], d[m][j][1]);
                d[m][j][2] = fmaf(s1, e[kPair ? m : 0][j][2], d[m][j][2]);
                d[m][j][3] = fmaf(s1, e[kPair ? m : 0][j][3], d[m][j][3]);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              const uint4 v = b.x[i][j][0];
              mma_16x8(d[m][j], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
              mma_16x8(d[m][j], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
            }
          }
        }
      }
      __syncwarp();
      // A stage that was not waited for is not handed on: its copy may still be on the way, and a loader that has not given
      // up must not announce a second one beside it. (Loaders that look at s_abort took 10% longer where few SMs are
      // used and each is fast: 64 tokens, top 8 of 64 experts on 20 SMs 2.80 instead of 2.54 ms.)
      if (lane == 0 && landed) mbar_arrive(smem_addr(&s_empty[stage]));
      if ((stage += kWorkers) >= stages) stage -= stages, phase ^= 1u;
      if (passed > 0) {
        leave_strip(cur.turn, [&](float4* sums) {
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int j = 0; j < kN; ++j)
              sums[(first * kM * kN + m * kN + j) * 32] = make_float4(d[m][j][0], d[m][j][1], d[m][j][2], d[m][j][3]);
        });
        for (advance(cur); passed > 1; --passed, advance(cur)) leave_strip(cur.turn, nothing);
        first = step;
        clear();
        if (then.u < units) enter_strip(then);
      }
      cur = then;
    }
    return;
  }

  // ---- the epilogue warps: a strip's shares added in their order, 16 x 8 results at a time. They take the
  // units (tiles) in turn, so that one ends a tile while another begins the next.
  const int index = warp - kWorkers - kLoaders;
  float* const acc_out = reinterpret_cast<float*>(smem + p.acc) + index * a.T * kRows;  // [T][kRows]
  if constexpr (kDown) pdl_wait();  // `out` may be what the first kernel reads
  auto put_h = [&](int lane_at, int c, float h) {
    uint16_t* to = a.h + static_cast<int64_t>(lane_at) * a.I + c;
    const uint32_t first = f32x2_to_bf16x2(h, 0.f) & 0xFFFFu;
    *to = static_cast<uint16_t>(first);
    if (kN == 1 && a.T <= kLayerPairTokens)
      to[static_cast<int64_t>(lanes) * a.I] = static_cast<uint16_t>(f32x2_to_bf16x2(h - __uint_as_float(first << 16), 0.f));
  };
  uint32_t strips = 0;
  for (int turn = 0; cur.u < units; turn = turn + 1 == kEpilogue ? 0 : turn + 1) {
    const Cursor unit = cur;
    if (turn != index) {
      cur.u += gridDim.x;
      enter(cur);
      continue;
    }
    for (; cur.u == unit.u && groups > 0; advance(cur), ++strips) {
      const Group q = unpack_group(lists.groups[cur.g]);
      const uint32_t slot = index * kSlots + strips % kSlots;
      const float4* sums = all_sums + slot * kWorkers * (kM * kN * 32) + lane;
      wait_for(&s_strip_full[slot], strips / kSlots & 1u);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kM * kN; ++i) {
        const int m = i / kN, j = i - m * kN;
        if (j * 8 >= q.n) continue;
        float4 v = sums[i * 32];
        for (int w = 1; w < parts; ++w) {
          const float4 o = sums[(w * (kM * kN) + i) * 32];
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        if (pairs) {  // both terms' products: the second's is four columns, two threads on
          auto add_second = [](float& first) {  // an infinity of h or of the matrix stays what the first term makes it
            const float second = __shfl_xor_sync(kFullMask, first, 2);
            if (fabsf(first) < INFINITY) first += second;
          };
          add_second(v.x), add_second(v.y), add_second(v.z), add_second(v.w);
        }
        // v: results of rows row8 and row8 + 8 for tokens 2 t and 2 t + 1 of the tile
        const float got[2][2] = {{v.x, v.y}, {v.z, v.w}};
        if (gated) {
          const int c = cur.tile * strip + m * 8 + row8;
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
              if (token < q.n) put_h(q.start + token, c, h);
            }
          }
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int in_strip = m * 16 + half * 8 + row8, c = cur.tile * kRows + in_strip;
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
                put_h(q.start + token, c, act_any(got[half][o] + b, a.act));
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_strip_empty[slot]));
    }
    if constexpr (kDown) {  // the tile's tokens: 8 results a thread
      constexpr int kEights = kRows / 8;
      bool finish = split == 1;
      if (split > 1) {
        for (int i = lane; i < a.T * kEights; i += 32) {
          const int token = i / kEights, c = (i - token * kEights) * 8;
          if (unit.tile * kRows + c >= a.H) continue;
          const float* v = acc_out + token * kRows + c;
          float* to = a.part + (static_cast<int64_t>(unit.part) * a.T + token) * a.H + unit.tile * kRows + c;
          *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(v);
          *reinterpret_cast<float4*>(to + 4) = *reinterpret_cast<const float4*>(v + 4);
        }
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) before = atomicAdd(a.done + unit.tile, 1u);
        finish = __shfl_sync(kFullMask, before, 0) == static_cast<uint32_t>(split) - 1u;
        if (finish && lane == 0) a.done[unit.tile] = 0u;
        __threadfence();
      }
      if (finish) {
        for (int i = lane; i < a.T * kEights; i += 32) {
          const int token = i / kEights, c = (i - token * kEights) * 8;
          if (unit.tile * kRows + c >= a.H) continue;
          float v[8];
          if (split == 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = acc_out[token * kRows + c + k];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll 4
            for (int s = 0; s < split; ++s) {
              const float* from = a.part + (static_cast<int64_t>(s) * a.T + token) * a.H + unit.tile * kRows + c;
              const float4 l = __ldcg(reinterpret_cast<const float4*>(from)), h = __ldcg(reinterpret_cast<const float4*>(from + 4));
              v[0] += l.x, v[1] += l.y, v[2] += l.z, v[3] += l.w, v[4] += h.x, v[5] += h.y, v[6] += h.z, v[7] += h.w;
            }
          }
          const int64_t at = static_cast<int64_t>(token) * a.H + unit.tile * kRows + c;
          if (a.residual != nullptr) {
            float r[8];
            unpack8(*reinterpret_cast<const uint4*>(a.residual + at), r);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += r[k];
          }
          st16(a.out + at, pack8(v));
        }
      }
      __syncwarp();
      for (int i = lane; i < a.T * kRows; i += 32) acc_out[i] = 0.f;
      __syncwarp();
      if (groups == 0) {
        cur.u += gridDim.x;
        enter(cur);
      }
    }
  }
}

template <class S, bool kDown>
cudaError_t launch_one(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  constexpr bool kFp8 = S::kFp8;
  constexpr int kRows = S::kRows;
  auto kern = layer_kernel<S, kDown>;
  const Plan p = plan_of<S>(a.T, a.K, a.E);
  if (p.stages < S::kWorkers || resident_ctas(reinterpret_cast<const void*>(kern), S::kThreads, p.total) < 1)
    return cudaErrorInvalidConfiguration;
  // 16-bit elements (two codes each); gated, the gate rows and the others of an expert are planes of their own
  const bool gated = !kDown && a.act == EP_ACT_SWIGLU;
  const uint64_t columns = static_cast<uint64_t>(kDown ? a.I : a.H) / (kFp8 ? 2 : 1), rows = kDown ? a.H : a.I;
  const uint64_t planes = static_cast<uint64_t>(a.E) * (gated ? 2 : 1);
  const uint32_t box_rows = gated ? kRows / 2 : kRows, box_planes = gated ? 2 : 1;
  const int whole = columns % 64 == 0;  // then one copy brings all columns of a stage
  CUtensorMap map;
  cudaError_t st;
  if (whole) {
    const uint64_t size[4] = {64, rows, planes, columns / 64}, stride[3] = {2 * columns, 2 * columns * rows, 128};
    const uint32_t box[4] = {64, box_rows, box_planes, S::kBoxes};
    st = make_strided_map(&map, kDown ? a.down : a.up, 4, size, stride, box);
  } else {
    const uint64_t size[3] = {columns, rows, planes};
    const uint32_t box[3] = {64, box_rows, box_planes};
    st = make_tensor_map(&map, kDown ? a.down : a.up, 3, size, box);
  }
  if (st != cudaSuccess) return st;
  return launch_chained(kern, dim3(num_sms), dim3(S::kThreads), p.total, stream, map, a, p, whole);
}

template <class S>
cudaError_t launch_both(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t st = launch_one<S, false>(a, num_sms, stream);
  return st != cudaSuccess ? st : launch_one<S, true>(a, num_sms, stream);
}

template <bool kFp8>
cudaError_t launch_typed(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  if (a.T <= 8) {
    // Matrices that are read, at most: 600 KB an SM lies between where the small shape is the faster one (0.33 MB: 16.6 and
    // 17.3 us) and where the other is (FP8, 0.66 MB: 37.4 and 34.0 us; bf16, 1.3 MB: 44.1 and 41.4).
    const int64_t lanes = static_cast<int64_t>(a.T) * a.K, experts = lanes < a.E ? lanes : a.E;
    const int64_t bytes = experts * (static_cast<int64_t>(a.Z) + a.I) * a.H * (kFp8 ? 1 : 2);
    if (bytes <= 614400ll * a.device_sms && plan_of<Shape<kFp8, 16, 8, true>>(a.T, a.K, a.E).stages >= 8)
      return launch_both<Shape<kFp8, 16, 8, true>>(a, num_sms, stream);
    // FP8, strips of 16 rows and of 32: 7168 x 2048 with 1, 2, 3, 4, 8 tokens 70, 97, 111, 127, 134 and 75, 104, 115, 130,
    // 135 us; 4096 x 2048 48, 65, 75, 84, 89 and 48, 63, 72, 80, 86. So up to two tokens those of 16 rows are as good or
    // better by up to 7%; from three on it is 1 to 4% either way, with how evenly the tiles of a size fill the SMs.
    if constexpr (kFp8)
      if (a.T > 2) return launch_both<Shape<kFp8, 32, 8, false>>(a, num_sms, stream);
    return launch_both<Shape<kFp8, 16, 8, false>>(a, num_sms, stream);
  }
  // Another group of the same expert reads its matrix again, from L2 as far as that holds it (the first kernel takes all
  // tiles of a group before the next group's, the second a tile's groups in turn); groups of 32 instead took as long or longer
  // (64 tokens, top 2 of 8 experts: 105 us instead of 108, of 4: 92 instead of 86; top 8 of 16: 282 and 285).
  return launch_both<Shape<kFp8, 32, 16, false>>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_layer(const LayerArgs& a, bool fp8, int num_sms, cudaStream_t stream) {
  return fp8 ? launch_typed<true>(a, num_sms, stream) : launch_typed<false>(a, num_sms, stream);
}

}  // namespace ep
