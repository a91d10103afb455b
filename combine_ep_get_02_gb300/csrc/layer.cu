// The experts' layer of a few tokens in two kernels, straight from the router's choice:
//
//   up    h_l = act(x_t W_up[e]^T + b_up[e])                      for every lane l = (t, k), e its expert
//   down  out_t = sum_k w_tk (h_l W_down[e]^T + b_down[e]) + residual_t
//
// Reading the chosen experts' matrices once is what it costs, so both kernels are one stream of
// matrix rows through shared memory: a warp keeps a ring of stages full of them (TMA) and eight warps
// multiply, whose threads fetch their own pieces of the tokens' rows (small, in L2) a few stages ahead. A work item is a strip of 16 or 32 matrix rows times all tokens
// of that expert (a group; tokens past kTokens are another group): the matrix rows are the 16 rows
// of mma.sync's A operand, the tokens its 8 columns, and the eight warps share the summed index.
// With at most 32 tokens to a matrix the tensor cores are far from being the limit, so the products go
// where their operands need least preparation: the fragments are read straight from rows as they
// lie in memory (the summed index is permuted alike for both), and FP8 codes become bf16 on the way.
#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kWarps = 8;                        // that multiply
constexpr int kThreads = (kWarps + 1) * 32;      // with the one that loads
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

// A place in the ring: the stage, and the parity of its barriers' phase.
struct Place {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) stage = 0, phase ^= 1u;
  }
};

// As mbar_wait_timed, which looks at the clock after its first try; here most waits end within a few.
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try<false>(bar, parity)) return true;
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
  uint32_t token, weight, groups, sums, beside, acc, ring, stages, total;
};

// A stage: 16 KB of matrix rows in columns of 128 bytes a row, as TMA writes them with the 128-byte swizzle.
constexpr int kStageBytes = 16384;
template <bool kFp8, int kRows, int kTokens>
struct Stage {
  static constexpr int kBoxes = kStageBytes / (kRows * 128);   // columns of 128 bytes
  static constexpr int kColumns = kBoxes * (kFp8 ? 128 : 64);  // of the summed index
  static constexpr int kPieces = 2 * kBoxes / kWarps;          // of 64 bytes a row, for each warp
  // What a warp's pieces meet: for each thread (of 4 tokens' in (16, 4)) 16 bytes of each token tile's row, twice
  // with FP8, and then the scales. Fetched kAhead stages ahead.
  static constexpr int kM = kRows / 16, kN = (kTokens + 7) / 8;
  static constexpr int kLanes = kTokens < 8 ? 4 * kTokens : 32;
  static constexpr int kBesideBytes = kPieces * kN * (kFp8 ? 2 : 1) * kLanes * 16 + (kFp8 ? kPieces * kM * 8 : 0);
  static constexpr int kAhead = kFp8 && kTokens > 16 ? 2 : 4;
  // Few tokens: both kernels' CTAs fit an SM together, so that the second has its lists and first stages ready
  // when the first ends. With more there is more to do, and the ring gets the whole SM.
  static constexpr int kCtas = kTokens <= (kFp8 ? 4 : 8) ? 2 : 1;
};

template <bool kFp8, int kRows, int kTokens>
Plan plan_of(int T, int K, int E) {
  using S = Stage<kFp8, kRows, kTokens>;
  const uint32_t lanes = static_cast<uint32_t>(T) * K;
  auto up = [](uint32_t n) { return (n + 127u) & ~127u; };
  Plan p;
  p.token = 0;
  p.weight = up(lanes * 2);
  p.groups = p.weight + up(lanes * 4);
  p.sums = p.groups + up(lanes * 4);
  p.beside = p.sums + 2 * kWarps * kRows * S::kN * 8 * 4;
  p.acc = p.beside + up(kWarps * S::kAhead * S::kBesideBytes);
  p.ring = (p.acc + static_cast<uint32_t>(T) * kRows * 4 + 1023u) & ~1023u;
  const uint32_t room = (S::kCtas == 2 ? 111u : 224u) * 1024u;  // of 113 or 227 KB, static memory among it
  p.stages = room > p.ring ? (room - p.ring) / kStageBytes : 0;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  uint32_t ring = p.stages * kStageBytes;
  const uint32_t scratch = (2 * lanes + 2 * static_cast<uint32_t>(E)) * 4;  // of the lists, before the ring is used
  if (ring < scratch) ring = scratch;
  p.total = p.ring + ring;
  return p;
}

// kDown: the second kernel. kRows: matrix rows of a strip, kTokens: of a group at most.
template <bool kFp8, bool kDown, int kRows, int kTokens>
__global__ void __launch_bounds__(kThreads, Stage<kFp8, kRows, kTokens>::kCtas)
    layer_kernel(const __grid_constant__ CUtensorMap matrices, LayerArgs a, Plan p, int whole) {
  using S = Stage<kFp8, kRows, kTokens>;
  constexpr int kM = S::kM, kN = S::kN, kHalves = kFp8 ? 2 : 1, kAhead = S::kAhead;
  constexpr int kColumns = S::kColumns, kPieces = S::kPieces;
  constexpr int kPiece = kFp8 ? 64 : 32;           // columns that a warp takes at once: 64 bytes of a matrix row
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages];
  __shared__ volatile int s_abort;
  __shared__ bool s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = static_cast<int>(p.stages);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init_count(smem_addr(&s_full[i]), 1);
      mbar_init_count(smem_addr(&s_empty[i]), kWarps);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&matrices);
  }
  if constexpr (!kDown) pdl_wait();
  // The second kernel may be placed as soon as what ran before the first is done: only h, which the warps
  // that multiply wait for, comes from the first.
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

  // The stages of this CTA in order: all of the summed index of a strip, the strips of a tile's groups, the tiles.
  struct Cursor {
    int64_t u;
    int tile, part, g, end, step;
  };
  auto enter = [&](Cursor& c) {
    if (c.u >= units) return;
    c.part = static_cast<int>(c.u / tiles);
    c.tile = static_cast<int>(c.u - static_cast<int64_t>(c.part) * tiles);
    c.g = kDown ? groups * c.part / split : c.part;
    c.end = kDown ? groups * (c.part + 1) / split : c.part + 1;
    c.step = 0;
  };
  auto advance = [&](Cursor& c) {
    if (++c.step < steps) return;
    c.step = 0;
    if (++c.g < c.end) return;
    c.u += gridDim.x;
    enter(c);
  };
  Cursor cur = {blockIdx.x, 0, 0, 0, 0, 0};
  // no group, no stage: there is still the output
  if (groups > 0) enter(cur);
  const uint8_t* const ring = smem + p.ring;
  Place at;

  if (warp == kWarps) {  // matrix rows: one thread, one copy a stage; what lies outside a matrix reads as zero
    if (elect_one() && groups > 0) {
      uint32_t n = 0;
      for (; cur.u < units; advance(cur), at.next(stages), ++n) {
        if (s_abort != 0 || !wait_stage(smem_addr(&s_empty[at.stage]), at.phase ^ 1u)) {
          if (s_abort == 0) atomicOr(a.err, kErrTimeout);
          s_abort = 1;  // the copies in flight end before the CTA does
          for (uint32_t m = n - min(n, p.stages); m < n; ++m)
            mbar_wait_timed<false>(smem_addr(&s_full[m % p.stages]), m / p.stages & 1u);
          break;
        }
        const Group q = unpack_group(lists.groups[cur.g]);
        const int plane = gated ? 2 * q.expert : q.expert, row = cur.tile * strip;
        const uint32_t bar = smem_addr(&s_full[at.stage]), to = smem_addr(ring + at.stage * kStageBytes);
        if (whole) {
          mbar_expect(bar, kStageBytes);
          tma_load_4d(to, &matrices, 0, row, plane, cur.step * S::kBoxes, bar);
        } else {  // columns that are no multiple of 128 bytes: box by box
          const int boxes = min(S::kBoxes, (sum - cur.step * kColumns + 63) / 64);
          mbar_expect(bar, boxes * kRows * 128);
          for (int i = 0; i < boxes; ++i) tma_load_3d(to + i * kRows * 128, &matrices, cur.step * kColumns + i * 64, row, plane, bar);
        }
      }
    }
    if constexpr (kDown) pdl_wait();  // no CTA of this kernel ends before the first kernel
    return;
  }

  // ---- the eight warps that multiply
  const int t = lane & 3, r8 = lane >> 2;
  // The matrix rows of threads r8 = 2 i and 2 i + 1 are 4 apart, so that with the swizzle the eight 16-byte
  // pieces that 8 threads read at once lie in different banks.
  const int row8 = r8 >> 1 | (r8 & 1) << 2;
  // [turn][warp][kM * kN][lane]: two buffers, so that one barrier a strip is enough
  float4* all_sums = reinterpret_cast<float4*>(smem + p.sums);
  const int lo_step = gated ? 8 : 16, hi_at = gated ? kRows / 2 : 8;  // rows of the strip: lo_step m + (0 or hi_at) + row8

  // The pieces of a stage that is `kAhead` ahead, by each thread for itself (so no barrier stands between
  // them and their use, but a warp's for the scales): zeros behind the last column.
  const uint16_t* const x = kDown ? a.h : a.x;
  const float* const scales = kDown ? a.down_sf : a.up_sf;
  const int scale_rows = (z_rows + 127) >> 7, scale_columns = sum >> 7;
  uint8_t* const beside = smem + p.beside + warp * (kAhead * S::kBesideBytes);
  const int slot = (kTokens < 8 ? lane & (S::kLanes - 1) : lane) * 16;
  const uint16_t* from[kN];         // of the strip that is fetched: this thread's tokens' rows
  const float* scale_at = nullptr;  // this lane's, of [kPieces][kM][2]
  Cursor ahead = cur;
  int place = 0;  // of kAhead
  auto fetch = [&] {
    if (ahead.u < units) {
      if (ahead.step == 0) {
        const Group q = unpack_group(lists.groups[ahead.g]);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const int i = q.start + j * 8 + r8;
          from[j] = j * 8 + r8 < q.n ? x + static_cast<int64_t>(kDown ? i : lists.token[i]) * sum + t * (kFp8 ? 16 : 8) : nullptr;
        }
        if constexpr (kFp8) {
          const int h = lane & 1, m = (lane >> 1) % kM;
          const int row = ahead.tile * strip + (gated ? m * 8 + h * a.I : m * 16 + h * 8);
          scale_at = scales + (static_cast<int64_t>(q.expert) * scale_rows + (row >> 7)) * scale_columns;
        }
      }
      const uint32_t to = smem_addr(beside + place * S::kBesideBytes);
      const int c0 = ahead.step * kColumns;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int column = c0 + (i * kWarps + warp) * kPiece;
        const int bytes = (kFp8 ? column < sum : column + t * 8 < sum) ? 16 : 0;
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            if (from[j] != nullptr)  // columns without a token are nobody's
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               to + ((i * kN + j) * kHalves + h) * (S::kLanes * 16) + slot),
                           "l"(from[j] + (bytes ? column + h * 8 : 0)), "r"(bytes)
                           : "memory");
      }
      if constexpr (kFp8) {
        const int column = c0 + (lane / (2 * kM) * kWarps + warp) * kPiece;
        if (lane < kPieces * kM * 2 && column < sum)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + kPieces * kN * kHalves * (S::kLanes * 16) + lane * 4),
                       "l"(scale_at + (column >> 7))
                       : "memory");
      }
      advance(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++place == kAhead) place = 0;
  };

  if constexpr (kDown) pdl_wait();
  uint32_t strips = 0;
  if (groups == 0) ahead.u = units;
#pragma unroll 1
  for (int i = 0; i < kAhead - 1; ++i) fetch();
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = static_cast<int>(u / tiles), tile = static_cast<int>(u - static_cast<int64_t>(part) * tiles);
    const int g0 = kDown ? groups * part / split : part, g1 = kDown ? groups * (part + 1) / split : part + 1;
    for (int g = g0; g < g1; ++g, ++strips) {
      const Group q = unpack_group(lists.groups[g]);
      float4* sums = all_sums + (strips & 1u) * (kWarps * kM * kN * 32);
      // tiles of 8 tokens; of two both are computed, as that costs less than asking
      const int used = kN > 2 ? (q.n + 15) >> 4 << 1 : kN;
      float d[kM][kN][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[m][j][i] = 0.f;
      for (int step = 0; step < steps; ++step) {
        const uint8_t* here = beside + (place + 1 == kAhead ? 0 : place + 1) * S::kBesideBytes + slot;
        const float* sf = reinterpret_cast<const float*>(here - slot + kPieces * kN * kHalves * (S::kLanes * 16));
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        // a wait that gives up is the last one: what follows is computed without, and reported
        const uint32_t bar = smem_addr(&s_full[at.stage]);
        if (!mbar_try<false>(bar, at.phase) && s_abort == 0 && !wait_stage(bar, at.phase)) {
          if (s_abort == 0) atomicOr(a.err, kErrTimeout);
          s_abort = 1;
        }
        __syncwarp();
        const uint8_t* stage = ring + at.stage * kStageBytes;
        const int columns = sum - step * kColumns;
#pragma unroll
        for (int b = 0; b < kPieces; ++b) {
          const int piece = b * kWarps + warp;
          if (piece * kPiece >= columns) break;
          const uint8_t* rows = stage + (piece >> 1) * (kRows * 128) + row8 * 128 + ((((piece & 1) << 2) + t) ^ row8) * 16;
          uint4 xv[kN][kHalves];
#pragma unroll
          for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              xv[j][h] = *reinterpret_cast<const uint4*>(here + ((b * kN + j) * kHalves + h) * (S::kLanes * 16));
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const uint4 lo = *reinterpret_cast<const uint4*>(rows + m * lo_step * 128);
            const uint4 hi = *reinterpret_cast<const uint4*>(rows + (m * lo_step + hi_at) * 128);
            if constexpr (kFp8) {
              const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u4[4] = {hi.x, hi.y, hi.z, hi.w};
              const float s0 = sf[(b * kM + m) * 2], s1 = sf[(b * kM + m) * 2 + 1];
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
                  const uint4 v = xv[j][0];
                  mma_16x8(d[m][j], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
                  mma_16x8(d[m][j], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
                }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_empty[at.stage]));
        at.next(stages);
      }
      // the eight warps' sums, in their order: a warp takes a tile of 16 x 8 of them
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (j < used) sums[(warp * kM * kN + m * kN + j) * 32 + lane] = make_float4(d[m][j][0], d[m][j][1], d[m][j][2], d[m][j][3]);
      consumers_sync();
#pragma unroll
      for (int i = static_cast<int>((warp - strips) & (kWarps - 1)); i < kM * kN; i += kWarps) {  // the warps take turns
        const int m = i / kN, j = i - m * kN;
        if (j >= used) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 o = sums[(w * kM * kN + i) * 32 + lane];
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        // v: results of rows row8 and row8 + 8 for tokens 2 t and 2 t + 1 of the tile
        const float got[2][2] = {{v.x, v.y}, {v.z, v.w}};
        if (gated) {
          const int c = tile * strip + m * 8 + row8;
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
            const int in_strip = m * 16 + half * 8 + row8, c = tile * kRows + in_strip;
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
    }
    if constexpr (kDown) {  // the tile's tokens: 8 results a thread
      consumers_sync();
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
  using S = Stage<kFp8, kRows, kTokens>;
  const Plan p = plan_of<kFp8, kRows, kTokens>(a.T, a.K, a.E);
  if (p.stages < 2 || resident_ctas(reinterpret_cast<const void*>(kern), kThreads, p.total) < 1) return cudaErrorInvalidConfiguration;
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
  return launch_chained(kern, dim3(num_sms), dim3(kThreads), p.total, stream, map, a, p, whole);
}

template <bool kFp8, int kRows, int kTokens>
cudaError_t launch_both(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t st = launch_one<kFp8, false, kRows, kTokens>(a, num_sms, stream);
  return st != cudaSuccess ? st : launch_one<kFp8, true, kRows, kTokens>(a, num_sms, stream);
}

template <bool kFp8>
cudaError_t launch_typed(const LayerArgs& a, int num_sms, cudaStream_t stream) {
  if (a.T <= 4) return launch_both<kFp8, 16, 4>(a, num_sms, stream);
  if (a.T <= 8) return launch_both<kFp8, 16, 8>(a, num_sms, stream);
  // tokens to a group: most experts' tokens are one group
  return 2 * a.T * a.K <= 21 * a.E ? launch_both<kFp8, 32, 16>(a, num_sms, stream) : launch_both<kFp8, 32, 32>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_layer(const LayerArgs& a, bool fp8, int num_sms, cudaStream_t stream) {
  return fp8 ? launch_typed<true>(a, num_sms, stream) : launch_typed<false>(a, num_sms, stream);
}

}  // namespace ep
