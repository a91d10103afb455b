// Router: logits -> the K chosen experts of every token, their weights, per-expert
// counts and the balance loss; and the gradient of the logits.
//
// With l the logits of a token (E of them), s = softmax(l) or sigmoid(l):
//   choice score c = l + b (softmax: single experts rank by l as they do by s; sums of two and
//   sums with a bias are those of logits) or s + b (sigmoid);
//   expert groups: a group's score is the sum of its two best c; the best `keep`
//   groups stay, ties to the lowest group;
//   the K best c are chosen in order, ties to the lowest expert; -inf is never chosen;
//   weight = scale * s_k, divided by the sum of s over the chosen when normalising;
//   p = s (softmax) or s / sum s (sigmoid); over a segment of n valid tokens, with
//   cnt_e lanes to expert e and P_e the sum of p_e: loss = sum_e (E cnt_e / (K n)) (P_e / n),
//   and the output is its mean over the segments.
//
// One warp takes a token: lane i holds E/32 of its logits, loaded 16 bytes at a time. Each
// lane meets the same experts in every token, so the probability sums stay in its
// registers over all the warp's tokens; a CTA's warps are summed in their order, the CTAs
// in fixed point, so every result repeats bit for bit.
// Reading the logits once is what the operator cannot do without; what bounds it is the
// instructions on them, about 560 a token at 256 experts, top 8, half of them the choice
// (comparisons run at half rate). Measured: 16 x 4096 tokens, 256 experts, top 8, softmax
// 48 us (67 MB of logits, 1.4 TB/s; 88 us with sigmoid scores and 8 groups, 92 with a bias), one
// segment of 65536 tokens 43 us; 64 tokens 7 us, of which 3.5 are the statistics' chain of one atomic
// and one load across the CTAs; the gradient of 16 x 4096 tokens
// 30 us, with sigmoid scores 32 (141 MB, 4.4 TB/s).
#include <type_traits>

#include "ep_device.cuh"
#include "moe_internal.cuh"

namespace ep {

namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.402823466e38f;
// A sum of sigmoids below this: every one of them is e^l to 2^-60, and quotients are taken of
// e^(l - largest l) instead, which does not leave the floats' range.
constexpr float kSmallSum = 0x1p-60f;
// Below this logit e^l is 0 even in 64 bits, and so is the score: tokens that have no other
// (the type's lowest value, say) have weights and probabilities of 0.
constexpr float kLeastLogit = -745.f;

// one instruction on this architecture
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}
// e^x and 1/x by the hardware's approximations (2 ulp, and 2^-22 of x for e^x); results below
// 2^-126 are zero
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}

// The sigmoid whose rounding the choice depends on: CUDA's expf, then correctly
// rounded operations, so that equal scores tie.
__device__ __forceinline__ float sigmoid_rn(float x) { return __frcp_rn(__fadd_rn(1.f, expf(-x))); }

// The sigmoid s and 1 - s, each from the smaller of e^x and e^-x, so that neither loses digits at
// its small end.
struct Sigmoids {
  float s, c;
};
__device__ __forceinline__ Sigmoids sigmoids_fast(float x) {
  const float t = exp_fast(-fabsf(x)), r = rcp_fast(1.f + t), q = t * r;
  return x >= 0.f ? Sigmoids{r, q} : Sigmoids{q, r};
}

// Expert of register j of a lane: 4 (or EPL, if less) consecutive experts per lane
// and step, so that a lane reads 16 bytes of fp32 at once.
template <int EPL>
__device__ __forceinline__ int expert_of(int j, int lane) {
  constexpr int V = EPL < 4 ? EPL : 4;
  return (j / V) * (32 * V) + lane * V + j % V;
}

// A token's logits; places past E are -inf.
template <int EPL, bool kBf16, bool kVec>
__device__ __forceinline__ void load_row(const void* base, int64_t token, int E, int lane, float (&l)[EPL]) {
  constexpr int V = EPL < 4 ? EPL : 4;
  if constexpr (kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + token * E;
#pragma unroll
    for (int j = 0; j < EPL; j += V) {
      const int e = expert_of<EPL>(j, lane);
      if constexpr (kVec && V == 4) {
        uint2 v = make_uint2(0xFF80FF80u, 0xFF80FF80u);  // -inf
        if (e < E) v = __ldg(reinterpret_cast<const uint2*>(p + e));
        const float2 a = bf16x2_to_f32x2(v.x), b = bf16x2_to_f32x2(v.y);
        l[j] = a.x, l[j + 1] = a.y, l[j + 2] = b.x, l[j + 3] = b.y;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          l[j + i] = e + i < E ? __uint_as_float(static_cast<uint32_t>(__ldg(p + e + i)) << 16) : -kInf;
      }
    }
  } else {
    const float* p = static_cast<const float*>(base) + token * E;
#pragma unroll
    for (int j = 0; j < EPL; j += V) {
      const int e = expert_of<EPL>(j, lane);
      if constexpr (kVec && V == 4) {
        float4 v = make_float4(-kInf, -kInf, -kInf, -kInf);
        if (e < E) v = __ldg(reinterpret_cast<const float4*>(p + e));
        l[j] = v.x, l[j + 1] = v.y, l[j + 2] = v.z, l[j + 3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[j + i] = e + i < E ? __ldg(p + e + i) : -kInf;
      }
    }
  }
}

// NaN and +inf count as -inf; returns whether the warp met one.
template <int EPL>
__device__ __forceinline__ bool clean(float (&l)[EPL]) {
  bool ok = true;
#pragma unroll
  for (int j = 0; j < EPL; ++j) ok = ok && l[j] < kInf;
  if (__all_sync(kFullMask, ok)) return false;
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (!(l[j] < kInf)) l[j] = -kInf;
  return true;
}

// A token's logits, all of them far below zero, become its scores up to a common factor; returns
// the lane's sum.
template <int EPL>
__device__ __forceinline__ float small_scores(float (&s)[EPL]) {
  float most = -kInf, total = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) most = fmaxf(most, s[j]);
  most = warp_max(most);
  if (most < kLeastLogit) most = 0.f;  // every score is 0
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    s[j] = exp_fast(s[j] - most);
    total += s[j];
  }
  return total;
}

struct Top2 {
  float a, b;
};
__device__ __forceinline__ Top2 top2_merge(Top2 x, Top2 y) {
  return Top2{fmaxf(x.a, y.a), fmaxf(fminf(x.a, y.a), fmaxf(x.b, y.b))};
}

// What a warp lists the candidates of a token in.
struct Candidates {
  float4 score[8];  // 32 scores
  int expert[32];
};

// The K best scores, best first, ties to the lowest expert: the lane that returns r >= 0 has
// the expert of place r in `mine` and its score in `mine_score`. `best` is the lane's largest
// score; -inf and NaN are never chosen, +inf does not occur.
//
// The K-th largest of the lanes' best scores bounds the K-th largest of all from below, so only
// scores that reach it can be chosen: K at least, and few more. They are listed in shared
// memory, a lane takes one, and its place is the number of larger ones (equal scores,
// which show as a place taken twice, are told apart by expert). More than 32 (many
// equal scores, or K near 32) take K rounds of finding the best instead (such rounds for
// every token: 68 us for 16 x 4096 tokens, 256 experts, top 8; with the list 52, and 45
// after its bound came from integer maxima).
template <int EPL>
__device__ __forceinline__ int choose(float (&c)[EPL], float best, int K, Candidates& list, int lane, int& mine,
                                      float& mine_score) {
  mine = -1;
  mine_score = 0.f;
  // by integer keys of the same order: their warp-wide maximum takes two thirds of the floats' time
  const uint32_t u = __float_as_uint(best);
  uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  for (int r = 1; r < K; ++r)
    if (key == __reduce_max_sync(kFullMask, key)) key = 0u;  // lanes that tie go together: the bound stays one
  key = __reduce_max_sync(kFullMask, key);
  const float bound = key <= 0x007FFFFFu ? kLowest : __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
  int count = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) count += c[j] >= bound;
  int at = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullMask, at, o);
    if (lane >= o) at += v;
  }
  const int n = __shfl_sync(kFullMask, at, 31);
  if (n <= 32) {
    at -= count;
    float* scores = reinterpret_cast<float*>(list.score);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (c[j] >= bound) {
        scores[at] = c[j];
        list.expert[at] = expert_of<EPL>(j, lane);
        ++at;
      }
    if (lane >= n) scores[lane] = -kInf;
    __syncwarp();
    mine_score = scores[lane];
    mine = list.expert[lane];
    int place = 0;
    for (int i = 0; 4 * i < n; ++i) {
      const float4 v = list.score[i];
      place += (v.x > mine_score) + (v.y > mine_score) + (v.z > mine_score) + (v.w > mine_score);
    }
    const unsigned seen = __reduce_or_sync(kFullMask, lane < n ? 1u << place : 0u);
    if (__popc(seen) != n)
      for (int i = 0; i < n; ++i) place += scores[i] == mine_score && list.expert[i] < mine;
    __syncwarp();
    return lane < n && place < K ? place : -1;
  }
  int place = -1;
  for (int r = 0; r < K; ++r) {
    float bc = -kInf;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (c[j] > bc) {
        bc = c[j];
        be = expert_of<EPL>(j, lane);
      }
    const float m = warp_max(bc);
    if (m == -kInf) break;  // fewer than K experts are available
    const int e = static_cast<int>(__reduce_min_sync(kFullMask, bc == m ? static_cast<uint32_t>(be) : 0xFFFFFFFFu));
    if (lane == r) {
      mine = e;
      mine_score = m;
      place = r;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (expert_of<EPL>(j, lane) == e) c[j] = -kInf;
  }
  return place;
}

// CTAs per SM that the registers are limited for: four (what kRouteCtas counts on) while a
// lane holds 8 experts at most.
template <int EPL, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kRouteThreads, EPL <= 8 ? 4 : EPL <= 16 ? 2 : 1) route_kernel(RouteArgs a) {
  extern __shared__ float s_mem[];
  __shared__ int s_valid[kRouteWarps];
  __shared__ Candidates s_list[kRouteWarps];
  __shared__ float s_part[kRouteWarps];
  __shared__ bool s_last;
  const RouteGeometry& g = a.g;
  const int E = g.E, K = g.K;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x / g.C, cta = blockIdx.x - seg * g.C;
  int* s_count = reinterpret_cast<int*>(s_mem);         // [E]
  float* s_rows = s_mem + E;                            // [kRouteWarps][E]
  float* s_row = s_rows + static_cast<size_t>(warp) * E;  // this warp's
  const bool stats = a.count != nullptr;
  for (int e = threadIdx.x; e < E; e += kRouteThreads) s_count[e] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  // the choice bias in shared memory; one that is NaN or +inf disables its expert
  bool bad = false;
  float* s_bias = s_rows + static_cast<size_t>(kRouteWarps) * E;  // [E], with a bias
  if (a.bias != nullptr) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float b = __ldg(a.bias + e);
      if (!(b < kInf)) {
        b = -kInf;
        bad = true;
      }
      s_bias[e] = b;
    }
    __syncthreads();
  }
  float prob[EPL];  // the warp's sums of p
#pragma unroll
  for (int j = 0; j < EPL; ++j) prob[j] = 0.f;
  int valid = 0;
  // Groups of a multiple of 4 experts are scored from the two best of every lane's 4
  // neighbours, others from the experts one by one: `cells` of a group, `parts` lanes a group;
  // every group is read from a place of its own on, so that the lanes' banks differ.
  constexpr bool kQuads = EPL >= 4;
  const int per_group = E / g.G;
  const bool quads = kQuads && per_group % 4 == 0;
  const int cells = quads ? per_group / 4 : per_group;
  int parts = 1;
  while (parts * 2 * g.G <= 32) parts *= 2;
  const int grp = lane / parts, part = lane - grp * parts;
  const int place = (part + grp * parts) % cells;
  const uint32_t group_magic = 0xFFFFFFFFu / static_cast<uint32_t>(per_group) + 1u;  // e / per_group, e < 2^16, by a high product

  // unsigned: T is below 2^31, so t + step does not wrap
  const uint32_t T = static_cast<uint32_t>(g.T), step = static_cast<uint32_t>(g.C * kRouteWarps);
  const int64_t first = static_cast<int64_t>(seg) * g.T;
  // the next token's logits load while this one is worked on
  float next[EPL];
  uint32_t t = static_cast<uint32_t>(cta * kRouteWarps + warp);
  uint8_t next_on = 1;
  if (t < T) {
    load_row<EPL, kBf16, kVec>(a.logits, first + t, E, lane, next);
    if (a.mask != nullptr) next_on = __ldg(a.mask + first + t);
  }
  for (; t < T; t += step) {
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = next[j];
    const bool on = next_on != 0;
    const int64_t token = first + t;
    if (t + step < T) {
      load_row<EPL, kBf16, kVec>(a.logits, token + step, E, lane, next);
      if (a.mask != nullptr) next_on = __ldg(a.mask + token + step);
    }
    if (!on) {  // a padding token: no expert, no weight, not counted
      if (lane < K) {
        a.idx[token * K + lane] = -1;
        a.weights[token * K + lane] = 0.f;
      }
      continue;
    }
    ++valid;
    // choice scores (in place of the logits when these are the scores), probabilities' sum
    float total = 0.f, top = 0.f, inv, best = -kInf;
    {
      float s[EPL];
      if (g.sigmoid) {
        bad |= clean<EPL>(l);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          s[j] = sigmoid_rn(l[j]);
          total += s[j];
          l[j] = l[j] > -kInf ? s[j] : -kInf;
          best = fmaxf(best, l[j]);
        }
        total = warp_sum(total);
        if (total < kSmallSum) {
          load_row<EPL, kBf16, kVec>(a.logits, token, E, lane, s);
          clean<EPL>(s);
          total = warp_sum(small_scores<EPL>(s));
        }
      } else {
        auto probabilities = [&] {
          best = -kInf;
#pragma unroll
          for (int j = 0; j < EPL; ++j) best = fmaxf(best, l[j]);
          top = warp_max(best);
          if (top == -kInf) top = 0.f;  // no expert is available: every p is 0
          total = 0.f;
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            s[j] = exp_fast(l[j] - top);
            total += s[j];
          }
          total = warp_sum(total);
        };
        probabilities();
        if (!(total < kInf)) {  // a NaN or +inf among the logits makes the sum NaN
          bad |= clean<EPL>(l);
          probabilities();
        }
      }
      inv = total > 0.f ? rcp_fast(total) : 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) prob[j] = fmaf(s[j], inv, prob[j]);
    }
    if (a.bias != nullptr) {
      best = -kInf;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = expert_of<EPL>(j, lane);
        if (e < E) l[j] = __fadd_rn(l[j], s_bias[e]);
        best = fmaxf(best, l[j]);
      }
      if (__any_sync(kFullMask, best == kInf)) {  // a sum past the largest float: not chosen
        bad = true;
        best = -kInf;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          if (l[j] == kInf) l[j] = -kInf;
          best = fmaxf(best, l[j]);
        }
      }
    }

    if (g.G > 1) {  // keep the groups whose two best experts score highest
      Top2 two{-kInf, -kInf};
      __syncwarp();
      if (quads) {
        if constexpr (kQuads) {
#pragma unroll
          for (int j = 0; j < EPL; j += 4) {
            const int e = expert_of<EPL>(j, lane);
            const Top2 q = top2_merge(top2_merge(Top2{l[j], -kInf}, Top2{l[j + 1], -kInf}),
                                      top2_merge(Top2{l[j + 2], -kInf}, Top2{l[j + 3], -kInf}));
            if (e < E) *reinterpret_cast<float2*>(s_row + e / 2) = make_float2(q.a, q.b);
          }
          __syncwarp();
          if (grp < g.G) {
            const float2* row = reinterpret_cast<const float2*>(s_row) + grp * cells;
            int i = place;
            for (int n = part; n < cells; n += parts) {
              const float2 q = row[i];
              two = top2_merge(two, Top2{q.x, q.y});
              i += parts;
              if (i >= cells) i -= cells;
            }
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int e = expert_of<EPL>(j, lane);
          if (e < E) s_row[e] = l[j];
        }
        __syncwarp();
        if (grp < g.G) {
          const float* row = s_row + grp * cells;
          int i = place;
          for (int n = part; n < cells; n += parts) {
            two = top2_merge(two, Top2{row[i], -kInf});
            i += parts;
            if (i >= cells) i -= cells;
          }
        }
      }
      for (int o = 1; o < parts; o <<= 1) {
        const Top2 other{__shfl_xor_sync(kFullMask, two.a, o), __shfl_xor_sync(kFullMask, two.b, o)};
        two = top2_merge(two, other);
      }
      // a group without two available experts goes after the others, but before what is -inf
      // here: groups already taken, and lanes that hold none
      float score = grp < g.G && part == 0 ? fmaxf(__fadd_rn(two.a, two.b), kLowest) : -kInf;
      uint32_t kept = 0;
      for (int r = 0; r < g.keep; ++r) {
        const int src = __ffs(__ballot_sync(kFullMask, score == warp_max(score))) - 1;
        kept |= 1u << (src / parts);
        if (lane == src) score = -kInf;
      }
      best = -kInf;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = expert_of<EPL>(kQuads && quads ? j / 4 * 4 : j, lane);
        if (!(kept >> (__umulhi(static_cast<uint32_t>(e), group_magic) & 31u) & 1u)) l[j] = -kInf;
        best = fmaxf(best, l[j]);
      }
    }
    int mine;
    float mine_score;
    const int place_of = choose<EPL>(l, best, K, s_list[warp], lane, mine, mine_score);
    if (place_of < 0) mine = -1;
    // weights of the chosen: the score is the logit, or the logit is read again (it is in L1)
    float w = 0.f, lv = -kInf;
    if (mine >= 0) {
      if (!g.sigmoid && a.bias == nullptr)
        lv = mine_score;
      else
        lv = kBf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + token * E + mine)) << 16)
                   : __ldg(static_cast<const float*>(a.logits) + token * E + mine);
    }
    if (g.sigmoid) {
      w = mine >= 0 ? sigmoid_rn(lv) : 0.f;
      if (g.normalize) {
        float sum = warp_sum(w);
        if (sum < kSmallSum) {
          const float m = warp_max(lv);
          w = mine >= 0 && m >= kLeastLogit ? exp_fast(lv - m) : 0.f;
          sum = warp_sum(w);
        }
        w = sum > 0.f ? __fdividef(w, sum) : 0.f;
      }
    } else if (g.normalize) {
      const float m = warp_max(lv);
      w = mine >= 0 ? exp_fast(lv - m) : 0.f;
      const float sum = warp_sum(w);
      w = sum > 0.f ? __fdividef(w, sum) : 0.f;
    } else {
      w = mine >= 0 ? exp_fast(lv - top) * inv : 0.f;
    }
    // places that no expert took are -1
    const int taken = __popc(__ballot_sync(kFullMask, place_of >= 0));
    if (place_of >= 0) {
      a.idx[token * K + place_of] = mine;
      a.weights[token * K + place_of] = w * g.scale;
    }
    if (lane >= taken && lane < K) {
      a.idx[token * K + lane] = -1;
      a.weights[token * K + lane] = 0.f;
    }
    if (stats && mine >= 0) atomicAdd(s_count + mine, 1);
  }
  if (bad) atomicOr(a.err, kErrNonfinite);
  if (!stats) return;

  // the CTA's sums, in the order of the warps
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = expert_of<EPL>(j, lane);
    if (e < E) s_row[e] = prob[j];
  }
  if (lane == 0) s_valid[warp] = valid;
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < kRouteWarps; ++w) n += s_valid[w];
  float dot = 0.f;
  const size_t row = static_cast<size_t>(seg) * E;
  if (g.C > 1) {
    // The CTAs of a segment are summed in 64-bit fixed point, in which the order of the
    // additions does not matter: a CTA's fp32 sum is rounded to 2^-prob_shift (2^-49 for a
    // segment of 4096 tokens). Partial sums of all CTAs, added by the last one, took 40 us
    // with one segment of 65536 tokens.
    const float unit = __int_as_float((127 + g.prob_shift) << 23);
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) p += s_rows[static_cast<size_t>(w) * E + e];
      atomicAdd(a.ws_prob + row + e, __float2ull_rn(p * unit));
      if (s_count[e] != 0) atomicAdd(a.ws_count + row + e, static_cast<uint32_t>(s_count[e]));
    }
    if (threadIdx.x == 0) atomicAdd(a.seg_valid + seg, static_cast<uint32_t>(n));
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(a.seg_done + seg, 1u) == static_cast<uint32_t>(g.C) - 1u;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    n = static_cast<int>(__ldcg(a.seg_valid + seg));
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      const float p = __ull2float_rn(__ldcg(a.ws_prob + row + e)) / unit;
      const int cnt = static_cast<int>(__ldcg(a.ws_count + row + e));
      a.ws_prob[row + e] = 0ull;
      a.ws_count[row + e] = 0u;
      a.prob_sum[row + e] = p;
      a.count[row + e] = cnt;
      dot = fmaf(p, static_cast<float>(cnt), dot);
    }
  } else {  // the segment's only CTA
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) p += s_rows[static_cast<size_t>(w) * E + e];
      const int cnt = s_count[e];
      a.prob_sum[row + e] = p;
      a.count[row + e] = cnt;
      dot = fmaf(p, static_cast<float>(cnt), dot);
    }
  }
  dot = warp_sum(dot);
  if (lane == 0) s_part[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
    for (int w = 0; w < kRouteWarps; ++w) sum += s_part[w];
    const float nf = static_cast<float>(n > 0 ? n : 1);
    const float seg_loss = sum * (static_cast<float>(E) / static_cast<float>(K)) / nf / nf;
    a.num_valid[seg] = n;
    if (g.C > 1) {
      a.seg_done[seg] = 0u;
      a.seg_valid[seg] = 0u;
    }
    if (g.B == 1) {
      *a.loss = seg_loss;
      return;
    }
    __stcg(a.seg_loss + seg, seg_loss);
    __threadfence();
    if (atomicAdd(a.done, 1u) == static_cast<uint32_t>(g.B) - 1u) {  // the last segment of all
      __threadfence();
      float loss = 0.f;
#pragma unroll 16
      for (int b = 0; b < g.B; ++b) {
        loss += __ldcg(a.seg_loss + b);
        a.seg_loss[b] = 0.f;
      }
      *a.loss = loss / static_cast<float>(g.B);
      *a.done = 0u;
    }
  }
}

// Gradient of the logits. The chosen experts and the counts are constants. With gw the
// weights' gradients and a_e = dL E cnt_e / (B K n^2) the loss's gradient of p_e:
//   softmax  dl = p (a - sum a p) + {chosen} scale q (gw - sum q gw), q = softmax over the chosen
//            (not normalised: dl = p (a - sum a p - scale sum p gw) + {chosen} scale p gw);
//   sigmoid  dl = (1 - s) [p (a - sum a p) + {chosen} scale q (gw - sum q gw)], q = s / sum of the
//            chosen s (not normalised: {chosen} scale s gw).
// A warp takes a token with the forward's lane layout; what goes to the K chosen
// experts reaches their lanes through a row of shared memory that is zero elsewhere.
template <int EPL, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kRouteThreads, EPL <= 8 ? 4 : EPL <= 16 ? 2 : 1) route_grad_kernel(RouteGradArgs a) {
  extern __shared__ float s_mem[];
  const RouteGeometry& g = a.g;
  const int E = g.E, K = g.K;
  constexpr int V = EPL < 4 ? EPL : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x / g.C, cta = blockIdx.x - seg * g.C;
  float* s_row = s_mem + static_cast<size_t>(warp) * E;
  for (int e = lane; e < E; e += 32) s_row[e] = 0.f;
  pdl_launch_dependents();
  pdl_wait();
  __syncwarp();

  float coef[EPL];
  {
    float f = 0.f;
    if (a.d_loss != nullptr) {
      const int n = __ldg(a.num_valid + seg);
      const float nf = static_cast<float>(n > 0 ? n : 1);
      f = __ldg(a.d_loss) * (static_cast<float>(E) / (static_cast<float>(g.B) * static_cast<float>(K))) / nf / nf;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = expert_of<EPL>(j, lane);
      coef[j] = a.d_loss != nullptr && e < E ? f * static_cast<float>(__ldg(a.count + static_cast<size_t>(seg) * E + e)) : 0.f;
    }
  }
  // unsigned: T is below 2^31, so t + step does not wrap
  const uint32_t T = static_cast<uint32_t>(g.T), step = static_cast<uint32_t>(g.C * kRouteWarps);
  const int64_t first = static_cast<int64_t>(seg) * g.T;
  float next[EPL];
  int64_t next_e = -1;
  float next_g = 0.f;
  uint8_t next_on = 1;
  auto fetch = [&](int64_t token) {
    load_row<EPL, kBf16, kVec>(a.logits, token, E, lane, next);
    next_e = -1;
    next_g = 0.f;
    if (lane < K) {
      next_e = __ldg(a.idx + token * K + lane);
      if (a.d_weights != nullptr) next_g = __ldg(a.d_weights + token * K + lane);
    }
    if (a.mask != nullptr) next_on = __ldg(a.mask + token);
  };
  uint32_t t = static_cast<uint32_t>(cta * kRouteWarps + warp);
  if (t < T) fetch(first + t);
  bool bad = false;
  for (; t < T; t += step) {
    const int64_t token = first + t;
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = next[j];
    const int64_t e64 = next_e;
    const float given = next_g;
    const bool on = next_on != 0;
    if (t + step < T) fetch(token + step);
    clean<EPL>(l);
    const bool chosen = on && e64 >= 0 && e64 < E;
    bad |= e64 < -1 || e64 >= E;
    const int e = chosen ? static_cast<int>(e64) : 0;
    const float gw = chosen ? given * g.scale : 0.f;  // what stands at an absent lane may be a NaN

    float lv = -kInf;
    if (chosen)
      lv = kBf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + token * E + e)) << 16)
                 : __ldg(static_cast<const float*>(a.logits) + token * E + e);
    if (!(lv < kInf)) lv = -kInf;
    // softmax: s[j] = e^(l - top), p = s / sum s. Sigmoid: s[j] = e^-l, of which both the score
    // 1 / (1 + s[j]) and one minus it, s[j] / (1 + s[j]), keep all their digits.
    float s[EPL];
    float total = 0.f, ap = 0.f, top = 0.f;  // ap: the sum of a p
    if (g.sigmoid) {
      auto sums = [&](int j) {
        const float v = rcp_fast(1.f + s[j]);
        total += v;
        ap = fmaf(coef[j], v, ap);
      };
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        s[j] = exp_fast(-l[j]);
        sums(j);
      }
      total = warp_sum(total);
      if (total < kSmallSum) {  // the quotients of logits that are shifted up to -42 at the largest
        load_row<EPL, kBf16, kVec>(a.logits, token, E, lane, s);
        clean<EPL>(s);
        float m = -kInf;
#pragma unroll
        for (int j = 0; j < EPL; ++j) m = fmaxf(m, s[j]);
        m = warp_max(m);
        if (m < kLeastLogit) m = kInf;  // every score is 0
        total = ap = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          s[j] = exp_fast(42.f - (s[j] - m));
          sums(j);
        }
        total = warp_sum(total);
      }
    } else {
      float m = -kInf;
#pragma unroll
      for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);
      top = warp_max(m);
      if (top == -kInf) top = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        s[j] = exp_fast(l[j] - top);
        total += s[j];
        ap = fmaf(coef[j], s[j], ap);
      }
      total = warp_sum(total);
    }
    const float inv = total > 0.f ? rcp_fast(total) : 0.f;
    ap = warp_sum(ap) * inv;
    // what goes to the chosen experts
    float gl, rest = 0.f;
    if (g.sigmoid) {
      const Sigmoids v = sigmoids_fast(lv);  // s = 0 where no expert is chosen
      if (g.normalize) {
        float q = v.s, sum = warp_sum(q);
        if (sum < kSmallSum) {
          const float m = warp_max(lv);
          q = lv > -kInf && m >= kLeastLogit ? exp_fast(lv - m) : 0.f;
          sum = warp_sum(q);
        }
        q = sum > 0.f ? __fdividef(q, sum) : 0.f;
        gl = q * (gw - warp_sum(q * gw)) * v.c;
      } else {
        gl = gw * v.s * v.c;
      }
    } else if (g.normalize) {
      const float m = warp_max(lv);
      float q = chosen && lv > -kInf ? exp_fast(lv - m) : 0.f;
      const float sum = warp_sum(q);
      q = sum > 0.f ? __fdividef(q, sum) : 0.f;
      gl = q * (gw - warp_sum(q * gw));
    } else {
      gl = chosen ? gw * exp_fast(lv - top) * inv : 0.f;
      rest = warp_sum(gl);
    }
    if (chosen) s_row[e] = gl;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < EPL; j += V) {
      const int e0 = expert_of<EPL>(j, lane);
      float d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float p = s[j + i] * inv, v = coef[j + i] - ap - rest;
        if (g.sigmoid) {
          const float score = rcp_fast(1.f + s[j + i]);
          p = score * inv;
          v *= fminf(score * s[j + i], 1.f);  // 0 * inf becomes 1
        }
        v *= p;
        if (e0 + i < E) v += s_row[e0 + i];
        d[i] = on ? v : 0.f;
      }
      if constexpr (kBf16) {
        uint16_t* o = static_cast<uint16_t*>(a.d_logits) + token * E + e0;
        if constexpr (kVec && V == 4) {
          if (e0 < E) *reinterpret_cast<uint2*>(o) = make_uint2(f32x2_to_bf16x2(d[0], d[1]), f32x2_to_bf16x2(d[2], d[3]));
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (e0 + i < E) o[i] = static_cast<uint16_t>(f32x2_to_bf16x2(d[i], 0.f) & 0xFFFFu);
        }
      } else {
        float* o = static_cast<float*>(a.d_logits) + token * E + e0;
        if constexpr (kVec && V == 4) {
          if (e0 < E) *reinterpret_cast<float4*>(o) = make_float4(d[0], d[1], d[2], d[3]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (e0 + i < E) o[i] = d[i];
        }
      }
    }
    __syncwarp();
    if (chosen) s_row[e] = 0.f;
    __syncwarp();
  }
  if (bad) atomicOr(a.err, kErrBadTopk);
}

template <int EPL, bool kBf16, bool kVec>
cudaError_t launch_fwd(const RouteArgs& a, cudaStream_t stream) {
  auto kern = route_kernel<EPL, kBf16, kVec>;
  const size_t smem = sizeof(float) * static_cast<size_t>(a.g.E) * (1 + kRouteWarps + (a.bias != nullptr));
  if (resident_ctas(reinterpret_cast<const void*>(kern), kRouteThreads, smem) < 1) return cudaErrorInvalidConfiguration;
  return launch_chained(kern, dim3(static_cast<unsigned>(a.g.B) * a.g.C), dim3(kRouteThreads), smem, stream, a);
}

template <int EPL, bool kBf16, bool kVec>
cudaError_t launch_bwd(const RouteGradArgs& a, cudaStream_t stream) {
  auto kern = route_grad_kernel<EPL, kBf16, kVec>;
  const size_t smem = sizeof(float) * static_cast<size_t>(a.g.E) * kRouteWarps;
  if (resident_ctas(reinterpret_cast<const void*>(kern), kRouteThreads, smem) < 1) return cudaErrorInvalidConfiguration;
  return launch_chained(kern, dim3(static_cast<unsigned>(a.g.B) * a.g.C), dim3(kRouteThreads), smem, stream, a);
}

// Logits per lane: the least of 1, 2, 4, 8, 16, 32, 128 that holds E. 128 serves more than 1024
// experts only and spills 1 to 5 KB a thread; the forward's 8 spills 12 bytes at the 64 registers that
// four CTAs an SM leave. Rows of a multiple of 4 logits load 4 at a time.
template <class Args, class Launch>
cudaError_t by_size(const Args& a, Launch launch) {
  const int E = a.g.E;
  if (E <= 32) return launch(std::integral_constant<int, 1>());
  if (E <= 64) return launch(std::integral_constant<int, 2>());
  if (E <= 128) return launch(std::integral_constant<int, 4>());
  if (E <= 256) return launch(std::integral_constant<int, 8>());
  if (E <= 512) return launch(std::integral_constant<int, 16>());
  if (E <= 1024) return launch(std::integral_constant<int, 32>());
  return launch(std::integral_constant<int, 128>());
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return by_size(a, [&](auto n) {
    constexpr int EPL = decltype(n)::value;
    if (a.g.bf16) return a.g.E % 4 == 0 ? launch_fwd<EPL, true, true>(a, stream) : launch_fwd<EPL, true, false>(a, stream);
    return a.g.E % 4 == 0 ? launch_fwd<EPL, false, true>(a, stream) : launch_fwd<EPL, false, false>(a, stream);
  });
}

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t stream) {
  return by_size(a, [&](auto n) {
    constexpr int EPL = decltype(n)::value;
    if (a.g.bf16) return a.g.E % 4 == 0 ? launch_bwd<EPL, true, true>(a, stream) : launch_bwd<EPL, true, false>(a, stream);
    return a.g.E % 4 == 0 ? launch_bwd<EPL, false, true>(a, stream) : launch_bwd<EPL, false, false>(a, stream);
  });
}

}  // namespace ep
