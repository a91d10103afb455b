// Router: logits -> the K chosen experts of every token, their weights, per-expert
// counts and the balance loss; and the gradient of the logits.
//
// With l the logits of a token (E of them), s = softmax(l) or sigmoid(l):
//   choice score c = l + b (softmax; the softmax keeps the order) or s + b (sigmoid);
//   expert groups: a group's score is the sum of its two best c; the best `keep`
//   groups stay, ties to the lowest group;
//   the K best c are chosen in order, ties to the lowest expert; -inf is never chosen;
//   weight = scale * s_k, divided by the sum of s over the chosen when normalising;
//   p = s (softmax) or s / sum s (sigmoid); over a segment of n valid tokens, with
//   cnt_e lanes to expert e and P_e the sum of p_e: loss = sum_e (E cnt_e / (K n)) (P_e / n),
//   and the output is its mean over the segments.
//
// One warp takes a token: lane i holds E/32 of its logits, loaded 16 bytes at a
// time, and keeps the best of its own; a round of the choice is one warp-wide
// maximum of order-preserving integer keys and one minimum of expert numbers, after
// which the lane that lost its best looks for its next. Each lane meets the same
// experts in every token, so the probability sums stay in its registers over all
// the warp's tokens; warps, then CTAs, are summed in a fixed order (the last CTA of a
// segment to arrive adds the others' partial sums), so every result repeats bit for bit.
// Reading the logits once is what the operator cannot do without.
#include <type_traits>

#include "ep_device.cuh"
#include "moe_internal.cuh"

namespace ep {

namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr float kTiny = 1e-30f;  // least divisor of a sum of sigmoids

// one instruction on this architecture
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}

// Unsigned key with the order of the floats: what may be chosen lies strictly between the
// keys of -inf and +inf; a NaN that arithmetic made is above, a negative one below.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

constexpr uint32_t kKeyNegInf = 0x007FFFFFu, kKeyPosInf = 0xFF800000u;

// The sigmoid whose rounding the choice depends on: CUDA's expf, then correctly
// rounded operations, so that equal scores tie.
__device__ __forceinline__ float sigmoid_rn(float x) { return __frcp_rn(__fadd_rn(1.f, expf(-x))); }

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

struct Top2 {
  float a, b;
};
__device__ __forceinline__ Top2 top2_merge(Top2 x, Top2 y) {
  return Top2{fmaxf(x.a, y.a), fmaxf(fminf(x.a, y.a), fmaxf(x.b, y.b))};
}

// A lane's best two keys not yet taken: most lanes give two experts at most, and one that
// gives a third looks for it among what comes after its last.
struct Best {
  uint32_t k1, k2;
  int e1, e2;
};
template <int EPL>
__device__ __forceinline__ Best best_two(const uint32_t (&key)[EPL], int lane, uint32_t below, int after) {
  Best b{0u, 0u, 0x7FFFFFFF, 0x7FFFFFFF};
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = expert_of<EPL>(j, lane);
    const uint32_t k = key[j] < below || (key[j] == below && e > after) ? key[j] : 0u;
    const bool first = k > b.k1, second = k > b.k2;
    b.e2 = first ? b.e1 : second ? e : b.e2;
    b.k2 = first ? b.k1 : second ? k : b.k2;
    b.e1 = first ? e : b.e1;
    b.k1 = first ? k : b.k1;
  }
  return b;
}

// CTAs per SM that the registers are limited for: four (what kRouteCtas counts on) while a
// lane holds 8 experts at most.
template <int EPL, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kRouteThreads, EPL <= 8 ? 4 : EPL <= 16 ? 2 : 1) route_kernel(RouteArgs a) {
  extern __shared__ float s_mem[];
  __shared__ int s_valid[kRouteWarps];
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

  float bias[EPL];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = expert_of<EPL>(j, lane);
    bias[j] = a.bias != nullptr && e < E ? __ldg(a.bias + e) : 0.f;
  }
  float prob[EPL];  // the warp's sums of p
#pragma unroll
  for (int j = 0; j < EPL; ++j) prob[j] = 0.f;
  int valid = 0;
  // group that this lane helps to score: `parts` lanes a group; every group is read from its
  // own place on, so that the lanes' banks differ
  const int per_group = E / g.G;
  int parts = 1;
  while (parts * 2 * g.G <= 32) parts *= 2;
  const int grp = lane / parts, part = lane - grp * parts;
  const int place = (part + grp * parts) % per_group;

  const int step = g.C * kRouteWarps;
  const int64_t first = static_cast<int64_t>(seg) * g.T;
  float next[EPL];
  int t = cta * kRouteWarps + warp;
  uint8_t next_on = 1;
  if (t < g.T) {
    load_row<EPL, kBf16, kVec>(a.logits, first + t, E, lane, next);
    if (a.mask != nullptr) next_on = __ldg(a.mask + first + t);
  }
  for (; t < g.T; t += step) {
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = next[j];
    const bool on = next_on != 0;
    const int64_t token = first + t;
    if (t + step < g.T) {
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
    bad |= clean<EPL>(l);
    // scores, the choice's keys, and the probabilities' sum
    uint32_t key[EPL];
    float total = 0.f, top = 0.f, inv;
    {
      float s[EPL];
      if (g.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          s[j] = sigmoid_rn(l[j]);
          total += s[j];
          key[j] = order_key(l[j] > -kInf ? __fadd_rn(s[j], bias[j]) : -kInf);
        }
      } else {
        float m = -kInf;
#pragma unroll
        for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);
        top = warp_max(m);
        if (top == -kInf) top = 0.f;  // no expert is available: every p is 0
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          s[j] = __expf(l[j] - top);
          total += s[j];
          key[j] = order_key(__fadd_rn(l[j], bias[j]));  // -0 + 0 is +0, so the two zeros tie
        }
      }
      total = warp_sum(total);
      inv = total > 0.f ? __frcp_rn(total) : 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) prob[j] = fmaf(s[j], inv, prob[j]);
    }

    if (g.G > 1) {  // keep the groups whose two best experts score highest
      __syncwarp();
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = expert_of<EPL>(j, lane);
        const uint32_t u = key[j] & 0x80000000u ? key[j] ^ 0x80000000u : ~key[j];
        if (e < E) s_row[e] = key[j] > kKeyNegInf && key[j] < kKeyPosInf ? __uint_as_float(u) : -kInf;
      }
      __syncwarp();
      Top2 best{-kInf, -kInf};
      if (grp < g.G) {
        const float* row = s_row + grp * per_group;
        int i = place;
        for (int n = part; n < per_group; n += parts) {
          best = top2_merge(best, Top2{row[i], -kInf});
          i += parts;
          if (i >= per_group) i -= per_group;
        }
      }
      for (int o = 1; o < parts; o <<= 1) {
        const Top2 other{__shfl_xor_sync(kFullMask, best.a, o), __shfl_xor_sync(kFullMask, best.b, o)};
        best = top2_merge(best, other);
      }
      uint32_t gk = grp < g.G && part == 0 ? order_key(__fadd_rn(best.a, best.b)) : 0u;
      uint32_t kept = 0;
      for (int r = 0; r < g.keep; ++r) {
        const uint32_t m = __reduce_max_sync(kFullMask, gk);
        const int src = __ffs(__ballot_sync(kFullMask, gk == m)) - 1;
        kept |= 1u << (src / parts);
        if (lane == src) gk = 0u;
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = expert_of<EPL>(j, lane);
        if (e < E && !(kept >> (e / per_group) & 1u)) key[j] = 0u;
      }
    }

    // K rounds: the warp's best key, its lowest expert; that lane goes on to its next best
    Best b = best_two<EPL>(key, lane, 0xFFFFFFFFu, -1);
    if (__any_sync(kFullMask, b.k1 >= kKeyPosInf)) {  // a choice score that is NaN or +inf: not chosen
      bad = true;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (key[j] >= kKeyPosInf) key[j] = 0u;
      b = best_two<EPL>(key, lane, 0xFFFFFFFFu, -1);
    }
    int mine = -1;
    for (int r = 0; r < K; ++r) {
      const uint32_t m = __reduce_max_sync(kFullMask, b.k1);
      if (m <= kKeyNegInf) break;  // fewer than K experts are available: the other lanes stay -1
      const int e = static_cast<int>(__reduce_min_sync(kFullMask, b.k1 == m ? static_cast<uint32_t>(b.e1) : 0xFFFFFFFFu));
      if (lane == r) mine = e;
      const bool gave = b.k1 == m && b.e1 == e;
      if (gave) {
        b.k1 = b.k2;
        b.e1 = b.e2;
        b.k2 = 0u;
        b.e2 = 0x7FFFFFFF;
      }
      if (EPL > 2 && gave && b.k1 == 0u) b = best_two<EPL>(key, lane, m, e);
    }
    // weights of the chosen: their logits are read again (they are in L1)
    float w = 0.f, lv = -kInf;
    if (mine >= 0)
      lv = kBf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + token * E + mine)) << 16)
                 : __ldg(static_cast<const float*>(a.logits) + token * E + mine);
    if (g.sigmoid) {
      w = mine >= 0 ? sigmoid_rn(lv) : 0.f;
      if (g.normalize) w = __fdividef(w, fmaxf(warp_sum(w), kTiny));
    } else if (g.normalize) {
      const float m = warp_max(lv);
      w = mine >= 0 ? __expf(lv - m) : 0.f;
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    } else {
      w = mine >= 0 ? __expf(lv - top) * inv : 0.f;
    }
    if (lane < K) {
      a.idx[token * K + lane] = mine;
      a.weights[token * K + lane] = w * g.scale;
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
  if (g.C > 1) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) p += s_rows[static_cast<size_t>(w) * E + e];
      a.cta_prob[static_cast<size_t>(blockIdx.x) * E + e] = p;
      a.cta_count[static_cast<size_t>(blockIdx.x) * E + e] = s_count[e];
    }
    if (threadIdx.x == 0) a.cta_valid[blockIdx.x] = n;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(a.seg_done + seg, 1u) == static_cast<uint32_t>(g.C) - 1u;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the segment's last CTA adds the partial sums in CTA order
    const size_t base = static_cast<size_t>(seg) * g.C;
    n = 0;
#pragma unroll 4
    for (int c = 0; c < g.C; ++c) n += __ldcg(a.cta_valid + base + c);
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float p = 0.f;
      int cnt = 0;
#pragma unroll 16
      for (int c = 0; c < g.C; ++c) {
        p += __ldcg(a.cta_prob + (base + c) * E + e);
        cnt += __ldcg(a.cta_count + (base + c) * E + e);
      }
      a.prob_sum[static_cast<size_t>(seg) * E + e] = p;
      a.count[static_cast<size_t>(seg) * E + e] = cnt;
      dot = fmaf(p, static_cast<float>(cnt), dot);
    }
  } else {  // the segment's only CTA
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) p += s_rows[static_cast<size_t>(w) * E + e];
      const int cnt = s_count[e];
      a.prob_sum[static_cast<size_t>(seg) * E + e] = p;
      a.count[static_cast<size_t>(seg) * E + e] = cnt;
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
    if (g.C > 1) a.seg_done[seg] = 0u;
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
      for (int b = 0; b < g.B; ++b) loss += __ldcg(a.seg_loss + b);
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
__global__ void __launch_bounds__(kRouteThreads) route_grad_kernel(RouteGradArgs a) {
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
  const int step = g.C * kRouteWarps;
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
  int t = cta * kRouteWarps + warp;
  if (t < g.T) fetch(first + t);
  bool bad = false;
  for (; t < g.T; t += step) {
    const int64_t token = first + t;
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = next[j];
    const int64_t e64 = next_e;
    const float gw = next_g * g.scale;
    const bool on = next_on != 0;
    if (t + step < g.T) fetch(token + step);
    clean<EPL>(l);
    const bool chosen = on && e64 >= 0 && e64 < E;
    bad |= e64 < -1 || e64 >= E;
    const int e = chosen ? static_cast<int>(e64) : 0;

    float lv = -kInf;
    if (chosen)
      lv = kBf16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + token * E + e)) << 16)
                 : __ldg(static_cast<const float*>(a.logits) + token * E + e);
    if (!(lv < kInf)) lv = -kInf;
    float s[EPL];
    float total = 0.f, top = 0.f;
    if (g.sigmoid) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        s[j] = __fdividef(1.f, 1.f + __expf(-l[j]));
        total += s[j];
      }
    } else {
      float m = -kInf;
#pragma unroll
      for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);
      top = warp_max(m);
      if (top == -kInf) top = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        s[j] = __expf(l[j] - top);
        total += s[j];
      }
    }
    total = warp_sum(total);
    const float inv = total > 0.f ? __frcp_rn(total) : 0.f;
    float ap = 0.f;  // sum of a p
#pragma unroll
    for (int j = 0; j < EPL; ++j) ap = fmaf(coef[j], s[j] * inv, ap);
    ap = warp_sum(ap);
    // what goes to the chosen experts
    float gl, rest = 0.f;
    if (g.sigmoid) {
      const float sv = chosen ? __fdividef(1.f, 1.f + __expf(-lv)) : 0.f;
      if (g.normalize) {
        const float q = __fdividef(sv, fmaxf(warp_sum(sv), kTiny));
        gl = q * (gw - warp_sum(q * gw)) * (1.f - sv);
      } else {
        gl = gw * sv * (1.f - sv);
      }
    } else if (g.normalize) {
      const float m = warp_max(lv);
      float q = chosen && lv > -kInf ? __expf(lv - m) : 0.f;
      const float sum = warp_sum(q);
      q = sum > 0.f ? q / sum : 0.f;
      gl = q * (gw - warp_sum(q * gw));
    } else {
      gl = chosen ? gw * __expf(lv - top) * inv : 0.f;
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
        const float p = s[j + i] * inv;
        float v = p * (coef[j + i] - ap - rest);
        if (g.sigmoid) v *= 1.f - s[j + i];
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
  const size_t smem = sizeof(float) * static_cast<size_t>(a.g.E) * (1 + kRouteWarps);
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

// Registers per lane: the least of 1, 2, 4, 8, 16, 32, 128 that holds E (128 spills; it
// serves more than 1024 experts only). Rows of a multiple of 4 logits load 4 at a time.
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
