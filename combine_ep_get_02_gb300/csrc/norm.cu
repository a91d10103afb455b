// Root-mean-square norm with the residual's addition, in bf16 and as FP8 rows with scales, and
// its gradients.
//
//   s = x + residual,  q = 1 / sqrt(mean s^2 + eps),  y = s q w
//   d_s = q (t - n mean(t n)) + d_sum,  d_w = sum over rows of d_y n     with t = d_y w, n = s q
//
// A row stays in its threads' registers between the sum over it and its use, so that each
// input is read once and each output written once: memory bounds both.
#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"
#include "tensor_core.cuh"

namespace ep {

namespace {

// 16 bytes that are read once; the same thread may write them later in the kernel (a sum that takes
// the place of its input), so this is no read-only load
__device__ __forceinline__ uint4 ld_once16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Eight neighbouring values as they lie in memory.
template <bool kFp32>
struct Eight;
template <>
struct Eight<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) { a = ld_once16(static_cast<const uint16_t*>(p) + i); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(a, f); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    st16(static_cast<uint16_t*>(p) + i, pack8(f));
  }
};
template <>
struct Eight<true> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = ld_once16(static_cast<const float*>(p) + i);
    b = ld_once16(static_cast<const float*>(p) + i + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[j]);
    st16(static_cast<float*>(p) + i, make_uint4(w[0], w[1], w[2], w[3]));
    st16(static_cast<float*>(p) + i + 4, make_uint4(w[4], w[5], w[6], w[7]));
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
  return v;
}

// The sum over the row's threads: a warp, or the CTA through `s` (of 32 floats; calls take
// turns between two of them, so that one barrier a sum is enough). Every thread gets the same.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* s) {
  v = warp_sum(v);
  if constexpr (kWarpRow) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? s[lane] : 0.f);
}

// Sums of squares past fp32's range: the values are taken 2^-80 as large, which holds the square of
// the largest of them, and what is below that does not count beside them.
constexpr float kShrink = 8.271806125530277e-25f;  // 2^-80

// 1 / sqrt(mean s^2 + eps) of the sum of squares so taken; eps counts where it is as large as they are
__device__ __forceinline__ float root_of_small(float small, int H, float eps) {
  return __frsqrt_rn(small / H + eps * kShrink * kShrink) * kShrink;
}

// Threads of a CTA at most: as many as the registers of kV chunks each leave room for.
template <int kV, bool kWarpRow, bool kGrad>
constexpr int threads_of = kWarpRow ? 128 : kV == 1 && !kGrad ? 1024 : 512;

// kV: chunks of 8 columns a thread holds; kWarpRow: a warp takes a row of its own.
template <bool kFp32, int kV, bool kWarpRow>
__global__ void __launch_bounds__(threads_of<kV, kWarpRow, false>) norm_kernel(NormArgs a) {
  __shared__ float s_sum[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int across = kWarpRow ? 32 : blockDim.x, at = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int chunks = a.H >> 3, G = a.H >> 7;
  const int64_t first = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarpRow ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    const int64_t base = row * a.H;
    Eight<kFp32> vx[kV], vr[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = v * across + at;
      vx[v].zero();
      vr[v].zero();
      if (c < chunks) {
        vx[v].load(a.x, base + c * 8);
        if (a.residual != nullptr) vr[v].load(a.residual, base + c * 8);
      }
    }
    float f[kV][8], ss = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      float r[8];
      vx[v].get(f[v]);
      vr[v].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.residual != nullptr) f[v][i] += r[i];  // -0 stays -0 without one
        ss = fmaf(f[v][i], f[v][i], ss);
      }
    }
    ss = row_sum<kWarpRow>(ss, s_sum[turn]);
    turn ^= 1;
    float q = __frsqrt_rn(ss / a.H + a.eps);
    if (ss == INFINITY) {
      float small = 0.f;
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) small = fmaf(f[v][i] * kShrink, f[v][i] * kShrink, small);
      small = row_sum<kWarpRow>(small, s_sum[turn]);
      turn ^= 1;
      q = root_of_small(small, a.H, a.eps);
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = v * across + at;
      const int64_t i0 = base + c * 8;
      const bool in = c < chunks;
      if (in && a.sum != nullptr) Eight<kFp32>::store(a.sum, i0, f[v]);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = f[v][i] * q;
      if (in && a.weight != nullptr) {
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.weight + c * 8)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= w[i];
      }
      if (in && a.y != nullptr) st16(a.y + i0, pack8(y));
      if (a.codes != nullptr) {  // 16 neighbouring threads hold the 128 columns of a scale
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
        const RowScale s = row_scale(amax, a.sf_pack);
        if (in) {
          uint32_t q4[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            q4[h] = f32x2_to_e4m3x2(__fmul_rn(y[4 * h], s.inv), __fmul_rn(y[4 * h + 1], s.inv)) |
                    f32x2_to_e4m3x2(__fmul_rn(y[4 * h + 2], s.inv), __fmul_rn(y[4 * h + 3], s.inv)) << 16;
          *reinterpret_cast<uint2*>(a.codes + i0) = make_uint2(q4[0], q4[1]);
          if ((c & 15) == 0) store_scale(a.sf, row, c >> 4, G, s, a.sf_pack);
        }
      }
    }
  }
}

// A CTA adds up d_weight over its rows (those of its index, then every gridDim-th) in registers and leaves the
// sums in the workspace, for norm_weight_kernel to add in the CTAs' order: no atomics, so that
// the order and with it the result is always the same.
template <bool kFp32, int kV, bool kWarpRow>
__global__ void __launch_bounds__(threads_of<kV, kWarpRow, true>) norm_grad_kernel(NormGradArgs a) {
  __shared__ float s_sum[4][32];
  pdl_launch_dependents();
  pdl_wait();
  const int across = kWarpRow ? 32 : blockDim.x, at = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int chunks = a.H >> 3;
  const int64_t first = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarpRow ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
  uint4 w[kV];
  float dw[kV][8];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * across + at;
    w[v] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (c < chunks && a.weight != nullptr) w[v] = __ldg(reinterpret_cast<const uint4*>(a.weight + c * 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    const int64_t base = row * a.H;
    if (a.mask != nullptr && __ldg(a.mask + row) == 0) {  // the same for all of the row's threads
      if (a.d_x != nullptr) {
        const float none[8] = {};
#pragma unroll
        for (int v = 0; v < kV; ++v)
          if (const int c = v * across + at; c < chunks) Eight<kFp32>::store(a.d_x, base + c * 8, none);
      }
      continue;
    }
    Eight<kFp32> vs[kV], vd[kV];
    uint4 vy[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = v * across + at;
      vs[v].zero();
      vd[v].zero();
      vy[v] = make_uint4(0u, 0u, 0u, 0u);
      if (c < chunks) {
        vs[v].load(a.sum, base + c * 8);
        vy[v] = ld_once16(a.d_y + base + c * 8);
        if (a.d_sum != nullptr && a.d_x != nullptr) vd[v].load(a.d_sum, base + c * 8);
      }
    }
    float ss = 0.f, ts = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      float s[8], y[8], g[8];
      vs[v].get(s);
      unpack8(vy[v], y);
      unpack8(w[v], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(s[i], s[i], ss);
        ts = fmaf(y[i] * g[i], s[i], ts);
      }
    }
    ss = row_sum<kWarpRow>(ss, s_sum[turn]);
    ts = row_sum<kWarpRow>(ts, s_sum[turn + 1]);
    turn ^= 2;
    float q = __frsqrt_rn(ss / a.H + a.eps);
    float mean = ts * q / a.H;  // of t n
    if (!(fabsf(ts) < INFINITY) || ss == INFINITY) {
      if (ss == INFINITY) {
        float small = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          float s[8];
          vs[v].get(s);
#pragma unroll
          for (int i = 0; i < 8; ++i) small = fmaf(s[i] * kShrink, s[i] * kShrink, small);
        }
        q = root_of_small(row_sum<kWarpRow>(small, s_sum[turn]), a.H, a.eps);
      }
      float tn = 0.f;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        float s[8], y[8], g[8];
        vs[v].get(s);
        unpack8(vy[v], y);
        unpack8(w[v], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) tn = fmaf(y[i] * g[i], s[i] * q, tn);
      }
      mean = row_sum<kWarpRow>(tn, s_sum[turn + 1]) / a.H;
      turn ^= 2;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = v * across + at;
      float s[8], y[8], g[8], d[8];
      vs[v].get(s);
      unpack8(vy[v], y);
      unpack8(w[v], g);
      vd[v].get(d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = s[i] * q;
        dw[v][i] = fmaf(y[i], n, dw[v][i]);
        d[i] = fmaf(q, fmaf(-n, mean, y[i] * g[i]), d[i]);
      }
      if (c < chunks && a.d_x != nullptr) Eight<kFp32>::store(a.d_x, base + c * 8, d);
    }
  }
  if (a.part == nullptr) return;
  const int64_t owner = kWarpRow ? first : blockIdx.x;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * across + at;
    if (c < chunks) {
      float* to = a.part + owner * a.H + c * 8;
      *reinterpret_cast<float4*>(to) = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
      *reinterpret_cast<float4*>(to + 4) = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
    }
  }
}

// The same for many rows of more than 512 columns: the CTAs, 512 threads of them to an SM, take their rows from rings in shared
// memory, which bulk copies of whole rows keep full, so that the next rows arrive while this one is added
// up (65536 x 7168 with d_sum: 598 instead of 853 us for the kernel above, whose CTAs load and
// add in turn). The one barrier of a row, for its sums, also says that the row before it is
// used up, and the thread that sends for rows does so behind it.
constexpr int kRingThreads = 512, kRingMax = 8;

template <bool kFp32, int kV>
__global__ void __launch_bounds__(kRingThreads, 1) norm_grad_ring_kernel(NormGradArgs a, int stages, uint32_t stage_bytes) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 s_sum[2][kRingThreads / 32];
  __shared__ float s_more[2][32];
  __shared__ __align__(8) uint64_t s_full[kRingMax];
  __shared__ volatile int s_abort;
  constexpr uint32_t kSize = kFp32 ? 4 : 2;
  const int at = threadIdx.x, across = blockDim.x, lane = at & 31, warp = at >> 5, chunks = a.H >> 3;
  const uint32_t row_bytes = a.H * kSize, y_bytes = a.H * 2;
  const bool through = a.d_sum != nullptr && a.d_x != nullptr;
  if (at == 0) {
    for (int i = 0; i < stages; ++i) mbar_init_count(smem_addr(&s_full[i]), 1);
    s_abort = 0;
    fence_barrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  // row, d_y, d_sum of one row; of a padding row nothing (but the barrier's phase passes)
  auto send = [&](int64_t row, int stage) {
    const uint32_t bar = smem_addr(&s_full[stage]), to = smem_addr(ring + stage * stage_bytes);
    if (a.mask != nullptr && __ldg(a.mask + row) == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_expect(bar, row_bytes + y_bytes + (through ? row_bytes : 0));
    auto copy = [&](uint32_t dst, const void* src, uint32_t bytes) {
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                   "l"(src), "r"(bytes), "r"(bar)
                   : "memory");
    };
    copy(to, static_cast<const uint8_t*>(a.sum) + row * row_bytes, row_bytes);
    copy(to + row_bytes, a.d_y + row * a.H, y_bytes);
    if (through) copy(to + row_bytes + y_bytes, static_cast<const uint8_t*>(a.d_sum) + row * row_bytes, row_bytes);
  };
  uint4 w[kV];
  float dw[kV][8];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * across + at;
    w[v] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (c < chunks && a.weight != nullptr) w[v] = __ldg(reinterpret_cast<const uint4*>(a.weight + c * 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  if (at == 0)
    for (int i = 0; i + 1 < stages; ++i)
      if (const int64_t row = blockIdx.x + static_cast<int64_t>(i) * gridDim.x; row < a.rows) send(row, i);
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const bool live = a.mask == nullptr || __ldg(a.mask + row) != 0;
    // a wait that gives up is the last one: the results are incomplete, and reported
    if (!mbar_try<false>(smem_addr(&s_full[stage]), phase) && s_abort == 0 && !mbar_wait_timed<false>(smem_addr(&s_full[stage]), phase)) {
      if (s_abort == 0) atomicOr(a.err, kErrTimeout);
      s_abort = 1;
    }
    const uint8_t* from = ring + stage * stage_bytes;
    auto chunk = [&](const uint8_t* p, int c, float (&f)[8]) {
      if constexpr (kFp32) {
        const float4 l = *reinterpret_cast<const float4*>(p + c * 32), h = *reinterpret_cast<const float4*>(p + c * 32 + 16);
        f[0] = l.x, f[1] = l.y, f[2] = l.z, f[3] = l.w, f[4] = h.x, f[5] = h.y, f[6] = h.z, f[7] = h.w;
      } else {
        unpack8(*reinterpret_cast<const uint4*>(p + c * 16), f);
      }
    };
    auto y_chunk = [&](int c, float (&f)[8]) { unpack8(*reinterpret_cast<const uint4*>(from + row_bytes + c * 16), f); };
    float ss = 0.f, ts = 0.f;
    if (live) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int c = v * across + at;
        if (c >= chunks) break;
        float s[8], y[8], g[8];
        chunk(from, c, s);
        y_chunk(c, y);
        unpack8(w[v], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(s[i], s[i], ss);
          ts = fmaf(y[i] * g[i], s[i], ts);
        }
      }
    }
    ss = warp_sum(ss);
    ts = warp_sum(ts);
    if (lane == 0) s_sum[turn][warp] = make_float2(ss, ts);
    __syncthreads();
    // the row before is used up by all: its stage may be filled again
    if (at == 0) {
      const int64_t next = row + static_cast<int64_t>(stages - 1) * gridDim.x;
      if (next < a.rows && s_abort == 0) send(next, stage == 0 ? stages - 1 : stage - 1);
    }
    const float2 part = lane < across >> 5 ? s_sum[turn][lane] : make_float2(0.f, 0.f);
    turn ^= 1;
    ss = warp_sum(part.x);
    ts = warp_sum(part.y);
    float q = __frsqrt_rn(ss / a.H + a.eps), mean = ts * q / a.H;
    if (live && (!(fabsf(ts) < INFINITY) || ss == INFINITY)) {  // the same for the whole CTA
      if (ss == INFINITY) {
        float small = 0.f;
        for (int v = 0; v < kV; ++v) {
          const int c = v * across + at;
          if (c >= chunks) break;
          float s[8];
          chunk(from, c, s);
          for (int i = 0; i < 8; ++i) small = fmaf(s[i] * kShrink, s[i] * kShrink, small);
        }
        q = root_of_small(row_sum<false>(small, s_more[0]), a.H, a.eps);
      }
      float tn = 0.f;
      for (int v = 0; v < kV; ++v) {
        const int c = v * across + at;
        if (c >= chunks) break;
        float s[8], y[8], g[8];
        chunk(from, c, s);
        y_chunk(c, y);
        unpack8(w[v], g);
        for (int i = 0; i < 8; ++i) tn = fmaf(y[i] * g[i], s[i] * q, tn);
      }
      mean = row_sum<false>(tn, s_more[1]) / a.H;
      __syncthreads();  // before the next row that comes here writes there
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int c = v * across + at;
      if (c >= chunks) break;
      float d[8] = {};
      if (live) {
        float s[8], y[8], g[8];
        chunk(from, c, s);
        y_chunk(c, y);
        unpack8(w[v], g);
        if (through) chunk(from + row_bytes + y_bytes, c, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = s[i] * q;
          dw[v][i] = fmaf(y[i], n, dw[v][i]);
          d[i] = fmaf(q, fmaf(-n, mean, y[i] * g[i]), d[i]);
        }
      }
      if (a.d_x != nullptr) Eight<kFp32>::store(a.d_x, row * a.H + c * 8, d);
    }
    if (++stage == stages) stage = 0, phase ^= 1u;
  }
  if (at == 0 && s_abort != 0)  // copies in flight end before the CTA does
    for (int i = 0; i < stages; ++i) {
      mbar_wait_timed<false>(smem_addr(&s_full[i]), 0);
      mbar_wait_timed<false>(smem_addr(&s_full[i]), 1);
    }
  if (a.part == nullptr) return;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int c = v * across + at;
    if (c < chunks) {
      float* to = a.part + static_cast<int64_t>(blockIdx.x) * a.H + c * 8;
      *reinterpret_cast<float4*>(to) = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
      *reinterpret_cast<float4*>(to + 4) = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
    }
  }
}

// d_weight: a CTA takes 32 columns; each of its 32 warps every 32nd partial sum, all on their way before the first is
// used, and adds them in pairs, then a warp a column the warps' sums in pairs: 10 roundings at most. (Chains of 38 terms in
// each of 8 warps: 1021 x 2048 fp32 off by 1.4e-7 of the norm and 12.4 us for the whole call, now 1.0e-7 and 10.1 us.)
constexpr int kWeightWarps = 32, kWeightTerms = (kNormGradCtas + kWeightWarps - 1) / kWeightWarps;

__global__ void __launch_bounds__(kWeightWarps * 32) norm_weight_kernel(const float* part, int parts, int H, float* d_weight) {
  __shared__ float s_sum[kWeightWarps][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v[kWeightTerms];
#pragma unroll
  for (int k = 0; k < kWeightTerms; ++k) {
    const int p = way + kWeightWarps * k;
    v[k] = p < parts && c < H ? __ldcg(part + static_cast<int64_t>(p) * H + c) : 0.f;
  }
#pragma unroll
  for (int step = 1; step < kWeightTerms; step *= 2)
#pragma unroll
    for (int k = 0; k + step < kWeightTerms; k += 2 * step) v[k] += v[k + step];
  s_sum[way][lane] = v[0];
  __syncthreads();
  const float s = warp_sum(s_sum[lane][way]);
  if (lane == 0 && blockIdx.x * 32 + way < H) d_weight[blockIdx.x * 32 + way] = s;
}

// How a row is spread: a warp for rows of up to 512 columns, else a CTA whose threads hold the fewest
// chunks of 8 columns that its threads suffice for where rows are few and each should be as fast as
// it can be, and `most` chunks otherwise.
struct Shape {
  int v, threads, rows;  // rows: a CTA works on at once
  bool warp_row;
};

Shape shape_of(int H, bool few, int most, int one_chunk_threads) {
  const int chunks = H / 8;
  if (chunks <= 64) return Shape{chunks <= 32 ? 1 : 2, 128, 4, true};
  int v = few ? (chunks <= one_chunk_threads ? 1 : 2) : most;
  if ((chunks + v - 1) / v > (v == 1 ? one_chunk_threads : 512)) v = 4;
  return Shape{v, ((chunks + v - 1) / v + 31) / 32 * 32, 1, false};
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args), const Args& a, const Shape& s, int64_t most, int num_sms, int* ctas,
                        cudaStream_t stream) {
  const int per_sm = resident_ctas(reinterpret_cast<const void*>(kernel), s.threads, 0);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  int64_t n = (a.rows + s.rows - 1) / s.rows;
  if (n > static_cast<int64_t>(num_sms) * per_sm) n = static_cast<int64_t>(num_sms) * per_sm;
  if (n > most) n = most;
  *ctas = static_cast<int>(n);
  return launch_chained(kernel, dim3(static_cast<unsigned>(n)), dim3(s.threads), 0, stream, a);
}

template <bool kFp32>
cudaError_t launch_norm_typed(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const Shape s = shape_of(a.H, a.rows <= num_sms, 4, 1024);
  int n;
  auto go = [&](void (*kernel)(NormArgs)) { return launch_rows(kernel, a, s, INT32_MAX, num_sms, &n, stream); };
  if (s.warp_row) return s.v == 1 ? go(norm_kernel<kFp32, 1, true>) : go(norm_kernel<kFp32, 2, true>);
  if (s.v == 1) return go(norm_kernel<kFp32, 1, false>);
  return s.v == 2 ? go(norm_kernel<kFp32, 2, false>) : go(norm_kernel<kFp32, 4, false>);
}

template <bool kFp32>
cudaError_t launch_norm_grad_typed(const NormGradArgs& a, int num_sms, cudaStream_t stream) {
  const Shape s = shape_of(a.H, a.rows <= num_sms, 2, 512);
  int n = 0;
  auto go = [&](void (*kernel)(NormGradArgs)) {
    return launch_rows(kernel, a, s, kNormGradCtas / s.rows, num_sms, &n, stream);
  };
  cudaError_t st;
  // threads of a CTA of the ring's: a chunk of 8 columns each in rows of up to 4096
  const int threads = a.H <= 1024 ? 128 : a.H <= 2048 ? 256 : kRingThreads, per_sm = kRingThreads / threads;
  const uint32_t stage_bytes = (static_cast<uint32_t>(a.H) * ((kFp32 ? 4 : 2) * (a.d_sum != nullptr ? 2 : 1) + 2) + 127u) & ~127u;
  const int stages = static_cast<int>(min(216u / per_sm * 1024u / stage_bytes, static_cast<uint32_t>(kRingMax)));
  if (!s.warp_row && a.rows >= 2 * num_sms && stages >= 3) {
    n = num_sms * per_sm < kNormGradCtas ? num_sms * per_sm : kNormGradCtas;
    if (n > a.rows) n = static_cast<int>(a.rows);
    auto ring = [&](void (*kernel)(NormGradArgs, int, uint32_t)) {
      const size_t smem = static_cast<size_t>(stages) * stage_bytes;
      if (resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem) < 1) return cudaErrorInvalidConfiguration;
      return launch_chained(kernel, dim3(n), dim3(threads), smem, stream, a, stages, stage_bytes);
    };
    const int v = (a.H / 8 + threads - 1) / threads;
    st = v <= 1 ? ring(norm_grad_ring_kernel<kFp32, 1>) : v <= 2 ? ring(norm_grad_ring_kernel<kFp32, 2>)
                                                                 : ring(norm_grad_ring_kernel<kFp32, 4>);
  } else if (s.warp_row) st = s.v == 1 ? go(norm_grad_kernel<kFp32, 1, true>) : go(norm_grad_kernel<kFp32, 2, true>);
  else if (s.v == 1) st = go(norm_grad_kernel<kFp32, 1, false>);
  else st = s.v == 2 ? go(norm_grad_kernel<kFp32, 2, false>) : go(norm_grad_kernel<kFp32, 4, false>);
  if (st != cudaSuccess || a.part == nullptr) return st;
  return launch_chained(norm_weight_kernel, dim3((a.H + 31) / 32), dim3(kWeightWarps * 32), 0, stream,
                        static_cast<const float*>(a.part), n * s.rows, a.H, a.d_weight);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int x_fp32, int num_sms, cudaStream_t stream) {
  return x_fp32 ? launch_norm_typed<true>(a, num_sms, stream) : launch_norm_typed<false>(a, num_sms, stream);
}

cudaError_t launch_norm_grad(const NormGradArgs& a, int x_fp32, int num_sms, cudaStream_t stream) {
  return x_fp32 ? launch_norm_grad_typed<true>(a, num_sms, stream) : launch_norm_grad_typed<false>(a, num_sms, stream);
}

}  // namespace ep
