// What the products need around the tensor cores: the tensor maps, FP8 rows as bf16,
// and the gradient through the activation with the bias gradient's sums.
#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// FP8 rows -> bf16, exactly: the codes (fp32 scales are applied to the products' sums), or codes
// times a power of two, one per 128 columns, packed four to a word (exact down to bf16's
// least numbers). A warp takes 2048 columns of a row, a lane 16 at a time: 16 bytes in, 32
// out. Rows past the last region are not part of any block and are left out. (Codes times fp32
// scales rounded to bf16 put the products' error at 2.8e-3 of their norm instead of the 1.7e-3 of
// their own rounding.) Measured: 65536 x 7168 in 226 us (1.4 GB, 6.2 TB/s).
__global__ void __launch_bounds__(kThreads)
    dequant_kernel(const uint8_t* x, const float* x_sf, uint16_t* out, int rows, int K, const int32_t* total) {
  pdl_launch_dependents();
  pdl_wait();
  if (total != nullptr) rows = max(0, min(rows, __ldg(total)));
  const int SW = ((K >> 7) + 3) >> 2, lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kThreads / 32), spans = (K + 2047) / 2048;
  const int units = rows * spans;  // their bytes fit memory, so their number fits 32 bits
  for (int u = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int r = u / spans, c0 = (u - r * spans) * 2048;
    const uint8_t* in = x + static_cast<int64_t>(r) * K;
    uint16_t* to = out + static_cast<int64_t>(r) * K;
    const float* sfs = x_sf + static_cast<int64_t>(r) * SW;
#pragma unroll 4
    for (int c = c0 + lane * 16; c < min(K, c0 + 2048); c += 512) {
      const int grp = c >> 7;
      float sf = 1.f;
      if (x_sf != nullptr) {
        const uint32_t e = __float_as_uint(__ldg(sfs + (grp >> 2))) >> (8 * (grp & 3)) & 0xFFu;
        sf = e ? __uint_as_float(e << 23) : __uint_as_float(0x00400000u);  // 2^(e-127)
      }
      const uint4 v = ld_stream16(in + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float f[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_fp8x2_storage_t p = static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu);
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(p, __NV_E4M3);  // exact
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * j] = q.x * sf;
        f[2 * j + 1] = q.y * sf;
      }
      st32(to + c, pack8(f), pack8(f + 8));  // a whole sector: with two 16-byte stores 285 us instead of 226
    }
  }
}

// dz = d_out * act'(z), rounded to bf16 for the products (their operands are bf16; it puts their error at
// 2.3e-3 of the gradients' norm, where their own rounding alone leaves 1.7e-3; a second
// bf16 term would double the products), and the bias gradient: the column
// sums of the unrounded dz over each tile of kDzRows rows, which the last CTA to finish of
// a group's tiles adds up in their order (a kernel of its own for that took 4 to 18 us). A CTA takes such a tile of one group and 128
// output columns: 16 threads across (8 columns each, 256 bytes of a row), 16 down, so that a
// few thousand rows already occupy every SM evenly. Memory bounds it, with GELU the arithmetic:
// 4096 x 4096 GELU 30 us (100 MB), 16384 x 1024 gated 29 us (168 MB, 5.8 TB/s).
constexpr int kSpan = kDzColumns, kAcross = kSpan / 8, kDown = kThreads / kAcross;
// Kept rows in a tile where there are so many that every CTA has several: a tile's column sums cost
// about as much as the rows of half a small tile (65536 x 2 x 2048: 272 us with 64 rows, 248 with 256).
constexpr int kKeptRows = 256;
constexpr int kBiasWays = 8;  // orders the bias gradients' sums, here and in bias_sum_kernel

struct DzArgs {
  Groups groups;
  int N, Z;
  const uint16_t* z;
  const uint16_t* d_out;
  uint16_t* dz;  // null: only the sums
  float* part;   // null: no sums
  float* d_bias;
  uint32_t* done;  // [E][spans]: tiles finished (returns to 0); null: the sums stay in part
  uint32_t* err;
  const uint8_t* codes = nullptr;  // z kept in 8 bits, in its place ...
  const float* z_sf = nullptr;     // ... with its scales
  int sf_pack = 0;
  uint16_t* h = nullptr;           // act(z) again; may be null
  int tile_rows = kDzRows;         // of a tile; kept rows: kDzRows or kKeptRows
};

// Eight columns of a kept row as they lie in memory, with their scale.
struct KeptEight {
  uint2 q;
  float s;
  __device__ __forceinline__ void load(const DzArgs& a, int64_t row, int c) {
    q = ld_stream8(a.codes + row * a.Z + c);
    s = load_scale(a.z_sf, row, c >> 7, a.Z >> 7, a.sf_pack);
  }
};

// Two floats that one instruction takes at once.
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma_two(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ uint32_t pack_two(Two a) {
  const float2 f = both(a);
  return f32x2_to_bf16x2(f.x, f.y);
}
// 1 / (1 + exp(-z)); 0 for z below -88, NaN for NaN
__device__ __forceinline__ Two sigmoid_two(Two z) {
  const float2 e = both(z * two(-1.4426950408889634f, -1.4426950408889634f));
  float a, b;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(e.y));
  const float2 o = both(two(a, b) + two(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(o.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(o.y));
  return two(a, b);
}
// act(z) and act'(z)
template <int kAct>
__device__ __forceinline__ void act_two(Two z, Two& v, Two& g) {
  if constexpr (kAct == EP_ACT_SILU || kAct == EP_ACT_SWIGLU) {
    const Two s = sigmoid_two(z);
    v = z * s;
    // s (1 + z (1 - s)); s + v (1 - s) from v + s is (z + 1) - z where s is 1: nothing is left of it from 2^24 on
    g = s * fma_two(z, fma_two(s, two(-1.f, -1.f), two(1.f, 1.f)), two(1.f, 1.f));
  } else {
    const float2 f = both(z);
    v = two(activate<kAct>(f.x), activate<kAct>(f.y));
    g = two(activate_grad<kAct>(f.x), activate_grad<kAct>(f.y));
  }
}
__device__ __forceinline__ Two two_of_bf16(uint32_t w) {
  const float2 f = bf16x2_to_f32x2(w);
  return two(f.x, f.y);
}
// the k-th two of eight kept columns
__device__ __forceinline__ Two two_of_kept(const KeptEight& e, int k, Two s) {
  const uint32_t w = k & 2 ? e.q.y : e.q.x;
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (k & 1)) & 0xFFFFu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
  return two(f.x, f.y) * s;
}

template <int kAct, bool kKept = false>
__global__ void __launch_bounds__(kThreads, kKept ? 2 : 0) dz_kernel(DzArgs a) {
  constexpr bool kGated = kAct == EP_ACT_SWIGLU;
  constexpr int kHalves = kGated ? 2 : 1;
  extern __shared__ int prefix[];  // [E + 1]
  __shared__ float s_sum[kDown][kHalves * kSpan];
  pdl_launch_dependents();
  pdl_wait();
  const int tile_rows = kKept ? a.tile_rows : kDzRows;
  build_prefix<kThreads>(a.groups, tile_rows, prefix, blockIdx.x == 0 ? a.err : nullptr);
  __shared__ bool s_last;
  const int across = threadIdx.x % kAcross, down = threadIdx.x / kAcross;
  const int spans = (a.N + kSpan - 1) / kSpan;
  if (a.done != nullptr)  // groups without a row
    for (int g = blockIdx.x; g < a.groups.E; g += gridDim.x)
      if (prefix[g] == prefix[g + 1])
        for (int c = threadIdx.x; c < a.Z; c += kThreads) a.d_bias[static_cast<int64_t>(g) * a.Z + c] = 0.f;
  const int64_t units = static_cast<int64_t>(prefix[a.groups.E]) * spans;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = static_cast<int>(u / spans), col = static_cast<int>(u - static_cast<int64_t>(tile) * spans) * kSpan + across * 8;
    const int g = group_of_tile(prefix, a.groups.E, tile);
    const GroupRows rows = group_rows(a.groups, g);
    const int m0 = (tile - prefix[g]) * tile_rows, n = min(tile_rows, rows.count - m0);
    const int64_t first = static_cast<int64_t>(rows.begin) + m0;
    float sum[kHalves * 8];
#pragma unroll
    for (int i = 0; i < kHalves * 8; ++i) sum[i] = 0.f;
    Two sum2[kKept ? kHalves * 4 : 1];
#pragma unroll
    for (int i = 0; i < (kKept ? kHalves * 4 : 1); ++i) sum2[i] = two(0.f, 0.f);
    if (col < a.N) {
      if constexpr (kKept) {
        // a thread's rows of the tile are all on their way before the first is used (65536 x 2 x 2048 gated: 281 us
        // instead of 385 with one after the other, and 272 once pairs of floats went through one instruction)
        constexpr int kRows = kDzRows / kDown;
        const bool needs_z = kAct != EP_ACT_NONE || a.h != nullptr;
#pragma unroll 1
        for (int r0 = 0; r0 < n; r0 += kDzRows) {
          KeptEight zg[kRows], zu[kGated ? kRows : 1];
          uint4 dv[kRows];
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kDown + down;
            if (r >= n) break;
            dv[i] = ld_stream16(a.d_out + (first + r) * a.N + col);
            if (needs_z) zg[i].load(a, first + r, col);
            if constexpr (kGated) zu[i].load(a, first + r, a.N + col);
          }
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int64_t row = first + r0 + i * kDown + down;
            if (r0 + i * kDown + down >= n) break;
            const uint32_t dw[4] = {dv[i].x, dv[i].y, dv[i].z, dv[i].w};
            uint32_t again[4], t[kHalves][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const Two d = two_of_bf16(dw[k]);
              if constexpr (kGated) {
                Two v, g;
                act_two<kAct>(two_of_kept(zg[i], k, two(zg[i].s, zg[i].s)), v, g);
                const Two u = two_of_kept(zu[i], k, two(zu[i].s, zu[i].s));
                const Two t0 = d * u * g, t1 = d * v;
                again[k] = pack_two(v * u);
                t[0][k] = pack_two(t0);
                t[1][k] = pack_two(t1);
                sum2[k] = sum2[k] + t0;
                sum2[4 + k] = sum2[4 + k] + t1;
              } else {
                Two v = two(0.f, 0.f), t0 = d;
                if (needs_z) {
                  Two g;
                  act_two<kAct>(two_of_kept(zg[i], k, two(zg[i].s, zg[i].s)), v, g);
                  if constexpr (kAct != EP_ACT_NONE) t0 = d * g;
                }
                again[k] = pack_two(v);
                t[0][k] = pack_two(t0);
                sum2[k] = sum2[k] + t0;
              }
            }
            if (a.h != nullptr) st16(a.h + row * a.N + col, make_uint4(again[0], again[1], again[2], again[3]));
            if (a.dz != nullptr) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                st16(a.dz + row * a.Z + h * a.N + col, make_uint4(t[h][0], t[h][1], t[h][2], t[h][3]));
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kHalves * 4; ++k) {
          const float2 f = both(sum2[k]);
          sum[2 * k] = f.x;
          sum[2 * k + 1] = f.y;
        }
      } else {
#pragma unroll 4
        for (int r = down; r < n; r += kDown) {
          const int64_t row = first + r;
          float d[8], t[kHalves * 8];
          unpack8(ld_stream16(a.d_out + row * a.N + col), d);
          if constexpr (kGated) {
            float zg[8], zu[8];
            unpack8(ld_stream16(a.z + row * a.Z + col), zg);
            unpack8(ld_stream16(a.z + row * a.Z + a.N + col), zu);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              t[i] = d[i] * zu[i] * activate_grad<kAct>(zg[i]);
              t[8 + i] = d[i] * activate<kAct>(zg[i]);
            }
          } else if constexpr (kAct == EP_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = d[i];
          } else {
            float zv[8];
            unpack8(ld_stream16(a.z + row * a.Z + col), zv);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = d[i] * activate_grad<kAct>(zv[i]);
          }
          if (a.dz != nullptr) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) st16(a.dz + row * a.Z + h * a.N + col, pack8(t + 8 * h));
          }
#pragma unroll
          for (int i = 0; i < kHalves * 8; ++i) sum[i] += t[i];
        }
      }
    }
    if (a.part != nullptr) {
      constexpr int kColumns = kHalves * kSpan;
      float* sums = &s_sum[0][0];
      const int tiles = prefix[g + 1] - prefix[g], span = col / kSpan;
      // column i of the CTA's, in z and in d_bias; past N: none
      auto column = [&](int i) {
        const int h = i / kSpan, c = span * kSpan + i - h * kSpan;
        return c < a.N ? h * a.N + c : -1;
      };
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_sum[down][h * kSpan + across * 8 + i] = sum[8 * h + i];
      __syncthreads();
      float* to = tiles == 1 && a.done != nullptr ? a.d_bias + static_cast<int64_t>(g) * a.Z : a.part + static_cast<int64_t>(tile) * a.Z;
      for (int i = threadIdx.x; i < kColumns; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kDown; ++k) s += s_sum[k][i];
        if (const int c = column(i); c >= 0) to[c] = s;
      }
      if (tiles > 1 && a.done != nullptr) {
        __threadfence();
        __syncthreads();
        uint32_t* done = a.done + static_cast<int64_t>(g) * spans + span;
        if (threadIdx.x == 0) s_last = atomicAdd(done, 1u) == static_cast<uint32_t>(tiles) - 1u;
        __syncthreads();
        if (s_last) {  // every kBiasWays-th tile, then the ways in order, as bias_sum_kernel
          __threadfence();
          for (int i = threadIdx.x; i < kBiasWays * kColumns; i += kThreads) {
            const int way = i / kColumns, c = column(i - way * kColumns);
            float s = 0.f;
            if (c >= 0) {
#pragma unroll 8
              for (int t = prefix[g] + way; t < prefix[g + 1]; t += kBiasWays)
                s += __ldcg(a.part + static_cast<int64_t>(t) * a.Z + c);
            }
            sums[i] = s;
          }
          __syncthreads();
          for (int i = threadIdx.x; i < kColumns; i += kThreads) {
            float s = sums[i];
#pragma unroll
            for (int w = 1; w < kBiasWays; ++w) s += sums[w * kColumns + i];
            if (const int c = column(i); c >= 0) a.d_bias[static_cast<int64_t>(g) * a.Z + c] = s;
          }
          if (threadIdx.x == 0) *done = 0u;
        }
      }
      __syncthreads();
    }
  }
}

// d_bias_g = the sum over the group's row tiles: 32 columns a CTA, 8 ways of every 8th tile,
// then the ways in order. (A thread for all tiles of a column took 18 us at 4096 rows.)
__global__ void __launch_bounds__(kThreads) bias_sum_kernel(Groups q, int tile_rows, int Z, const float* part, float* d_bias) {
  constexpr int kWays = kBiasWays;
  static_assert(kWays == kThreads / 32, "a warp a way");
  extern __shared__ int prefix[];
  __shared__ float s_sum[kWays][32];
  pdl_launch_dependents();
  pdl_wait();
  build_prefix<kThreads>(q, tile_rows, prefix, nullptr);
  const int way = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int spans = (Z + 31) / 32;
  const int64_t units = static_cast<int64_t>(q.E) * spans;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int g = static_cast<int>(u / spans), c = static_cast<int>(u - static_cast<int64_t>(g) * spans) * 32 + lane;
    float s = 0.f;
    if (c < Z) {
#pragma unroll 8
      for (int t = prefix[g] + way; t < prefix[g + 1]; t += kWays) s += __ldcg(part + static_cast<int64_t>(t) * Z + c);
    }
    s_sum[way][lane] = s;
    __syncthreads();
    if (way == 0 && c < Z) {
#pragma unroll
      for (int w = 1; w < kWays; ++w) s += s_sum[w][lane];
      d_bias[static_cast<int64_t>(g) * Z + c] = s;
    }
    __syncthreads();
  }
}

template <int kAct, bool kKept = false>
cudaError_t launch_dz(DzArgs a, int num_sms, cudaStream_t stream) {
  auto kern = dz_kernel<kAct, kKept>;
  const size_t smem = sizeof(int) * (static_cast<size_t>(a.groups.E) + 1);
  const int per_sm = resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t ctas = static_cast<int64_t>(num_sms) * per_sm, spans = (a.N + kSpan - 1) / kSpan;
  if (kKept && max_row_tiles(a.groups, kKeptRows) * spans >= 8 * ctas) a.tile_rows = kKeptRows;
  const int64_t most = max_row_tiles(a.groups, a.tile_rows) * spans;
  if (a.part == nullptr || most > ctas || a.groups.E * ((a.N + kSpan - 1) / kSpan) > kDzCounters) a.done = nullptr;
  const cudaError_t st = launch_chained(kern, dim3(static_cast<unsigned>(most < ctas ? most : ctas)), dim3(kThreads), smem, stream, a);
  if (st != cudaSuccess || a.part == nullptr || a.done != nullptr) return st;
  const int sum_per_sm = resident_ctas(reinterpret_cast<const void*>(bias_sum_kernel), kThreads, smem);
  if (sum_per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t need = static_cast<int64_t>(a.groups.E) * ((a.Z + 31) / 32);
  const int64_t sum_ctas = static_cast<int64_t>(num_sms) * sum_per_sm;
  return launch_chained(bias_sum_kernel, dim3(static_cast<unsigned>(need < sum_ctas ? need : sum_ctas)), dim3(kThreads),
                        smem, stream, a.groups, a.tile_rows, a.Z, static_cast<const float*>(a.part), a.d_bias);
}

}  // namespace

cudaError_t make_strided_map(CUtensorMap* map, const void* base, int dims, const uint64_t* size, const uint64_t* stride,
                             const uint32_t* box) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  // the driver's function, looked up once per process
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  cuuint64_t sizes[4], strides[3];
  cuuint32_t boxes[4], steps[4];
  for (int i = 0; i < dims; ++i) {
    sizes[i] = size[i];
    boxes[i] = box[i];
    steps[i] = 1;
    if (i + 1 < dims) strides[i] = stride[i];
  }
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(dims), const_cast<void*>(base),
                            sizes, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            box[0] == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_tensor_map(CUtensorMap* map, const void* base, int dims, const uint64_t* size, const uint32_t* box) {
  uint64_t stride[3], bytes = 2;
  for (int i = 0; i + 1 < dims; ++i) stride[i] = bytes *= size[i];
  return make_strided_map(map, base, dims, size, stride, box);
}

cudaError_t launch_dequant(const ProductGeometry& g, const uint8_t* x, const float* x_sf, uint16_t* out, int num_sms,
                           cudaStream_t stream) {
  const int per_sm = resident_ctas(reinterpret_cast<const void*>(dequant_kernel), kThreads, 0);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t need = (static_cast<int64_t>(g.groups.rows) * ((g.K + 2047) / 2048) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t ctas = static_cast<int64_t>(num_sms) * per_sm;
  const int32_t* total = g.groups.region == nullptr ? nullptr : g.groups.region + g.groups.E / g.groups.L;
  return launch_chained(dequant_kernel, dim3(static_cast<unsigned>(need < ctas ? need : ctas)), dim3(kThreads), 0, stream,
                        x, x_sf, out, g.groups.rows, g.K, total);
}

cudaError_t launch_product_dz(const ProductGradArgs& p, int num_sms, cudaStream_t stream) {
  const DzArgs a = {p.g.groups, p.g.N, p.g.Z, p.z, p.d_out, p.dz, p.part, p.d_bias, p.done, p.err};
  switch (p.g.act) {
    case EP_ACT_RELU: return launch_dz<EP_ACT_RELU>(a, num_sms, stream);
    case EP_ACT_SILU: return launch_dz<EP_ACT_SILU>(a, num_sms, stream);
    case EP_ACT_GELU: return launch_dz<EP_ACT_GELU>(a, num_sms, stream);
    case EP_ACT_SWIGLU: return launch_dz<EP_ACT_SWIGLU>(a, num_sms, stream);
    default: return launch_dz<EP_ACT_NONE>(a, num_sms, stream);
  }
}

cudaError_t launch_checkpoint_grad(const CheckpointGradArgs& p, int num_sms, cudaStream_t stream) {
  DzArgs a = {p.groups, p.N, p.Z, nullptr, p.d_h, p.d_z, p.part, p.d_bias, p.done, p.err};
  a.codes = p.codes;
  a.z_sf = p.sf;
  a.sf_pack = p.sf_pack;
  a.h = p.h;
  switch (p.act) {
    case EP_ACT_RELU: return launch_dz<EP_ACT_RELU, true>(a, num_sms, stream);
    case EP_ACT_SILU: return launch_dz<EP_ACT_SILU, true>(a, num_sms, stream);
    case EP_ACT_GELU: return launch_dz<EP_ACT_GELU, true>(a, num_sms, stream);
    case EP_ACT_SWIGLU: return launch_dz<EP_ACT_SWIGLU, true>(a, num_sms, stream);
    default: return launch_dz<EP_ACT_NONE, true>(a, num_sms, stream);
  }
}

}  // namespace ep
