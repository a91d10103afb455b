// Rows of an expanded layout's blocks kept in 8 bits (the dispatch's FP8 rows: e4m3 codes and a scale
// per 128 columns), and back in bf16. Rows outside the blocks' lanes are neither read nor written.
#include "dispatch_common.cuh"

#include "block_internal.cuh"
#include "fp8_rows.cuh"
#include "product_common.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 256, kAcross = kSpan / 16, kDown = kThreads / kAcross;  // columns a CTA takes, 16 a thread

// A CTA takes 64 rows of a block and 256 columns: 16 threads across, 16 columns each (8 neighbouring
// threads share a scale), 16 rows down. Memory bounds it: nothing is read or written twice.
template <bool kBack>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(CheckpointArgs a) {
  extern __shared__ int prefix[];  // [E + 1]
  pdl_launch_dependents();
  pdl_wait();
  build_prefix<kThreads>(a.groups, kDzRows, prefix, blockIdx.x == 0 ? a.err : nullptr);
  const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;  // rows are whole ones, the tensor may begin inside one
  const int across = threadIdx.x % kAcross, down = threadIdx.x / kAcross;
  const int spans = (a.F + kSpan - 1) / kSpan, G = a.F >> 7;
  const int64_t units = static_cast<int64_t>(prefix[a.groups.E]) * spans;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = static_cast<int>(u / spans), col = static_cast<int>(u - static_cast<int64_t>(tile) * spans) * kSpan + across * 16;
    const int g = group_of_tile(prefix, a.groups.E, tile);
    const GroupRows rows = group_rows(a.groups, g);
    const int m0 = (tile - prefix[g]) * kDzRows, n = min(kDzRows, rows.count - m0);
    const bool in = col < a.F;  // the same for the 8 threads of a scale
    constexpr int kRows = kDzRows / kDown;  // of a thread: all on their way before the first is used
    const int64_t row0 = static_cast<int64_t>(rows.begin) + m0 + down, at0 = row0 * a.F + col;
    const int64_t step = static_cast<int64_t>(kDown) * a.F;
    if constexpr (kBack) {
      uint4 q[kRows];
      float s[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (in && i * kDown + down < n) {
          q[i] = ld_stream16(static_cast<const uint8_t*>(a.in) + at0 + i * step);
          s[i] = load_scale(a.sf, row0 + i * kDown, col >> 7, G, a.sf_pack);
        }
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (in && i * kDown + down < n) {
          float f[16];
          e4m3x4_to_f32(q[i].x, f);
          e4m3x4_to_f32(q[i].y, f + 4);
          e4m3x4_to_f32(q[i].z, f + 8);
          e4m3x4_to_f32(q[i].w, f + 12);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] *= s[i];
          uint16_t* to = static_cast<uint16_t*>(a.out) + at0 + i * step;
          if (sectors) st32(to, pack8(f), pack8(f + 8));
          else st16(to, pack8(f)), st16(to + 8, pack8(f + 8));
        }
    } else {
      uint4 lo[kRows], hi[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
        if (in && i * kDown + down < n) {
          lo[i] = ld_stream16(static_cast<const uint16_t*>(a.in) + at0 + i * step);
          hi[i] = ld_stream16(static_cast<const uint16_t*>(a.in) + at0 + i * step + 8);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {  // whole warps take part in the maxima
        const bool there = in && i * kDown + down < n;
        const CastUnit c = cast_unit(lo[i], hi[i], there, a.sf_pack);
        if (there) {
          st16(static_cast<uint8_t*>(a.out) + at0 + i * step, c.q);
          if ((across & 7) == 0) store_scale(a.sf, row0 + i * kDown, col >> 7, G, RowScale{0.f, c.sf, c.sf_byte}, a.sf_pack);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_checkpoint(const CheckpointArgs& a, bool back, int num_sms, cudaStream_t stream) {
  auto kern = back ? checkpoint_kernel<true> : checkpoint_kernel<false>;
  const size_t smem = sizeof(int) * (static_cast<size_t>(a.groups.E) + 1);
  const int per_sm = resident_ctas(reinterpret_cast<const void*>(kern), kThreads, smem);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int64_t most = max_row_tiles(a.groups, kDzRows) * ((a.F + kSpan - 1) / kSpan);
  const int64_t ctas = static_cast<int64_t>(num_sms) * per_sm;
  return launch_chained(kern, dim3(static_cast<unsigned>(most < ctas ? most : ctas)), dim3(kThreads), smem, stream, a);
}

}  // namespace ep
