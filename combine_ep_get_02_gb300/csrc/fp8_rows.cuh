// The FP8 rows of the dispatch outside of it: the scale of 128 columns, its place, and values of codes.
#pragma once

#include "ep_device.cuh"

namespace ep {

// Scale of a group of 128 columns whose largest magnitude is amax (at least 1e-4), as the dispatch's
// cast has it: fp32 amax / 448 with the factor 448 / amax, or the least power of two 2^e that is not below
// amax / 448 (amax = m 2^k: e = k - 8, or k - 7 where m > 1.75) with the factor 2^-e.
struct RowScale {
  float inv;  // codes are e4m3(value * inv)
  float sf;
  uint8_t byte;  // e + 127
};
__device__ __forceinline__ RowScale row_scale(float amax, int sf_pack) {
  amax = fmaxf(amax, 1e-4f);
  RowScale s;
  if (sf_pack) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    s.inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    s.sf = 0.f;
    s.byte = static_cast<uint8_t>(e + 127);
  } else {
    s.inv = __fdiv_rn(448.f, amax);
    s.sf = __fdiv_rn(amax, 448.f);
    s.byte = 0;
  }
  return s;
}

// Writes the scale of group g of a row of G groups; packed rows are whole words, and the thread of the last
// group fills the last word's other bytes with zeros.
__device__ __forceinline__ void store_scale(float* sf, int64_t row, int g, int G, const RowScale& s, int sf_pack) {
  if (!sf_pack) {
    sf[row * G + g] = s.sf;
    return;
  }
  uint8_t* bytes = reinterpret_cast<uint8_t*>(sf) + row * ((G + 3) / 4 * 4);
  bytes[g] = s.byte;
  if (g == G - 1)
    for (int i = G; i < (G + 3) / 4 * 4; ++i) bytes[i] = 0;
}

// The scale of group g of a row.
__device__ __forceinline__ float load_scale(const float* sf, int64_t row, int g, int G, int sf_pack) {
  if (!sf_pack) return __ldg(sf + row * G + g);
  const uint32_t e = __ldg(reinterpret_cast<const uint8_t*>(sf) + row * ((G + 3) / 4 * 4) + g);
  return e ? __uint_as_float(e << 23) : __uint_as_float(0x00400000u);  // 2^(e - 127)
}

// 32 bytes, 32-byte aligned: a whole sector, which two 16-byte stores write in two.
__device__ __forceinline__ void st32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Four codes -> four floats; exact.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h) & 0xFFFFu), __NV_E4M3);
    const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&r));
    f[2 * h] = q.x;
    f[2 * h + 1] = q.y;
  }
}

}  // namespace ep
