// fp8_values.cuh -- bf16 values to 8 bits with a power-of-two scale for each block of 128: what
// the quantiser and the norm that quantises share on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp8.cuh"
#include "simple.cuh"

namespace boost_gb300 {

constexpr uint32_t kInf = 0x7f80u;      // bf16 infinity

// The larger magnitude in each half of a pair of magnitudes; a NaN gives way.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The same, but a NaN stays.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Whether a pair of magnitudes holds an infinity or a NaN: 0x7f80 and above carry into bit 15.
__device__ __forceinline__ bool not_finite2(uint32_t m) {
  return ((m + 0x00800080u) & 0x80008000u) != 0;
}

// Magnitudes of a pair, infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  uint32_t m = w & 0x7fff7fffu;
  if ((m & kInf) == kInf) m &= 0xffff0000u;
  if ((m & kInf << 16) == kInf << 16) m &= 0xffffu;
  return m;
}

__device__ __forceinline__ uint32_t larger_half(uint32_t w) {
  return max(w & 0xffffu, w >> 16);     // magnitudes order as integers
}

// Scale byte of a block whose largest finite magnitude has the bf16 bits m: its exponent less 8
// (15), and one more where the fraction is above 1.75, which adding 0x1f carries over.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  const int e = static_cast<int>((m + 0x1fu) >> 7) - (FMT == BOOST_E4M3 ? 8 : 15);
  return e < 0 ? 0 : e;
}

// The byte that is stored: 127 (a scale of 1) for zeros, which any factor leaves as they are.
__device__ __forceinline__ uint8_t stored_byte(uint32_t byte, uint32_t m, bool inside) {
  return static_cast<uint8_t>(inside && m != 0 ? byte : 127u);
}

// 2^(127 - byte), the factor that takes the block's values to 8 bits (byte <= 247, so the
// exponent field 254 - byte is that of a normal number).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two values to 8 bits, nearest even. A scaled finite value never exceeds fmax, so
// saturation only meets infinities, which the caller mends (mend_inf).
template <int FMT>
__device__ __forceinline__ uint32_t to8(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE,
                                  FMT == BOOST_E4M3 ? __NV_E4M3 : __NV_E5M2);
}

// One bf16 value's 8 bits where it is an infinity: NaN in e4m3, infinity in e5m2.
template <int FMT>
__device__ __forceinline__ uint32_t mend_inf(uint32_t bits16, uint32_t q8) {
  if ((bits16 & 0x7fffu) != kInf) return q8;
  return ((bits16 >> 8) & 0x80u) | (FMT == BOOST_E4M3 ? 0x7fu : 0x7cu);
}

// Two products in one instruction.
__device__ __forceinline__ float2 mul2(float a, float b, float f) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(f));
  return r;
}

// 8 values (a vector's four words) times `inv` to 8 bytes; with `mend` there may be infinities.
template <int FMT>
__device__ __forceinline__ uint2 quant8(const uint32_t* w, float inv, bool mend) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = mul2(bf16_lo(w[i]), bf16_hi(w[i]), inv);
    p[i] = to8<FMT>(v.x, v.y);
  }
  if (mend) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = mend_inf<FMT>(w[i] & 0xffffu, p[i] & 0xffu) |
             mend_inf<FMT>(w[i] >> 16, p[i] >> 8) << 8;
  }
  return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
}

// Largest finite magnitudes of kRows rows over the kLanes lanes (a power of two) that hold a
// block; two rows go through the shuffles in the halves of a word. Returns whether a block of
// the warp holds an infinity (or nothing but NaN). Without kMayInf every value is known to be
// finite.
template <int kRows, int kWords, int kLanes, bool kMayInf = true>
__device__ __forceinline__ bool block_tops(const uint32_t (&w)[kRows][kWords],
                                           uint32_t (&top)[kRows]) {
  uint32_t two[kRows / 2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    uint32_t m = w[r][0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = max2(m, w[r][i] & 0x7fff7fffu);
    top[r] = m;
  }
#pragma unroll
  for (int r = 0; r < kRows / 2; ++r)              // the larger half of each row's word
    two[r] = max2(__byte_perm(top[2 * r], top[2 * r + 1], 0x5410),
                  __byte_perm(top[2 * r], top[2 * r + 1], 0x7632));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
    for (int r = 0; r < kRows / 2; ++r)
      two[r] = max2(two[r], __shfl_xor_sync(0xffffffffu, two[r], o));
  bool special = false;
#pragma unroll
  for (int r = 0; r < kRows / 2; ++r) {
    top[2 * r] = two[r] & 0xffffu;
    top[2 * r + 1] = two[r] >> 16;
    if (kMayInf) special |= not_finite2(two[r]);
  }
  if (kMayInf) special = __any_sync(0xffffffffu, special);
  if (special) {                                   // again over the finite values
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      uint32_t f = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) f = max2(f, finite2(w[r][i]));
      f = larger_half(f);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, o));
      top[r] = f;
    }
  }
  return special;
}

}  // namespace boost_gb300
