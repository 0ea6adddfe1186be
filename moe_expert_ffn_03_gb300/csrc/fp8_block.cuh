// 8 bits with one f32 scale per block of 128: the rule, for the kernels that write such tensors.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int B8 = 128;                          // values of a block along a row or a column
constexpr float B8_TINY = 0x1p-100f;             // the smallest magnitude a scale is made for: 448 / amax stays finite

// Codes of four values times their factors.
__device__ __forceinline__ uint32_t block8_codes4(const float* v, const float* up) {
  const float2 a = __fmul2_rn(make_float2(v[0], v[1]), make_float2(up[0], up[1]));
  const float2 b = __fmul2_rn(make_float2(v[2], v[3]), make_float2(up[2], up[3]));
  return cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
}

// The factor codes are made with, and the scale that gives their values back, from the block's largest
// magnitude (float bits): each one division, rounded once.  A block with a NaN or an Inf has NaN codes: its
// factor is NaN, and so is what any value gives times that.
struct Block8 {
  float up;                                      // 448 / amax
  __device__ __forceinline__ explicit Block8(uint32_t amax_bits) {
    up = amax_bits >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : __fdiv_rn(448.f, fmaxf(__uint_as_float(amax_bits), B8_TINY));
  }
  __device__ __forceinline__ explicit Block8(float up_) { up = up_; }
  static __device__ __forceinline__ float scale(uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? 1.f : __fdiv_rn(fmaxf(__uint_as_float(amax_bits), B8_TINY), 448.f);
  }
  __device__ __forceinline__ uint32_t codes4(const float* v) const {
    const float f[4] = {up, up, up, up};
    return block8_codes4(v, f);
  }
  __device__ __forceinline__ uint8_t code(float v) const { return uint8_t(cvt_e4m3x2(v * up, 0.f)); }
};

}  // namespace
}  // namespace moe
