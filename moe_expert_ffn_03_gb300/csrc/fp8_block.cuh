// 8 bits with one f32 scale per block of 128: the rule, for the kernels that write such tensors.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int B8 = 128;                          // values of a block along a row or a column
constexpr float B8_TINY = 0x1p-100f;             // the smallest magnitude a scale is made for: 448 / amax stays finite

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
    return cvt_e4m3x2(v[0] * up, v[1] * up) | (cvt_e4m3x2(v[2] * up, v[3] * up) << 16);
  }
  __device__ __forceinline__ uint8_t code(float v) const { return uint8_t(cvt_e4m3x2(v * up, 0.f)); }
};

}  // namespace
}  // namespace moe
