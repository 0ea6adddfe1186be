// 8 bits with one f32 scale per block of 128: the rule, for the kernels that write such tensors.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int B8 = 128;                          // values of a block along a row or a column
constexpr float B8_TINY = 0x1p-100f;             // the smallest magnitude a scale is made for: 448 / amax stays finite

// The factor codes are made with, and the scale that gives their values back, from the block's largest
// magnitude (float bits): each one division, rounded once.  A block with a NaN or an Inf has NaN codes.
struct Block8 {
  float up;                                      // 448 / amax
  bool bad;
  __device__ __forceinline__ explicit Block8(uint32_t amax_bits) {
    bad = amax_bits >= 0x7F800000u;
    up = __fdiv_rn(448.f, fmaxf(__uint_as_float(amax_bits), B8_TINY));
  }
  __device__ __forceinline__ Block8(float up_, bool bad_) : up(up_), bad(bad_) {}
  static __device__ __forceinline__ float scale(uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? 1.f : __fdiv_rn(fmaxf(__uint_as_float(amax_bits), B8_TINY), 448.f);
  }
  __device__ __forceinline__ uint32_t codes4(const float* v) const {
    const uint32_t q = cvt_e4m3x2(v[0] * up, v[1] * up) | (cvt_e4m3x2(v[2] * up, v[3] * up) << 16);
    return bad ? 0x7F7F7F7Fu : q;
  }
  __device__ __forceinline__ uint8_t code(float v) const { return bad ? 0x7Fu : uint8_t(cvt_e4m3x2(v * up, 0.f)); }
};

}  // namespace
}  // namespace moe
