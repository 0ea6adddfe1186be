// Helpers of the row-wise kernels (layer norm, the gated activation, 8-bit checkpoints):
// vectors of a row, sums over the threads of a row, and the 8-bit checkpoint's blocks.
//
// A row is shared by `tpr` threads (whole warps); a block holds blockDim/tpr rows.  A vector is
// VEC columns: 16 bytes (8 values of bf16, 4 of f32) for rows whose length and pitch are
// multiples of 8, one value for all others.  A warp's lanes hold neighbouring vectors, so the
// 32 columns of a checkpoint block sit in 32 / VEC neighbouring lanes of one warp.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace {

// ---- VEC values of a row as they lie in memory, and as floats -------------------------------
// Activations are read once: loads go past L1, which is left to the weights.  (Evict-first hints on
// loads and stores cost 3 to 7%: 479 us, 450 without, for the gated activation's backward pass at
// 196608 x 1408.)
template <typename T>
constexpr int kWide = 16 / int(sizeof(T));
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = __ldcg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_weight(const __nv_bfloat16* p) { q = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
  }
};
template <>
struct Raw<float, 4> {
  float4 q;
  __device__ __forceinline__ void load(const float* p) { q = __ldcg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void zero() { q = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const { v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w; }
};
template <>
struct Raw<__nv_bfloat16, 4> {                    // weights beside f32 activations
  uint2 q;
  __device__ __forceinline__ void load_weight(const __nv_bfloat16* p) { q = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void zero() { q = make_uint2(0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
  }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  __nv_bfloat16 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *p; }
  __device__ __forceinline__ void load_weight(const __nv_bfloat16* p) { q = *p; }
  __device__ __forceinline__ void zero() { q = __float2bfloat16_rn(0.f); }
  __device__ __forceinline__ void get(float* v) const { v[0] = __bfloat162float(q); }
};
template <>
struct Raw<float, 1> {
  float q;
  __device__ __forceinline__ void load(const float* p) { q = *p; }
  __device__ __forceinline__ void zero() { q = 0.f; }
  __device__ __forceinline__ void get(float* v) const { v[0] = q; }
};

template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* v) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  if constexpr (VEC == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4)
      *reinterpret_cast<float4*>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}

// VEC values of a weight vector (bf16, or f32 when f32 is set) from column col.
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int64_t col, float* v) {
  if constexpr (VEC == 1) {
    v[0] = f32 ? __ldg(static_cast<const float*>(w) + col)
               : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + col));
  } else if (f32) {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + col + j));
      v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + col + j));
      v[j] = bf16_lo(q.x); v[j + 1] = bf16_hi(q.x); v[j + 2] = bf16_lo(q.y); v[j + 3] = bf16_hi(q.y);
    }
  }
}

// A thread's NV vectors of a weight for a whole kernel: bf16 weights stay in registers as they lie
// in memory, f32 ones (twice the registers) are read again for every row, from L1.
template <int VEC, int NV>
struct Weight {
  const void* w;
  bool f32;
  int col0;
  Raw<__nv_bfloat16, VEC> r[NV];
  __device__ __forceinline__ Weight(const void* w_, bool f32_, int col0_, int H) : w(w_), f32(f32_), col0(col0_) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r[i].zero();
      if (w != nullptr && !f32 && col0 + i * (32 * VEC) < H)
        r[i].load_weight(static_cast<const __nv_bfloat16*>(w) + col0 + i * (32 * VEC));
    }
  }
  // vector i, inside the row; zeros without a weight
  __device__ __forceinline__ void get(int i, float* v) const {
    if (f32 && w != nullptr) {
      load_weight<VEC>(w, true, col0 + i * (32 * VEC), v);
      return;
    }
    r[i].get(v);
  }
};

// ---- arithmetic on vectors: two float32 operations per instruction where they are wide ---------
// (each rounded to nearest, as the single ones).
template <int VEC>
__device__ __forceinline__ void v_add(float* a, const float* b) {            // a += b
  if constexpr (VEC == 1) a[0] += b[0];
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const float2 r = __fadd2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]));
      a[j] = r.x;
      a[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void v_mul(float* a, const float* b) {            // a *= b
  if constexpr (VEC == 1) a[0] *= b[0];
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const float2 r = __fmul2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]));
      a[j] = r.x;
      a[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void v_fma(float* c, const float* a, const float* b) {   // c = a * b + c
  if constexpr (VEC == 1) c[0] = fmaf(a[0], b[0], c[0]);
  else
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const float2 r = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), make_float2(c[j], c[j + 1]));
      c[j] = r.x;
      c[j + 1] = r.y;
    }
}
template <int VEC>
__device__ __forceinline__ void v_fill(float* a, float x) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) a[j] = x;
}
template <int VEC>
__device__ __forceinline__ void v_copy(float* a, const float* b) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) a[j] = b[j];
}
// Largest |v| as float bits; a NaN or Inf among the values gives an exponent field of 255.
template <int VEC>
__device__ __forceinline__ uint32_t v_amax(const float* v) {
  if constexpr (VEC == 1) return abs_bits(v[0]);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j + 1 < VEC; j += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[j])), "f"(fabsf(v[j + 1])));
  return abs_bits(m);
}

// ---- rows on their way: a ring of 16-byte pieces in shared memory ----------------------------
// Every thread copies with cp.async the pieces that it alone will read, so the ring needs no
// barrier: cp_async_wait<N> returns when all but the thread's last N groups have landed.
template <int BYTES>                              // 4, 8 or 16
__device__ __forceinline__ void ring_copy(uint8_t* smem, const void* gmem) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ void ring_get(const uint8_t* p, float* v) {
  Raw<T, kWide<T>> r;
  r.q = *reinterpret_cast<const decltype(r.q)*>(p);
  r.get(v);
}

// ---- sums over the threads of a row -------------------------------------------------------
// N sums at once over the tpr threads of a row, in a fixed order; the row's threads call it
// together.  group: the row's place in its block; rows of more than one warp (at most 8 a block of
// 512 threads) meet at the barrier of that number plus one, 0 being the whole block's.  buf: 32 * N floats of shared memory; two calls in a
// row use different ones, so one barrier per call is enough.
template <int N>
__device__ __forceinline__ void row_sum(float* v, int tpr, int group, float* buf) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], off);
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = tpr >> 5, first = group * per;
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[warp * N + n] = v[n];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    // every warp adds the row's partial sums in the same tree
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = lane < per ? buf[(first + lane) * N + n] : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
      v[n] = s;
    }
  }
}

// ---- 8-bit checkpoints ----------------------------------------------------------------------
// One power-of-two scale per 32 consecutive values of a row and E4M3 codes, the quantization
// rule of the MX tensors; the last block of a row may be short.  Codes [rows][cols] row-major,
// scale codes [rows][ceil(cols/32)] row-major (these tensors feed no MMA, so the scales need
// no tile layout).
//
// Quantizes this thread's VEC values of its block (all lanes of the warp call it; lanes past the
// row's end bring zeros) and, when `in` is set, stores the codes at `codes` and, from the block's
// first lane (`first`), the scale code at `scale`.
template <int VEC>
__device__ __forceinline__ void store_act8(const float* v, bool in, uint8_t* codes, uint8_t* scale, bool first) {
  uint32_t amax = v_amax<VEC>(v);
  if constexpr (VEC == 1) {
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  } else {
#pragma unroll
    for (int off = 1; off < 32 / VEC; off *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  }
  if (!in) return;
  const uint32_t c = mx_scale_code(amax);
  const float m = c == 255u ? 0.f : mx_inv_scale(c);
  if constexpr (VEC == 1) {
    *codes = c == 255u ? 0x7Fu : uint8_t(cvt_e4m3x2(v[0] * m, 0.f));
  } else {
    uint32_t q[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      q[i] = cvt_e4m3x2(v[4 * i] * m, v[4 * i + 1] * m) | (cvt_e4m3x2(v[4 * i + 2] * m, v[4 * i + 3] * m) << 16);
      if (c == 255u) q[i] = 0x7F7F7F7Fu;
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(codes) = q[0];
  }
  if (first) *scale = uint8_t(c);
}

// 2^(c - 127); c = 0 is 2^-127 (subnormal), c = 255 only meets NaN codes.
__device__ __forceinline__ float act8_scale(uint32_t c) { return __uint_as_float(c == 0u ? 0x00400000u : c << 23); }

// Two E4M3 codes (low half of w) as floats.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A thread's VEC codes (as stored by store_act8) and their block's scale code.
template <int VEC>
struct Act8 {
  uint32_t q[VEC == 8 ? 2 : 1];
  uint32_t c;
  __device__ __forceinline__ void take(const uint8_t* p) {        // the codes at p
    if constexpr (VEC == 8) {
      const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
      q[0] = w.x;
      q[1] = w.y;
    } else if constexpr (VEC == 4) {
      q[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
    } else {
      q[0] = *p;
    }
  }
  __device__ __forceinline__ void get(float* v) const {
    const float s = act8_scale(c);
    if constexpr (VEC == 1) {
      v[0] = e4m3x2_to_float2(q[0]).x * s;
    } else {
      const float2 s2 = make_float2(s, s);
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float2 a = __fmul2_rn(e4m3x2_to_float2(q[i]), s2), b = __fmul2_rn(e4m3x2_to_float2(q[i] >> 16), s2);
        v[4 * i] = a.x;
        v[4 * i + 1] = a.y;
        v[4 * i + 2] = b.x;
        v[4 * i + 3] = b.y;
      }
    }
  }
};

}  // namespace
}  // namespace moe
