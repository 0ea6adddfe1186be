// Root-mean-square norm, forward and backward, with the residual's addition and an output in 8 bits (one f32
// scale per 128 values of a row) for the products that read it.
//
//   h = x (+ residual);  rstd = 1 / sqrt(mean h^2 + eps);  n = h * rstd;  y = n * gamma
// and with d = dy * gamma:
//   dx = rstd * (d - n * mean (d * n)) (+ dres);  dgamma = sum over rows of dy * n
//
// Everything between the loads and the stores is float32; the sum h is normalised before it is rounded, and
// the 8-bit rows are made of y before it is rounded.  Each activation is read once and written once, so memory
// bounds both passes.  Rows are laid out on threads and on the ring as in the layer norm (norm.cuh).
#include <cfloat>

#include "fp8_block.cuh"
#include "norm.cuh"

namespace moe {
namespace {

// Factors for rows whose mean square (with eps) is above float32's range or below 2^-120: squares of
// values below 2^128 are below 2^96 after RMS_LARGE, those of subnormal ones normal numbers after RMS_SMALL.
constexpr float RMS_LARGE = 0x1p-80f, RMS_SMALL = 0x1p100f;
__device__ __forceinline__ bool rms_in_range(float var) { return var >= 0x1p-120f && var <= FLT_MAX; }

// y of this thread's vectors of a row in 8 bits.  The 128 values of a block are in 128 / VEC neighbouring
// lanes, single columns in a warp's lanes and four vectors; past the row's end v holds zeros.
template <int VEC, int NV, typename P>
__device__ __forceinline__ void store_block8(const float (*v)[VEC], const P& at, int H, uint8_t* codes, float* scale,
                                             int64_t rows) {
  if constexpr (VEC > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t amax = v_amax<VEC>(v[i]);
#pragma unroll
      for (int off = 1; off < B8 / VEC; off *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
      if (at.col(i) >= H) continue;
      const Block8 b(amax);
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(codes + at.col(i)) = make_uint2(b.codes4(v[i]), b.codes4(v[i] + 4));
      else
        *reinterpret_cast<uint32_t*>(codes + at.col(i)) = b.codes4(v[i]);
      if (at.col(i) % B8 == 0) scale[int64_t(at.col(i) / B8) * rows] = Block8::scale(amax);
    }
  } else {
    static_assert(NV % 4 == 0, "a block is four vectors of single columns");
#pragma unroll
    for (int g = 0; g < NV; g += 4) {
      uint32_t amax = 0;
#pragma unroll
      for (int i = g; i < g + 4; ++i) amax = max(amax, abs_bits(v[i][0]));
      amax = __reduce_max_sync(0xFFFFFFFFu, amax);
      const Block8 b(amax);
#pragma unroll
      for (int i = g; i < g + 4; ++i)
        if (at.col(i) < H) codes[at.col(i)] = b.code(v[i][0]);
      if (at.col(g) % B8 == 0 && at.col(g) < H) scale[int64_t(at.col(g) / B8) * rows] = Block8::scale(amax);
    }
  }
}

// n -> y = n * gamma in place, then what the caller wants of it.
template <typename T, int VEC, int NV, typename P, typename G>
__device__ __forceinline__ void rms_outputs(const RmsArgs& a, const P& at, int64_t row, float (*n)[VEC], const G& gamma) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float g[VEC];
    v_fill<VEC>(g, 0.f);
    if (at.col(i) < a.H) gamma.get(i, g);
    v_mul<VEC>(n[i], g);
    if (a.y != nullptr && at.col(i) < a.H) store_vec<VEC>(static_cast<T*>(a.y) + row * a.ld_out + at.col(i), n[i]);
  }
  if (a.codes != nullptr) store_block8<VEC, NV>(n, at, a.H, a.codes + row * a.H, a.scales + row, a.rows);
}

// The rows of this thread's row group whose mean square (with eps) is above float32's range or below 2^-120,
// once more, on times a power of two: a loop of its own behind the kernel's.  Where h has taken the place
// of x or the residual by then, the row is h as stored.  sums[flip] is the buffer that the kernel's last sum has
// not used; from there on they take turns, also where a row turns out to be within range.
template <typename T, int VEC, int NV>
__device__ __noinline__ void rms_fwd_rescaled(const RmsArgs& a, int tpr, float (*sums)[32], int flip) {
  const Place<VEC, NV, 2, 0> at(tpr, nullptr);
  const Weight<VEC, NV> gamma(a.gamma, a.w_f32, at.col0, a.H);
  const float inv_H = 1.f / float(a.H);
  const bool summed = a.h != nullptr && (a.h == a.x || a.h == a.residual);
  const T* x = static_cast<const T*>(summed ? a.h : a.x);
  const T* res = static_cast<const T*>(summed ? nullptr : a.residual);
  float h[NV][VEC];
  // the row, and its mean square times f^2
  const auto load = [&](int64_t row, float f) {
    float w[VEC], sum[VEC];
    v_fill<VEC>(w, f);
    v_fill<VEC>(sum, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v_fill<VEC>(h[i], 0.f);
      if (at.col(i) >= a.H) continue;
      Raw<T, VEC> r;
      r.load(x + row * a.ld_in + at.col(i));
      r.get(h[i]);
      if (res != nullptr) {
        float v[VEC];
        r.load(res + row * a.ld_in + at.col(i));
        r.get(v);
        v_add<VEC>(h[i], v);
      }
      v_mul<VEC>(h[i], w);
      v_fma<VEC>(sum, h[i], h[i]);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += sum[j];
    row_sum<1>(s, tpr, at.group, sums[flip]);
    flip ^= 1;
    return s[0] * inv_H;
  };
  for (int64_t row = int64_t(blockIdx.x) * at.groups + at.group; row < a.rows; row += int64_t(gridDim.x) * at.groups) {
    const float var = load(row, 1.f) + a.eps;
    // bf16 rows as stored are not quite the sums: those near the bounds are taken along
    if (summed ? var >= 0x1p-119f && var <= 0x1p127f : rms_in_range(var)) continue;
    const float f = var < 1.f ? RMS_SMALL : RMS_LARGE;
    const float ms = load(row, f);
    float rstd = inv_sqrt(ms + a.eps * f * f);   // of the row as it is held
    if (at.t == 0 && a.rstd != nullptr) a.rstd[row] = ms == 0.f ? inv_sqrt(a.eps) : rstd * f;
    if (ms == 0.f && a.eps > 0.f) rstd = 0.f;    // eps * f * f may have gone under
    float w[VEC];
    v_fill<VEC>(w, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (at.col(i) < a.H) v_mul<VEC>(h[i], w);
    }
    rms_outputs<T, VEC, NV>(a, at, row, h, gamma);
  }
}

// A persistent grid: block b takes the row groups b, b + grid, ...  The next groups' x (and residual) are on
// their way to shared memory while the current one is summed.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(max_block(VEC), 1) rms_fwd_kernel(const __grid_constant__ RmsArgs a, int tpr) {
  constexpr int STG = ring_stages(VEC, 2 * NV);
  __shared__ float sums[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const Place<VEC, NV, 2, STG> at(tpr, ring);
  const float inv_H = 1.f / float(a.H);
  const int64_t step = int64_t(gridDim.x) * at.groups;
  const bool has_res = a.residual != nullptr;
  const auto fetch = [&](int64_t row, int st) {
    if constexpr (VEC > 1) {
      if (row < a.rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.ld_in + at.col0;
        const T* res = static_cast<const T*>(a.residual) + row * a.ld_in + at.col0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (at.col(i) < a.H) {
            ring_copy<16>(at.piece(st, 0, i), x + i * (32 * VEC));
            if (has_res) ring_copy<16>(at.piece(st, 1, i), res + i * (32 * VEC));
          }
      }
      cp_async_commit();
    }
  };
  // single columns: the next row's in registers instead, loaded unconditionally (column 0 past the row's end) so that
  // all are in flight at once (20000 x 1001 bf16 with a residual and 8-bit rows: 60 us, 68 when loaded as they are needed)
  constexpr int PRE = VEC == 1 && NV <= 8 ? NV : 0;
  Raw<T, 1> px[PRE + 1], pr[PRE + 1];
  const auto fetch_singles = [&](int64_t row) {
    if (PRE == 0 || row >= a.rows) return;
#pragma unroll
    for (int i = 0; i < PRE; ++i) {
      const int64_t off = row * a.ld_in + (at.col(i) < a.H ? at.col(i) : 0);
      px[i].load(static_cast<const T*>(a.x) + off);
      pr[i].zero();
      if (has_res) pr[i].load(static_cast<const T*>(a.residual) + off);
    }
  };
  if constexpr (VEC > 1) at.clear();
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * at.groups + at.group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  fetch_singles(row);
  const Weight<VEC, NV> gamma(a.gamma, a.w_f32, at.col0, a.H);
  int st = 0, flip = 0;
  bool odd = false;                               // the same in all of a row group's threads
  for (; row < a.rows; row += step, flip ^= 1) {
    if constexpr (VEC > 1) {
      fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
      cp_async_wait<STG - 1>();
    }
    float h[NV][VEC], sq[VEC];
    v_fill<VEC>(sq, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[VEC];
      if constexpr (VEC > 1) {
        ring_get<T>(at.piece(st, 0, i), h[i]);
        if (has_res) {
          ring_get<T>(at.piece(st, 1, i), v);
          v_add<VEC>(h[i], v);
        }
      } else {
        const bool in = at.col(i) < a.H;
        Raw<T, 1> x, r;
        if constexpr (PRE > 0) {
          x = px[i];
          r = pr[i];
        } else {
          const int64_t off = row * a.ld_in + (in ? at.col(i) : 0);
          x.load(static_cast<const T*>(a.x) + off);
          r.zero();
          if (has_res) r.load(static_cast<const T*>(a.residual) + off);
        }
        x.get(h[i]);
        r.get(v);
        h[i][0] = in ? h[i][0] + v[0] : 0.f;
      }
      v_fma<VEC>(sq, h[i], h[i]);
    }
    fetch_singles(row + step);
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += sq[j];
    row_sum<1>(s, tpr, at.group, sums[flip]);
    if (a.h != nullptr) {
      T* ho = static_cast<T*>(a.h) + row * a.ld_out + at.col0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (at.col(i) < a.H) store_vec<VEC>(ho + i * (32 * VEC), h[i]);
    }
    const float var = s[0] * inv_H + a.eps, rstd = inv_sqrt(var);
    odd |= !rms_in_range(var);
    if (at.t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    float rs[VEC];
    v_fill<VEC>(rs, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) v_mul<VEC>(h[i], rs);
    rms_outputs<T, VEC, NV>(a, at, row, h, gamma);
  }
  if (odd) rms_fwd_rescaled<T, VEC, NV>(a, tpr, sums, flip);
}

// A persistent grid and a ring as in the forward pass.  A thread keeps its columns' sums of dgamma in
// registers; at the end the block's groups are added in order and written as one partial sum per block,
// which rms_weight_grad_kernel adds in block order.  The second pass over a row finds it in registers where a
// thread has up to 16 columns, and reads the ring again where it has more.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(max_block(VEC), 1) rms_bwd_kernel(const RmsArgs a, int tpr, float* partial) {
  constexpr int STG = ring_stages(VEC, 3 * NV);
  constexpr bool HOLD = VEC * NV <= 16;
  __shared__ float sums[2][32];
  extern __shared__ __align__(16) uint8_t ring[]; // operands dy, dres, kept rows
  const Place<VEC, NV, 3, STG> at(tpr, ring);
  const int64_t step = int64_t(gridDim.x) * at.groups;
  const bool has_res = a.dres != nullptr;
  const auto fetch = [&](int64_t row, int st) {
    if constexpr (VEC > 1) {
      if (row < a.rows) {
        const int64_t off = row * a.ld_in + at.col0;
        const T* dy = static_cast<const T*>(a.dy) + off;
        const T* res = static_cast<const T*>(a.dres) + off;
        const T* x = static_cast<const T*>(a.x) + off;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (at.col(i) < a.H) {
            const int d = i * (32 * VEC);
            ring_copy<16>(at.piece(st, 0, i), dy + d);
            ring_copy<16>(at.piece(st, 2, i), x + d);
            if (has_res) ring_copy<16>(at.piece(st, 1, i), res + d);
          }
      }
      cp_async_commit();
    }
  };
  // single columns: the next row's in registers instead, as in the forward pass, up to four columns a thread (20000 x 1001
  // bf16: 63 us, 128 without; more do not fit the registers that 1024 threads have)
  constexpr int PRE = VEC == 1 && NV <= 4 ? NV : 0;
  Raw<T, 1> pd[PRE + 1], px[PRE + 1], pr[PRE + 1];
  const auto fetch_singles = [&](int64_t row) {
    if (PRE == 0 || row >= a.rows) return;
#pragma unroll
    for (int i = 0; i < PRE; ++i) {
      const int64_t off = row * a.ld_in + (at.col(i) < a.H ? at.col(i) : 0);
      pd[i].load(static_cast<const T*>(a.dy) + off);
      px[i].load(static_cast<const T*>(a.x) + off);
      pr[i].zero();
      if (has_res) pr[i].load(static_cast<const T*>(a.dres) + off);
    }
  };
  float dg[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) v_fill<VEC>(dg[i], 0.f);
  const float inv_H = 1.f / float(a.H);
  int flip = 0, st = 0;
  if constexpr (VEC > 1) at.clear();
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * at.groups + at.group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  fetch_singles(row);
  const Weight<VEC, NV> gamma(a.gamma, a.w_f32, at.col0, a.H);
  float next = row < a.rows ? a.rstd[row] : 0.f;
  for (; row < a.rows; row += step, flip ^= 1) {
    const float rstd = next;
    if constexpr (VEC > 1) fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
    next = row + step < a.rows ? a.rstd[row + step] : 0.f;
    if constexpr (VEC > 1) cp_async_wait<STG - 1>();
    float rs[VEC];
    v_fill<VEC>(rs, rstd);
    // dy and n (0 past the row's end) of vector i
    const auto get = [&](int i, float* d, float* n) {
      if constexpr (VEC > 1) {
        ring_get<T>(at.piece(st, 0, i), d);
        ring_get<T>(at.piece(st, 2, i), n);
      } else {
        const bool in = at.col(i) < a.H;
        if constexpr (PRE > 0) {
          pd[i].get(d);
          px[i].get(n);
        } else {
          const int64_t off = row * a.ld_in + (in ? at.col(i) : 0);
          Raw<T, 1> r;
          r.load(static_cast<const T*>(a.dy) + off);
          r.get(d);
          r.load(static_cast<const T*>(a.x) + off);
          r.get(n);
        }
        d[0] = in ? d[0] : 0.f;
        n[0] = in ? n[0] : 0.f;
      }
      v_mul<VEC>(n, rs);
    };
    float s2[VEC];
    float kn[HOLD ? NV : 1][VEC], kd[HOLD ? NV : 1][VEC];         // n and d * gamma, for the second pass
    v_fill<VEC>(s2, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&n)[VEC] = kn[HOLD ? i : 0], (&d)[VEC] = kd[HOLD ? i : 0], g[VEC];
      get(i, d, n);
      v_fill<VEC>(g, 0.f);
      if (at.col(i) < a.H) gamma.get(i, g);
      v_fma<VEC>(dg[i], d, n);
      v_mul<VEC>(d, g);
      v_fma<VEC>(s2, d, n);
    }
    Raw<T, 1> kr[PRE + 1];                       // this row's dres
#pragma unroll
    for (int i = 0; i < PRE; ++i) kr[i] = pr[i];
    fetch_singles(row + step);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += s2[j];
    row_sum<1>(s, tpr, at.group, sums[flip]);
    float m2[VEC];
    v_fill<VEC>(m2, -(s[0] * inv_H));
    T* dx = static_cast<T*>(a.dx) + row * a.ld_out + at.col0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (at.col(i) >= a.H) continue;
      float (&n)[VEC] = kn[HOLD ? i : 0], (&d)[VEC] = kd[HOLD ? i : 0], v[VEC];
      if constexpr (!HOLD) {
        float g[VEC];
        get(i, d, n);
        gamma.get(i, g);
        v_mul<VEC>(d, g);
      }
      v_fill<VEC>(v, 0.f);
      if (has_res) {
        if constexpr (VEC > 1) {
          ring_get<T>(at.piece(st, 1, i), v);
        } else if constexpr (PRE > 0) {
          kr[i].get(v);
        } else {
          Raw<T, 1> r;
          r.load(static_cast<const T*>(a.dres) + row * a.ld_in + at.col0 + i * 32);
          r.get(v);
        }
      }
      v_fma<VEC>(d, n, m2);
      v_fma<VEC>(v, d, rs);
      store_vec<VEC>(dx + i * (32 * VEC), v);
    }
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
  }
  // The block's row groups, added in order: every group's sums to shared memory (the ring is
  // free by now), then all threads add columns.
  float* fold = reinterpret_cast<float*>(ring);   // [group][H]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = at.col(i);
    if (col >= a.H) continue;
    float* f = fold + size_t(at.group) * a.H + col;
    if constexpr (VEC > 1) {
#pragma unroll
      for (int j = 0; j < VEC; j += 4)
        *reinterpret_cast<float4*>(f + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
    } else {
      f[0] = dg[i][0];
    }
  }
  __syncthreads();
  pdl_launch_dependents();
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
    float sum = fold[c];
    for (int g = 1; g < at.groups; ++g) sum += fold[size_t(g) * a.H + c];
    partial[int64_t(blockIdx.x) * a.H + c] = sum;
  }
}

// dgamma from the blocks' partial sums [parts][H]: 32 columns per block, 32 warps each add every 32nd
// part, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) rms_weight_grad_kernel(const float* __restrict__ partial, int parts, int H, bool w_f32,
                                                              void* dgamma) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  pdl_wait();
  float s = 0.f;
  if (col < H) {
#pragma unroll 5
    for (int p = warp; p < parts; p += 32) s += partial[int64_t(p) * H + col];
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= H) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += acc[w][lane];
  if (w_f32) static_cast<float*>(dgamma)[col] = s;
  else static_cast<__nv_bfloat16*>(dgamma)[col] = __float2bfloat16_rn(s);
}

template <typename T, int VEC, int NV>
cudaError_t rms_fwd_shape(const RmsArgs& a, const RowShape& s, cudaStream_t st) {
  static Resident known;
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  const size_t smem = size_t(ring_stages(VEC, 2 * NV)) * 2 * NV * 16 * s.block;
  int64_t most = 0;
  if (const cudaError_t e = resident_blocks(rms_fwd_kernel<T, VEC, NV>, s, smem, known, &most); e != cudaSuccess) return e;
  return launch_pdl(rms_fwd_kernel<T, VEC, NV>, dim3(unsigned(need < most ? need : most)), dim3(unsigned(s.block)),
                    smem, st, a, s.tpr);
}

template <typename T, int VEC, int NV>
cudaError_t rms_bwd_shape(const RmsArgs& a, const RowShape& s, float* partial, int* parts, cudaStream_t st) {
  static Resident known;
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  const size_t ring = size_t(ring_stages(VEC, 3 * NV)) * 3 * NV * 16 * s.block;
  const size_t fold = size_t(rpb) * a.H * sizeof(float);          // H <= tpr * VEC * NV: at most 64 KB
  const size_t smem = ring > fold ? ring : fold;
  int64_t grid = 0;
  if (const cudaError_t e = resident_blocks(rms_bwd_kernel<T, VEC, NV>, s, smem, known, &grid); e != cudaSuccess) return e;
  grid = grid < kNormMaxParts ? grid : kNormMaxParts;
  grid = grid < need ? grid : need;
  *parts = int(grid);
  return launch_pdl(rms_bwd_kernel<T, VEC, NV>, dim3(unsigned(grid)), dim3(unsigned(s.block)), smem, st, a, s.tpr,
                    partial);
}

template <typename T>
RowShape rms_shape(const RmsArgs& a, int wide_nv) {
  return row_shape(a.H, a.H % 8 == 0 && a.ld_in % 8 == 0 && a.ld_out % 8 == 0 ? kWide<T> : 1, wide_nv);
}

template <typename T>
cudaError_t rms_fwd_t(const RmsArgs& a, cudaStream_t st) {
  const RowShape s = rms_shape<T>(a, 4);
  return with_shape<T>(s, [&](auto vec, auto nv) { return rms_fwd_shape<T, vec.value, nv.value>(a, s, st); });
}

template <typename T>
cudaError_t rms_bwd_t(const RmsArgs& a, float* partial, int* parts, cudaStream_t st) {
  const RowShape s = rms_shape<T>(a, sizeof(T) == 2 ? 2 : 4);
  return with_shape<T>(s, [&](auto vec, auto nv) { return rms_bwd_shape<T, vec.value, nv.value>(a, s, partial, parts, st); });
}

}  // namespace

size_t rms_ws_bytes(int64_t rows, int H) {
  const int64_t parts = rows < kNormMaxParts ? rows : kNormMaxParts;
  return size_t(parts < 1 ? 1 : parts) * size_t(H) * sizeof(float);
}

cudaError_t launch_rms_fwd(const RmsArgs& a, bool x_f32, cudaStream_t st) {
  return x_f32 ? rms_fwd_t<float>(a, st) : rms_fwd_t<__nv_bfloat16>(a, st);
}

cudaError_t launch_rms_bwd(const RmsArgs& a, bool x_f32, float* partial, cudaStream_t st) {
  int parts = 0;
  if (a.rows > 0) {
    const cudaError_t e = x_f32 ? rms_bwd_t<float>(a, partial, &parts, st) : rms_bwd_t<__nv_bfloat16>(a, partial, &parts, st);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(rms_weight_grad_kernel, dim3(unsigned((a.H + 31) / 32)), dim3(1024), 0, st,
                    static_cast<const float*>(partial), parts, a.H, a.w_f32, a.dgamma);
}

}  // namespace moe
