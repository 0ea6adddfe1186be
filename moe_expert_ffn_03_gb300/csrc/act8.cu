// The gated activation as an operator of its own, forward and backward, and activations kept
// in 8 bits between the two passes.
//
//   forward   a = silu(g) * u * p                     (g, u the halves of a row of gu)
//   backward  dg = da * p * u * silu'(g),  du = da * p * silu(g),  dp = sum da * silu(g) * u,
//             and a again (the next layer's weight gradient needs it, so it is not kept)
// with s = 1 / (1 + e^-g): silu(g) = g s, silu'(g) = s (1 + g (1 - s)).
//
// All of it is elementwise along a row apart from dp, so the kernels are bound by memory.  A
// row is shared by tpr threads that walk its columns tpr * VEC at a time.
#include "kernels.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int ROW_BLOCK = 256;

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <int VEC>
__global__ void __launch_bounds__(ROW_BLOCK) swiglu_fwd_kernel(const SwigluArgs a, int tpr) {
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = int64_t(blockIdx.x) * (ROW_BLOCK / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows;
  const int nb = (a.I + 31) >> 5;                 // checkpoint blocks of g (and of u)
  pdl_wait();
  const __nv_bfloat16* gp = a.gu + row * a.ld_gu;
  const float p = a.prob != nullptr && live ? a.prob[row] : 1.f;
  for (int c0 = 0; c0 < a.I; c0 += tpr * VEC) {
    const int col = c0 + t * VEC;
    const bool in = live && col < a.I;
    Raw<__nv_bfloat16, VEC> rg, ru;
    rg.zero();
    ru.zero();
    if (in) {
      rg.load(gp + col);
      ru.load(gp + a.I + col);
    }
    float g[VEC], u[VEC];
    rg.get(g);
    ru.get(u);
    if (a.codes != nullptr) {
      store_act8<VEC>(g, in, a.codes, a.scales, row, 2 * int64_t(a.I), 0, col, 2 * nb, 0);
      store_act8<VEC>(u, in, a.codes, a.scales, row, 2 * int64_t(a.I), a.I, col, 2 * nb, nb);
    }
    if (in) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j] * p;
      store_vec<VEC>(a.a + row * a.ld_a + col, g);
    }
  }
}

template <int VEC, bool Q8>
__global__ void __launch_bounds__(ROW_BLOCK) swiglu_bwd_kernel(const SwigluArgs a, int tpr) {
  __shared__ float sums[32];
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = int64_t(blockIdx.x) * (ROW_BLOCK / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows;
  const int nb = (a.I + 31) >> 5;
  pdl_wait();
  const float p = a.prob != nullptr && live ? a.prob[row] : 1.f;
  float dp[1] = {0.f};
  if (live) {
    for (int col = t * VEC; col < a.I; col += tpr * VEC) {
      float g[VEC], u[VEC], da[VEC];
      if constexpr (Q8) {
        Act8<VEC> qg, qu;
        qg.load(a.codes, a.scales, row, 2 * int64_t(a.I), 0, col, 2 * nb, 0);
        qu.load(a.codes, a.scales, row, 2 * int64_t(a.I), a.I, col, 2 * nb, nb);
        qg.get(g);
        qu.get(u);
      } else {
        Raw<__nv_bfloat16, VEC> rg, ru;
        rg.load(a.gu + row * a.ld_gu + col);
        ru.load(a.gu + row * a.ld_gu + a.I + col);
        rg.get(g);
        ru.get(u);
      }
      Raw<__nv_bfloat16, VEC> r;
      r.load(a.da + row * a.ld_da + col);
      r.get(da);
      float du[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float s = sigmoid(g[j]);
        const float silu = g[j] * s;
        const float dap = da[j] * p;
        dp[0] += da[j] * (silu * u[j]);
        du[j] = dap * silu;
        da[j] = silu * u[j] * p;                       // a
        g[j] = dap * u[j] * (s * (1.f + g[j] * (1.f - s)));
      }
      __nv_bfloat16* o = a.dgu + row * a.ld_dgu + col;
      store_vec<VEC>(o, g);
      store_vec<VEC>(o + a.I, du);
      if (a.a != nullptr) store_vec<VEC>(a.a + row * a.ld_a + col, da);
    }
  }
  if (a.dprob == nullptr) return;
  row_sum<1>(dp, tpr, int(threadIdx.x / tpr), sums);
  if (live && t == 0) a.dprob[row] = dp[0];
}

template <typename T, int VEC>
__global__ void __launch_bounds__(ROW_BLOCK) act8_pack_kernel(const T* __restrict__ src, int64_t rows, int cols,
                                                              int64_t ld, uint8_t* codes, uint8_t* scales, int tpr) {
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = int64_t(blockIdx.x) * (ROW_BLOCK / tpr) + threadIdx.x / tpr;
  const bool live = row < rows;
  pdl_wait();
  for (int c0 = 0; c0 < cols; c0 += tpr * VEC) {
    const int col = c0 + t * VEC;
    const bool in = live && col < cols;
    Raw<T, VEC> r;
    r.zero();
    if (in) r.load(src + row * ld + col);
    float v[VEC];
    r.get(v);
    store_act8<VEC>(v, in, codes, scales, row, cols, 0, col, (cols + 31) >> 5, 0);
  }
}

// dst = the kept values, times gamma plus beta where given (the layer norm's output from its
// kept normalised input).
template <typename T, int VEC>
__global__ void __launch_bounds__(ROW_BLOCK) act8_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int cols, const void* gamma, const void* beta,
                                                                bool w_f32, T* dst, int64_t ld, int tpr) {
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = int64_t(blockIdx.x) * (ROW_BLOCK / tpr) + threadIdx.x / tpr;
  pdl_wait();
  if (row >= rows) return;
  for (int col = t * VEC; col < cols; col += tpr * VEC) {
    Act8<VEC> q;
    q.load(codes, scales, row, cols, 0, col, (cols + 31) >> 5, 0);
    float v[VEC];
    q.get(v);
    if (gamma != nullptr) {
      float g[VEC], b[VEC];
      load_weight<VEC>(gamma, w_f32, col, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] = 0.f;
      if (beta != nullptr) load_weight<VEC>(beta, w_f32, col, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = v[j] * g[j] + b[j];
    }
    store_vec<VEC>(dst + row * ld + col, v);
  }
}

// Threads per row: a warp walks a row by itself when there are rows enough to fill the GPU
// with warps; fewer rows are shared by up to a whole block.
int threads_per_row(int64_t rows, int cols, int vec) {
  int tpr = 32;
  while (tpr < ROW_BLOCK && tpr * vec < cols && rows * tpr < int64_t(152) * 2048) tpr *= 2;
  return tpr;
}
dim3 row_grid(int64_t rows, int tpr) { return dim3(unsigned((rows + ROW_BLOCK / tpr - 1) / (ROW_BLOCK / tpr))); }

template <typename T>
cudaError_t pack_t(const void* src, int64_t rows, int cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                   cudaStream_t st) {
  const T* s = static_cast<const T*>(src);
  const bool vec = cols % 8 == 0 && ld % 8 == 0;
  const int tpr = threads_per_row(rows, cols, vec ? kWide<T> : 1);
  if (vec)
    return launch_pdl(act8_pack_kernel<T, kWide<T>>, row_grid(rows, tpr), dim3(ROW_BLOCK), 0, st, s, rows, cols, ld, codes,
                      scales, tpr);
  return launch_pdl(act8_pack_kernel<T, 1>, row_grid(rows, tpr), dim3(ROW_BLOCK), 0, st, s, rows, cols, ld, codes,
                    scales, tpr);
}

template <typename T>
cudaError_t unpack_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, const void* gamma,
                     const void* beta, bool w_f32, void* dst, int64_t ld, cudaStream_t st) {
  T* d = static_cast<T*>(dst);
  const bool vec = cols % 8 == 0 && ld % 8 == 0;
  const int tpr = threads_per_row(rows, cols, vec ? kWide<T> : 1);
  if (vec)
    return launch_pdl(act8_unpack_kernel<T, kWide<T>>, row_grid(rows, tpr), dim3(ROW_BLOCK), 0, st, codes, scales, rows, cols,
                      gamma, beta, w_f32, d, ld, tpr);
  return launch_pdl(act8_unpack_kernel<T, 1>, row_grid(rows, tpr), dim3(ROW_BLOCK), 0, st, codes, scales, rows, cols,
                    gamma, beta, w_f32, d, ld, tpr);
}

}  // namespace

cudaError_t launch_swiglu_fwd(const SwigluArgs& a, cudaStream_t st) {
  const bool vec = a.I % 8 == 0 && a.ld_gu % 8 == 0 && a.ld_a % 8 == 0;
  const int tpr = threads_per_row(a.rows, a.I, vec ? 8 : 1);
  const dim3 grid = row_grid(a.rows, tpr);
  if (vec) return launch_pdl(swiglu_fwd_kernel<8>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
  return launch_pdl(swiglu_fwd_kernel<1>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
}

cudaError_t launch_swiglu_bwd(const SwigluArgs& a, cudaStream_t st) {
  const bool q8 = a.codes != nullptr;
  const bool vec = a.I % 8 == 0 && (q8 || a.ld_gu % 8 == 0) && a.ld_da % 8 == 0 && a.ld_dgu % 8 == 0 &&
                   (a.a == nullptr || a.ld_a % 8 == 0);
  const int tpr = threads_per_row(a.rows, a.I, vec ? 8 : 1);
  const dim3 grid = row_grid(a.rows, tpr);
  if (vec) {
    if (q8) return launch_pdl(swiglu_bwd_kernel<8, true>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
    return launch_pdl(swiglu_bwd_kernel<8, false>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
  }
  if (q8) return launch_pdl(swiglu_bwd_kernel<1, true>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
  return launch_pdl(swiglu_bwd_kernel<1, false>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
}

cudaError_t launch_act8_pack(const void* src, bool f32, int64_t rows, int cols, int64_t ld, uint8_t* codes,
                             uint8_t* scales, cudaStream_t st) {
  return f32 ? pack_t<float>(src, rows, cols, ld, codes, scales, st)
             : pack_t<__nv_bfloat16>(src, rows, cols, ld, codes, scales, st);
}

cudaError_t launch_act8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, const void* gamma,
                               const void* beta, bool w_f32, void* dst, bool f32, int64_t ld, cudaStream_t st) {
  return f32 ? unpack_t<float>(codes, scales, rows, cols, gamma, beta, w_f32, dst, ld, st)
             : unpack_t<__nv_bfloat16>(codes, scales, rows, cols, gamma, beta, w_f32, dst, ld, st);
}

}  // namespace moe
