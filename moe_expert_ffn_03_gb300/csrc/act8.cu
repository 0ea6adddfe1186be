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
// Vectors of a thread that are loaded before the first is worked on: with one, the loads of a row's
// next vector wait for the stores of the last (forward 371 -> 340 us at 196608 x 1408, unpack
// 31 -> 23 us at 8192 x 5632).  The backward pass on wide vectors, with three streams to write and
// 16 more registers a vector, is faster with one (480 us; 518 with two).
constexpr int unroll_fwd(int vec) { return vec == 1 ? 4 : 2; }
constexpr int unroll_bwd(int vec) { return vec == 1 ? 4 : 1; }
constexpr int unroll_act8(int) { return 4; }

// 1 / (1 + e^-g): the exponential and the reciprocal are the approximate instructions (about
// 1 + 1.2 |g| and 1 units in the last place, as in the fused layer).  Results below 2^-126 are 0, so
// silu(g) and silu'(g) are 0 below g = -87.3, where they are 1e-36 and less.
template <int VEC>
__device__ __forceinline__ void v_sigmoid(float* s, const float* g) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[j]) : "f"(1.f + __expf(-g[j])));
}

// A thread's place in a row that tpr threads walk: its row, whether there is one, its first column.
struct RowPlace {
  int64_t row;
  int t;
  __device__ __forceinline__ explicit RowPlace(int tpr)
      : row(int64_t(blockIdx.x) * (ROW_BLOCK / tpr) + threadIdx.x / tpr), t(threadIdx.x & (tpr - 1)) {}
};

// Bound by memory: 196608 x 1408 with checkpoint 322 us, 6.9 TB/s; 32768 x 14336 539 us, 7.0 TB/s.
template <int VEC, bool KEEP>
__global__ void __launch_bounds__(ROW_BLOCK) swiglu_fwd_kernel(const SwigluArgs a, int tpr) {
  constexpr int U = unroll_fwd(VEC);
  const RowPlace at(tpr);
  const int nb = (a.I + 31) >> 5;                 // checkpoint blocks of g (and of u)
  pdl_wait();
  if (at.row >= a.rows) return;                   // whole warps
  const int col0 = at.t * VEC, step = tpr * VEC;
  const __nv_bfloat16* gp = a.gu + at.row * a.ld_gu + col0;
  __nv_bfloat16* ap = a.a + at.row * a.ld_a + col0;
  uint8_t* codes = a.codes + at.row * 2 * a.I + col0;
  uint8_t* scales = a.scales + at.row * 2 * nb + (col0 >> 5);
  float p[VEC];
  v_fill<VEC>(p, a.prob != nullptr ? a.prob[at.row] : 1.f);
  for (int left = a.I - col0, base = a.I; base > 0; base -= U * step, left -= U * step) {
    Raw<__nv_bfloat16, VEC> rg[U], ru[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      rg[k].zero();
      ru[k].zero();
      if (left > k * step) {                      // this thread's columns are inside the row
        rg[k].load(gp + k * step);
        ru[k].load(gp + k * step + a.I);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (base <= k * step) break;                // whole rows' threads
      const bool in = left > k * step;
      float g[VEC], u[VEC], s[VEC];
      rg[k].get(g);
      ru[k].get(u);
      if constexpr (KEEP) {
        store_act8<VEC>(g, in, codes + k * step, scales + k * (step >> 5), (col0 & 31) == 0);
        store_act8<VEC>(u, in, codes + k * step + a.I, scales + k * (step >> 5) + nb, (col0 & 31) == 0);
      }
      if (in) {
        v_sigmoid<VEC>(s, g);
        v_mul<VEC>(s, g);
        v_mul<VEC>(s, u);
        v_mul<VEC>(s, p);
        store_vec<VEC>(ap + k * step, s);
      }
    }
    gp += U * step;
    ap += U * step;
    codes += U * step;
    scales += U * (step >> 5);
  }
}

// Bound by memory: from the checkpoint 196608 x 1408 449 us, 6.2 TB/s; 32768 x 14336 725 us, 6.5 TB/s.
template <int VEC, bool Q8>
__global__ void __launch_bounds__(ROW_BLOCK) swiglu_bwd_kernel(const SwigluArgs a, int tpr) {
  constexpr int U = unroll_bwd(VEC);
  __shared__ float sums[32];
  const RowPlace at(tpr);
  const int nb = (a.I + 31) >> 5;
  pdl_wait();
  if (at.row >= a.rows) return;                   // whole rows: row_sum's barriers are a row's own
  const int col0 = at.t * VEC, step = tpr * VEC;
  const __nv_bfloat16* gp = a.gu + at.row * a.ld_gu + col0;
  const __nv_bfloat16* dp_ = a.da + at.row * a.ld_da + col0;
  const uint8_t* codes = a.codes + at.row * 2 * a.I + col0;
  const uint8_t* scales = a.scales + at.row * 2 * nb + (col0 >> 5);
  __nv_bfloat16* o = a.dgu + at.row * a.ld_dgu + col0;
  __nv_bfloat16* ap = a.a + at.row * a.ld_a + col0;
  float p[VEC], dp[VEC];
  v_fill<VEC>(p, a.prob != nullptr ? a.prob[at.row] : 1.f);
  v_fill<VEC>(dp, 0.f);
  for (int left = a.I - col0; left > 0; left -= U * step) {
    Raw<__nv_bfloat16, VEC> r[U], rg[U], ru[U];    // rg, ru or qg, qu
    Act8<VEC> qg[U], qu[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (left <= k * step) break;
      r[k].load(dp_ + k * step);
      if constexpr (Q8) {
        qg[k].take(codes + k * step);
        qu[k].take(codes + k * step + a.I);
        qg[k].c = scales[k * (step >> 5)];
        qu[k].c = scales[k * (step >> 5) + nb];
      } else {
        rg[k].load(gp + k * step);
        ru[k].load(gp + k * step + a.I);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (left <= k * step) break;
      float g[VEC], u[VEC], d[VEC], s[VEC], w[VEC];
      if constexpr (Q8) {
        qg[k].get(g);
        qu[k].get(u);
      } else {
        rg[k].get(g);
        ru[k].get(u);
      }
      r[k].get(d);
      v_sigmoid<VEC>(s, g);
      v_mul<VEC>(g, s);                            // silu(g) = g s
      v_fill<VEC>(w, 1.f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] -= s[j];
      v_fma<VEC>(s, g, w);                         // silu'(g) = s + g s (1 - s)
      v_copy<VEC>(w, g);
      v_mul<VEC>(w, u);                            // silu(g) u
      v_fma<VEC>(dp, d, w);
      v_mul<VEC>(w, p);                            // a
      v_mul<VEC>(d, p);
      v_mul<VEC>(s, u);
      v_mul<VEC>(s, d);                            // dg
      v_mul<VEC>(g, d);                            // du
      store_vec<VEC>(o + k * step, s);
      store_vec<VEC>(o + k * step + a.I, g);
      if (a.a != nullptr) store_vec<VEC>(ap + k * step, w);
    }
    gp += U * step;
    dp_ += U * step;
    codes += U * step;
    scales += U * (step >> 5);
    o += U * step;
    ap += U * step;
  }
  if (a.dprob == nullptr) return;
  float sum[1] = {0.f};
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[0] += dp[j];
  row_sum<1>(sum, tpr, int(threadIdx.x / tpr), sums);
  if (at.t == 0) a.dprob[at.row] = sum[0];
}

// Bound by memory: 8192 x 5632 bf16 22.7 us, 6.1 TB/s.
template <typename T, int VEC>
__global__ void __launch_bounds__(ROW_BLOCK) act8_pack_kernel(const T* __restrict__ src, int64_t rows, int cols,
                                                              int64_t ld, uint8_t* codes, uint8_t* scales, int tpr) {
  constexpr int U = unroll_act8(VEC);
  const RowPlace at(tpr);
  pdl_wait();
  if (at.row >= rows) return;                     // whole warps
  const int col0 = at.t * VEC, step = tpr * VEC;
  src += at.row * ld + col0;
  codes += at.row * cols + col0;
  scales += at.row * ((cols + 31) >> 5) + (col0 >> 5);
  for (int left = cols - col0, base = cols; base > 0; base -= U * step, left -= U * step) {
    Raw<T, VEC> r[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      r[k].zero();
      if (left > k * step) r[k].load(src + k * step);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (base <= k * step) break;                // whole rows' threads
      float v[VEC];
      r[k].get(v);
      store_act8<VEC>(v, left > k * step, codes + k * step, scales + k * (step >> 5), (col0 & 31) == 0);
    }
    src += U * step;
    codes += U * step;
    scales += U * (step >> 5);
  }
}

// dst = the kept values, times gamma plus beta where given (the layer norm's output from its
// kept normalised input).  Bound by memory: 8192 x 5632 bf16 23.3 us, 6.0 TB/s.
template <typename T, int VEC>
__global__ void __launch_bounds__(ROW_BLOCK) act8_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int cols, const void* gamma, const void* beta,
                                                                bool w_f32, T* dst, int64_t ld, int tpr) {
  constexpr int U = unroll_act8(VEC);
  const RowPlace at(tpr);
  pdl_wait();
  if (at.row >= rows) return;
  const int col0 = at.t * VEC, step = tpr * VEC;
  codes += at.row * cols + col0;
  scales += at.row * ((cols + 31) >> 5) + (col0 >> 5);
  dst += at.row * ld + col0;
  for (int col = col0; col < cols; col += U * step) {
    Act8<VEC> q[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (col + k * step >= cols) break;
      q[k].take(codes + k * step);
      q[k].c = scales[k * (step >> 5)];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (col + k * step >= cols) break;
      float v[VEC];
      q[k].get(v);
      if (gamma != nullptr) {
        float g[VEC], b[VEC];
        load_weight<VEC>(gamma, w_f32, col + k * step, g);
        v_fill<VEC>(b, 0.f);
        if (beta != nullptr) load_weight<VEC>(beta, w_f32, col + k * step, b);
        v_fma<VEC>(b, v, g);
        v_copy<VEC>(v, b);
      }
      store_vec<VEC>(dst + k * step, v);
    }
    codes += U * step;
    scales += U * (step >> 5);
    dst += U * step;
  }
}

// Threads per row: a warp walks a row by itself when there are rows enough to fill the GPU
// with warps; fewer rows are shared by up to a whole block, and so are rows of at least `steps` = 4
// steps a thread: long rows shared by a block touch fewer places of memory at once (gated activation of
// 14336 columns, forward 593 -> 554 us; two steps a thread already cost 1408 columns 11%).
int threads_per_row(int64_t rows, int cols, int vec, int steps = 1 << 20) {
  int tpr = 32;
  while (tpr < ROW_BLOCK && tpr * vec < cols &&
         (rows * tpr < int64_t(152) * 2048 || int64_t(tpr) * 2 * vec * steps <= cols))
    tpr *= 2;
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
  const int tpr = vec ? threads_per_row(a.rows, a.I, 8, 4) : threads_per_row(a.rows, a.I, 1);
  const dim3 grid = row_grid(a.rows, tpr);
  if (a.codes != nullptr) {
    if (vec) return launch_pdl(swiglu_fwd_kernel<8, true>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
    return launch_pdl(swiglu_fwd_kernel<1, true>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
  }
  if (vec) return launch_pdl(swiglu_fwd_kernel<8, false>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
  return launch_pdl(swiglu_fwd_kernel<1, false>, grid, dim3(ROW_BLOCK), 0, st, a, tpr);
}

cudaError_t launch_swiglu_bwd(const SwigluArgs& a, cudaStream_t st) {
  const bool q8 = a.codes != nullptr;
  const bool vec = a.I % 8 == 0 && (q8 || a.ld_gu % 8 == 0) && a.ld_da % 8 == 0 && a.ld_dgu % 8 == 0 &&
                   (a.a == nullptr || a.ld_a % 8 == 0);
  const int tpr = vec ? threads_per_row(a.rows, a.I, 8, 4) : threads_per_row(a.rows, a.I, 1);
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
