// Layer norm, forward and backward, with its normalised input optionally kept in 8 bits.
//
//   h = x (+ residual);  mu = mean h;  rstd = 1 / sqrt(mean (h - mu)^2 + eps)
//   n = (h - mu) * rstd;  y = n * gamma + beta
// and with d = dy * gamma:
//   dx = rstd * (d - mean d - n * mean (d * n)) (+ dres)
//   dgamma = sum over rows of dy * n;  dbeta = sum over rows of dy
//
// Everything between the loads and the stores is float32: the variance is that of the centred
// values (a second pass over registers), and the sum h is normalised before it is rounded.
// Both kernels are bound by memory: each activation is read once and written once.
#include "kernels.cuh"
#include "rows.cuh"

namespace moe {
namespace {

// Threads of the largest block each shape is launched with (row_shape below).
constexpr int max_block(int vec, int nv) { return vec == 8 ? (nv <= 2 ? 256 : 512) : (nv <= 8 ? 512 : 1024); }

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(max_block(VEC, NV)) norm_fwd_kernel(const NormArgs a, int tpr) {
  __shared__ float sums[2][32];
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows;
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + row * a.ld_in;
  const T* res = static_cast<const T*>(a.residual) + row * a.ld_in;
  float h[NV][VEC];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * VEC;
    Raw<T, VEC> r, q;
    r.zero();
    q.zero();
    if (live && col < a.H) {
      r.load(x + col);
      if (a.residual != nullptr) q.load(res + col);
    }
    r.get(h[i]);
    float v[VEC];
    q.get(v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      h[i][j] += v[j];
      s[0] += h[i][j];
    }
  }
  row_sum<1>(s, tpr, sums[0]);
  const float inv_H = 1.f / float(a.H);
  const float mu = __fdiv_rn(s[0], float(a.H));   // exact for a constant row whose sum is
  if (a.h != nullptr && live) {
    T* ho = static_cast<T*>(a.h) + row * a.ld_out;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * VEC;
      if (col < a.H) store_vec<VEC>(ho + col, h[i]);
    }
  }
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (i * tpr + t) * VEC < a.H;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      h[i][j] = in ? h[i][j] - mu : 0.f;
      s[0] += h[i][j] * h[i][j];
    }
  }
  row_sum<1>(s, tpr, sums[1]);
  const float rstd = 1.f / sqrtf(s[0] * inv_H + a.eps);
  if (live && t == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ld_out;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * tpr + t) * VEC;
    const bool in = live && col < a.H;
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[i][j] *= rstd;
    if (a.codes != nullptr)
      store_act8<VEC>(h[i], in, a.codes, a.scales, row, a.H, 0, col, (a.H + 31) >> 5, 0);
    if (in) {
      float g[VEC], b[VEC];
      load_weight<VEC>(a.gamma, a.w_f32, col, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] = 0.f;
      if (a.beta != nullptr) load_weight<VEC>(a.beta, a.w_f32, col, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] = h[i][j] * g[j] + b[j];
      store_vec<VEC>(y + col, b);
    }
  }
}

// A persistent grid: block b takes the row groups b, b + grid, ... and keeps its threads'
// columns of dgamma and dbeta in registers; at the end the block's groups are added in order
// and written as one partial sum per block, which norm_weight_grad_kernel adds in block order.
template <typename T, int VEC, int NV, bool Q8>
__global__ void __launch_bounds__(max_block(VEC, NV)) norm_bwd_kernel(const NormArgs a, int tpr,
                                                                                 float* partial) {
  __shared__ float sums[2][64];
  extern __shared__ float fold[];                 // [2][H], used when the block holds several rows
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  const float inv_H = 1.f / float(a.H);
  int flip = 0;
  pdl_wait();
  for (int64_t row0 = int64_t(blockIdx.x) * groups; row0 < a.rows; row0 += int64_t(gridDim.x) * groups, flip ^= 1) {
    const int64_t row = row0 + group;
    const bool live = row < a.rows;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_in;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_in;
    const float mu = !Q8 && live ? a.mean[row] : 0.f;
    const float rstd = live ? a.rstd[row] : 0.f;
    float n[NV][VEC], d[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * VEC;
      const bool in = live && col < a.H;
      Raw<T, VEC> r;
      r.zero();
      if (in) r.load(dy + col);
      r.get(d[i]);
      if constexpr (Q8) {
        Act8<VEC> q;
        q.zero();
        if (in) q.load(a.codes, a.scales, row, a.H, 0, col, (a.H + 31) >> 5, 0);
        q.get(n[i]);
      } else {
        Raw<T, VEC> q;
        q.zero();
        if (in) q.load(x + col);
        q.get(n[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) n[i][j] = in ? (n[i][j] - mu) * rstd : 0.f;
      }
      float g[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] = 0.f;
      if (in) load_weight<VEC>(a.gamma, a.w_f32, col, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dg[i][j] += d[i][j] * n[i][j];
        db[i][j] += d[i][j];
        d[i][j] *= g[j];
        s[0] += d[i][j];
        s[1] += d[i][j] * n[i][j];
      }
    }
    row_sum<2>(s, tpr, sums[flip]);
    const float m1 = s[0] * inv_H, m2 = s[1] * inv_H;
    if (live) {
      T* dx = static_cast<T*>(a.dx) + row * a.ld_out;
      const T* res = static_cast<const T*>(a.dres) + row * a.ld_in;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * VEC;
        if (col >= a.H) continue;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = 0.f;
        if (a.dres != nullptr) {
          Raw<T, VEC> r;
          r.load(res + col);
          r.get(v);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += rstd * (d[i][j] - m1 - n[i][j] * m2);
        store_vec<VEC>(dx + col, v);
      }
    }
  }
  // the block's row groups, added in order
  for (int g = 1; g < groups; ++g) {
    __syncthreads();
    if (group == g) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int col = (i * tpr + t) * VEC + j;
          if (col < a.H) {
            fold[col] = dg[i][j];
            fold[a.H + col] = db[i][j];
          }
        }
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int col = (i * tpr + t) * VEC + j;
          if (col < a.H) {
            dg[i][j] += fold[col];
            db[i][j] += fold[a.H + col];
          }
        }
    }
  }
  if (group == 0) {
    float* p = partial + int64_t(blockIdx.x) * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int col = (i * tpr + t) * VEC + j;
        if (col < a.H) {
          p[col] = dg[i][j];
          p[a.H + col] = db[i][j];
        }
      }
  }
}

// dgamma and dbeta from the blocks' partial sums [parts][2][H]: 32 columns per block, eight
// warps each add every eighth part, then the eight sums are added in order.
__global__ void __launch_bounds__(256) norm_weight_grad_kernel(const float* __restrict__ partial, int parts, int H,
                                                              bool w_f32, void* dgamma, void* dbeta) {
  __shared__ float acc[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;         // 0 .. 2H-1: dgamma, then dbeta
  pdl_wait();
  float s = 0.f;
  if (col < 2 * H)
    for (int p = warp; p < parts; p += 8) s += partial[int64_t(p) * 2 * H + col];
  acc[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= 2 * H) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) s += acc[w][lane];
  void* out = col < H ? dgamma : dbeta;
  if (out == nullptr) return;
  const int c = col < H ? col : col - H;
  if (w_f32) static_cast<float*>(out)[c] = s;
  else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
}

struct RowShape {
  bool vec;      // 8-wide vectors
  int nv;        // vectors per thread
  int tpr;       // threads per row
  int block;     // threads per block
};

// Threads and vectors per row.  Wide rows: 2 vectors a thread up to 256 threads (4096
// columns), 4 above.  Single columns: 8 a thread up to 512 threads, then 16 and 1024.
RowShape row_shape(int H, bool vec) {
  RowShape s{vec, vec ? 2 : 8, 32, 256};
  const int n = vec ? H / 8 : H;                  // vectors of a row
  if (n > s.nv * (vec ? 256 : 512)) s.nv *= 2;
  while (s.tpr * s.nv < n) s.tpr *= 2;
  s.block = s.tpr > 256 ? s.tpr : 256;
  return s;
}

bool vec_ok(const NormArgs& a) { return a.H % 8 == 0 && a.ld_in % 8 == 0 && a.ld_out % 8 == 0; }

template <typename T>
cudaError_t norm_fwd_t(const NormArgs& a, cudaStream_t st) {
  const RowShape s = row_shape(a.H, vec_ok(a));
  const int64_t rpb = s.block / s.tpr;
  const dim3 grid(unsigned((a.rows + rpb - 1) / rpb));
  if (s.vec) {
    if (s.nv == 2) return launch_pdl(norm_fwd_kernel<T, 8, 2>, grid, dim3(s.block), 0, st, a, s.tpr);
    return launch_pdl(norm_fwd_kernel<T, 8, 4>, grid, dim3(s.block), 0, st, a, s.tpr);
  }
  if (s.nv == 8) return launch_pdl(norm_fwd_kernel<T, 1, 8>, grid, dim3(s.block), 0, st, a, s.tpr);
  return launch_pdl(norm_fwd_kernel<T, 1, 16>, grid, dim3(s.block), 0, st, a, s.tpr);
}

template <typename T, bool Q8>
cudaError_t norm_bwd_t(const NormArgs& a, float* partial, int max_parts, int* parts, cudaStream_t st) {
  const RowShape s = row_shape(a.H, vec_ok(a));
  const int64_t rpb = s.block / s.tpr;
  const int64_t need = (a.rows + rpb - 1) / rpb;
  *parts = int(need < max_parts ? need : max_parts);
  const dim3 grid = dim3(unsigned(*parts));
  const size_t smem = rpb > 1 ? size_t(2) * a.H * sizeof(float) : 0;   // at most 2 * 2048 floats (tpr <= 128)
  if (s.vec) {
    if (s.nv == 2) return launch_pdl(norm_bwd_kernel<T, 8, 2, Q8>, grid, dim3(s.block), smem, st, a, s.tpr, partial);
    return launch_pdl(norm_bwd_kernel<T, 8, 4, Q8>, grid, dim3(s.block), smem, st, a, s.tpr, partial);
  }
  if (s.nv == 8) return launch_pdl(norm_bwd_kernel<T, 1, 8, Q8>, grid, dim3(s.block), smem, st, a, s.tpr, partial);
  return launch_pdl(norm_bwd_kernel<T, 1, 16, Q8>, grid, dim3(s.block), smem, st, a, s.tpr, partial);
}

}  // namespace

// Partial sums the backward may write: two blocks of 256 threads per SM of the largest part.
constexpr int kNormMaxParts = 608;
size_t norm_ws_bytes(int64_t rows, int H) {
  const int64_t parts = rows < kNormMaxParts ? rows : kNormMaxParts;
  return size_t(parts < 1 ? 1 : parts) * 2 * size_t(H) * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool x_f32, cudaStream_t st) {
  return x_f32 ? norm_fwd_t<float>(a, st) : norm_fwd_t<__nv_bfloat16>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool x_f32, float* partial, cudaStream_t st) {
  int parts = 0;
  if (a.rows > 0) {
    const bool q8 = a.codes != nullptr;
    const cudaError_t e =
        x_f32 ? (q8 ? norm_bwd_t<float, true>(a, partial, kNormMaxParts, &parts, st)
                    : norm_bwd_t<float, false>(a, partial, kNormMaxParts, &parts, st))
              : (q8 ? norm_bwd_t<__nv_bfloat16, true>(a, partial, kNormMaxParts, &parts, st)
                    : norm_bwd_t<__nv_bfloat16, false>(a, partial, kNormMaxParts, &parts, st));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_weight_grad_kernel, dim3(unsigned((2 * a.H + 31) / 32)), dim3(256), 0, st,
                    static_cast<const float*>(partial), parts, a.H, a.w_f32, a.dgamma, a.dbeta);
}

}  // namespace moe
