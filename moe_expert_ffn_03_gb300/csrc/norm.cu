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
#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "rows.cuh"

namespace moe {
namespace {

// A row has at most 512 threads.  Blocks of that size an SM is to hold: two where a thread has few
// columns (VEC * NV), else one.
constexpr int MAX_TPR = 512;
constexpr int min_blocks(int vec, int nv) { return vec * nv <= 8 ? 2 : 1; }
// Rows a block has on their way or in work at once (VEC > 1): up to three, as the 16-byte pieces
// of all resident blocks fit in shared memory (`pieces` per thread and row).
constexpr int ring_stages(int vec, int nv, int pieces) {
  if (vec == 1) return 0;
  const int most = 200 * 1024 / (min_blocks(vec, nv) * MAX_TPR * pieces * 16);
  return most > 3 ? 3 : most;
}

// A persistent grid: block b takes the row groups b, b + grid, ...  The next groups' x (and
// residual) are on their way to shared memory while the current one is summed, so the two
// barriers of a row (mean, then the variance of the centred values) cost no memory time.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(MAX_TPR, min_blocks(VEC, NV)) norm_fwd_kernel(const NormArgs a, int tpr) {
  constexpr int STG = ring_stages(VEC, NV, 2 * NV);
  __shared__ float sums[2][32];
  extern __shared__ __align__(16) uint8_t ring[]; // [stage][x, residual][vector][thread] of 16 bytes
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int pitch = int(blockDim.x) * 16;
  const float inv_H = 1.f / float(a.H);
  const int64_t step = int64_t(gridDim.x) * groups;
  const auto piece = [&](int st, int op, int i) {
    return ring + ((st * 2 + op) * NV + i) * pitch + threadIdx.x * 16;
  };
  const auto fetch = [&](int64_t row, int st) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * VEC;
        const bool in = row < a.rows && col < a.H;
        const int64_t at = in ? row * a.ld_in + col : 0;
        ring_copy<16>(piece(st, 0, i), static_cast<const T*>(a.x) + at, in);
        if (a.residual != nullptr) ring_copy<16>(piece(st, 1, i), static_cast<const T*>(a.residual) + at, in);
      }
      cp_async_commit();
    }
  };
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * groups + group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  int st = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * groups; row0 < a.rows; row0 += step, row += step) {
    const bool live = row < a.rows;
    if constexpr (VEC > 1) {
      fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
      cp_async_wait<STG - 1>();
    }
    float h[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = 0.f;
      if constexpr (VEC > 1) {
        ring_get<T>(piece(st, 0, i), h[i]);
        if (a.residual != nullptr) ring_get<T>(piece(st, 1, i), v);
      } else {
        const int col = i * tpr + t;
        Raw<T, 1> x, r;
        x.zero();
        r.zero();
        if (live && col < a.H) {
          x.load(static_cast<const T*>(a.x) + row * a.ld_in + col);
          if (a.residual != nullptr) r.load(static_cast<const T*>(a.residual) + row * a.ld_in + col);
        }
        x.get(h[i]);
        r.get(v);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[i][j] += v[j];
        s[0] += h[i][j];
      }
    }
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
    row_sum<1>(s, tpr, sums[0]);
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
  if constexpr (VEC > 1) cp_async_wait<0>();     // rows past the end bring zeros, but they are still copies
}

// A persistent grid and a ring as in the forward pass.  A thread keeps its columns' sums of
// dgamma and dbeta in registers; at the end the block's groups are added in order and written
// as one partial sum per block, which norm_weight_grad_kernel adds in block order.  The second
// pass over a row reads the ring again rather than hold the row in registers.
template <typename T, int VEC, int NV, bool Q8>
__global__ void __launch_bounds__(MAX_TPR, min_blocks(VEC, NV))
    norm_bwd_kernel(const NormArgs a, int tpr, float* partial) {
  constexpr int STG = ring_stages(VEC, NV, 3 * NV);
  __shared__ float sums[2][64];
  extern __shared__ __align__(16) uint8_t ring[]; // [stage][dy, dres, kept][vector][thread] of 16 bytes
  const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int pitch = int(blockDim.x) * 16;
  const int nb = (a.H + 31) >> 5;
  const int64_t step = int64_t(gridDim.x) * groups;
  const auto piece = [&](int st, int op, int i) {
    return ring + ((st * 3 + op) * NV + i) * pitch + threadIdx.x * 16;
  };
  const auto fetch = [&](int64_t row, int st) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * VEC;
        const bool in = row < a.rows && col < a.H;
        const int64_t at = in ? row * a.ld_in + col : 0;
        ring_copy<16>(piece(st, 0, i), static_cast<const T*>(a.dy) + at, in);
        if constexpr (Q8) ring_copy<VEC>(piece(st, 2, i), a.codes + (in ? row * a.H + col : 0), in);
        else ring_copy<16>(piece(st, 2, i), static_cast<const T*>(a.x) + at, in);
        if (a.dres != nullptr) ring_copy<16>(piece(st, 1, i), static_cast<const T*>(a.dres) + at, in);
      }
      cp_async_commit();
    }
  };
  // per row: mean, rstd and the scale codes of this thread's vectors, one row ahead in registers
  struct Small {
    float mu, rstd;
    uint32_t c[NV];
  };
  const auto fetch_small = [&](int64_t row) {
    Small m;
    const bool live = row < a.rows;
    m.mu = !Q8 && live ? a.mean[row] : 0.f;
    m.rstd = live ? a.rstd[row] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * VEC;
      m.c[i] = Q8 && live && col < a.H ? a.scales[row * nb + (col >> 5)] : 0;
    }
    return m;
  };
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  const float inv_H = 1.f / float(a.H);
  int flip = 0, st = 0;
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * groups + group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  Small next = fetch_small(row);
  for (int64_t row0 = int64_t(blockIdx.x) * groups; row0 < a.rows; row0 += step, row += step, flip ^= 1) {
    const bool live = row < a.rows;
    const Small m = next;
    if constexpr (VEC > 1) fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
    next = fetch_small(row + step);
    if constexpr (VEC > 1) cp_async_wait<STG - 1>();
    // dy and the normalised values (0 past the row's end) of vector i
    const auto get = [&](int i, float* d, float* n) {
      const int col = (i * tpr + t) * VEC;
      const bool in = live && col < a.H;
      if constexpr (VEC > 1) {
        ring_get<T>(piece(st, 0, i), d);
        if constexpr (Q8) {
          Act8<VEC> q;
          q.q[0] = reinterpret_cast<const uint32_t*>(piece(st, 2, i))[0];
          if constexpr (VEC == 8) q.q[1] = reinterpret_cast<const uint32_t*>(piece(st, 2, i))[1];
          q.c = m.c[i];
          q.get(n);
        } else {
          ring_get<T>(piece(st, 2, i), n);
        }
      } else {
        Raw<T, 1> r, x;
        r.zero();
        x.zero();
        if (in) r.load(static_cast<const T*>(a.dy) + row * a.ld_in + col);
        r.get(d);
        if constexpr (Q8) {
          Act8<1> q;
          q.q[0] = in ? a.codes[row * a.H + col] : 0;
          q.c = m.c[i];
          q.get(n);
        } else {
          if (in) x.load(static_cast<const T*>(a.x) + row * a.ld_in + col);
          x.get(n);
        }
      }
      if constexpr (!Q8)
#pragma unroll
        for (int j = 0; j < VEC; ++j) n[j] = in ? (n[j] - m.mu) * m.rstd : 0.f;
    };
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * VEC;
      float n[VEC], d[VEC], g[VEC];
      get(i, d, n);
#pragma unroll
      for (int j = 0; j < VEC; ++j) g[j] = 0.f;
      if (col < a.H) load_weight<VEC>(a.gamma, a.w_f32, col, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dg[i][j] += d[j] * n[j];
        db[i][j] += d[j];
        const float w = d[j] * g[j];
        s[0] += w;
        s[1] += w * n[j];
      }
    }
    row_sum<2>(s, tpr, sums[flip]);
    const float m1 = s[0] * inv_H, m2 = s[1] * inv_H;
    if (live) {
      T* dx = static_cast<T*>(a.dx) + row * a.ld_out;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + t) * VEC;
        if (col >= a.H) continue;
        float n[VEC], d[VEC], g[VEC], v[VEC];
        get(i, d, n);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = 0.f;
        if (a.dres != nullptr) {
          if constexpr (VEC > 1) {
            ring_get<T>(piece(st, 1, i), v);
          } else {
            Raw<T, 1> r;
            r.load(static_cast<const T*>(a.dres) + row * a.ld_in + col);
            r.get(v);
          }
        }
        load_weight<VEC>(a.gamma, a.w_f32, col, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += m.rstd * (d[j] * g[j] - m1 - n[j] * m2);
        store_vec<VEC>(dx + col, v);
      }
    }
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
  }
  if constexpr (VEC > 1) cp_async_wait<0>();
  // the block's row groups, added in order (the ring's memory is free by now)
  float* fold = reinterpret_cast<float*>(ring);   // [2][H]
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
  pdl_launch_dependents();
  if (group == 0) {
    float* p = partial + int64_t(blockIdx.x) * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * tpr + t) * VEC;
      if (col >= a.H) continue;
#pragma unroll
      for (int j = 0; j < VEC; j += VEC > 1 ? 4 : 1) {
        if constexpr (VEC > 1) {
          *reinterpret_cast<float4*>(p + col + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
          *reinterpret_cast<float4*>(p + a.H + col + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
        } else {
          p[col] = dg[i][0];
          p[a.H + col] = db[i][0];
        }
      }
    }
  }
}

// dgamma and dbeta from the blocks' partial sums [parts][2][H]: 32 columns per block, 32 warps
// each add every 32nd part, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* __restrict__ partial, int parts, int H,
                                                               bool w_f32, void* dgamma, void* dbeta) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;         // 0 .. 2H-1: dgamma, then dbeta
  pdl_wait();
  float s = 0.f;
  if (col < 2 * H) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) s += partial[int64_t(p) * 2 * H + col];
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= 2 * H) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += acc[w][lane];
  void* out = col < H ? dgamma : dbeta;
  if (out == nullptr) return;
  const int c = col < H ? col : col - H;
  if (w_f32) static_cast<float*>(out)[c] = s;
  else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
}

constexpr int kMaxDevices = 64;

struct RowShape {
  int vec;       // columns of a vector
  int nv;        // vectors per thread
  int tpr;       // threads per row
  int block;     // threads per block
};

// Threads and vectors per row: as few vectors a thread as 512 threads allow (wide) or at least 8
// (single columns, where nothing else keeps loads in flight).
RowShape row_shape(int H, int vec) {
  RowShape s{vec, vec > 1 ? 1 : 8, 32, 256};
  const int n = (H + vec - 1) / vec;              // vectors of a row
  while (s.nv * MAX_TPR < n) s.nv *= 2;
  while (s.tpr * s.nv < n) s.tpr *= 2;
  s.block = s.tpr > 256 ? s.tpr : 256;
  return s;
}

bool vec_ok(const NormArgs& a) { return a.H % 8 == 0 && a.ld_in % 8 == 0 && a.ld_out % 8 == 0; }

// Sets a kernel's dynamic shared memory limit once per device, and says how many blocks of a
// persistent grid the device holds at once (0: look-up failed).
template <typename K>
int64_t resident_blocks(K* kernel, int block, size_t smem, std::atomic<bool>* set) {
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (smem > 40 * 1024 && (dev >= kMaxDevices || !set[dev].load(std::memory_order_acquire))) {
    // above the 48 KB (static memory included) that need no asking; one call serves all sizes
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess) return 0;
    if (dev < kMaxDevices) set[dev].store(true, std::memory_order_release);
  }
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, block, smem) != cudaSuccess || per < 1)
    return 0;
  return int64_t(sms) * per;
}

template <typename T, int VEC, int NV>
cudaError_t norm_fwd_shape(const NormArgs& a, const RowShape& s, cudaStream_t st) {
  static std::atomic<bool> set[kMaxDevices];
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  const size_t smem = size_t(ring_stages(VEC, NV, 2 * NV)) * 2 * NV * 16 * s.block;
  const int64_t most = resident_blocks(norm_fwd_kernel<T, VEC, NV>, s.block, smem, set);
  if (most == 0) return cudaErrorInvalidConfiguration;
  return launch_pdl(norm_fwd_kernel<T, VEC, NV>, dim3(unsigned(need < most ? need : most)), dim3(unsigned(s.block)),
                    smem, st, a, s.tpr);
}

// Partial sums the backward may write: four blocks of 256 threads per SM.
constexpr int kNormMaxParts = 608;

template <typename T, int VEC, int NV, bool Q8>
cudaError_t norm_bwd_shape(const NormArgs& a, const RowShape& s, float* partial, int* parts, cudaStream_t st) {
  static std::atomic<bool> set[kMaxDevices];
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  size_t smem = size_t(ring_stages(VEC, NV, 3 * NV)) * 3 * NV * 16 * s.block;
  if (rpb > 1 && smem < size_t(2) * a.H * sizeof(float)) smem = size_t(2) * a.H * sizeof(float);  // H <= 1024 here
  int64_t grid = resident_blocks(norm_bwd_kernel<T, VEC, NV, Q8>, s.block, smem, set);
  if (grid == 0) return cudaErrorInvalidConfiguration;
  grid = grid < kNormMaxParts ? grid : kNormMaxParts;
  grid = grid < need ? grid : need;
  *parts = int(grid);
  return launch_pdl(norm_bwd_kernel<T, VEC, NV, Q8>, dim3(unsigned(grid)), dim3(unsigned(s.block)), smem, st, a, s.tpr,
                    partial);
}

// Calls f with the vector width and count of a row shape as compile-time constants.
template <typename T, typename F>
cudaError_t with_shape(const RowShape& s, F f) {
  constexpr int W = kWide<T>;
  if (s.vec == 1) {
    if (s.nv == 8) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
    if (s.nv == 16) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
  }
  if (s.nv == 1) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 1>{});
  if (s.nv == 2) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 2>{});
  if (s.nv == 4) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 4>{});
  if constexpr (W == 4) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 8>{});
  return cudaErrorInvalidConfiguration;           // H above 16384
}

template <typename T>
RowShape shape_of(const NormArgs& a) {
  return row_shape(a.H, a.H % 8 == 0 && a.ld_in % 8 == 0 && a.ld_out % 8 == 0 ? kWide<T> : 1);
}

template <typename T>
cudaError_t norm_fwd_t(const NormArgs& a, cudaStream_t st) {
  const RowShape s = shape_of<T>(a);
  return with_shape<T>(s, [&](auto vec, auto nv) { return norm_fwd_shape<T, vec.value, nv.value>(a, s, st); });
}

template <typename T, bool Q8>
cudaError_t norm_bwd_t(const NormArgs& a, float* partial, int* parts, cudaStream_t st) {
  const RowShape s = shape_of<T>(a);
  return with_shape<T>(s, [&](auto vec, auto nv) { return norm_bwd_shape<T, vec.value, nv.value, Q8>(a, s, partial, parts, st); });
}

}  // namespace

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
    const cudaError_t e = x_f32 ? (q8 ? norm_bwd_t<float, true>(a, partial, &parts, st)
                                      : norm_bwd_t<float, false>(a, partial, &parts, st))
                                : (q8 ? norm_bwd_t<__nv_bfloat16, true>(a, partial, &parts, st)
                                      : norm_bwd_t<__nv_bfloat16, false>(a, partial, &parts, st));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_weight_grad_kernel, dim3(unsigned((2 * a.H + 31) / 32)), dim3(1024), 0, st,
                    static_cast<const float*>(partial), parts, a.H, a.w_f32, a.dgamma, a.dbeta);
}

}  // namespace moe
