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
// Where a row's sum or squares would leave float32's range, the row is worked on times a power of two,
// which changes no quotient: every finite row has the norm of its definition.
// Each activation is read once and written once; wide rows are held by the instructions per vector
// and their latency at 16 warps an SM before they are held by memory.
#include <cfloat>

#include "norm.cuh"

namespace moe {
namespace {

// The mean of a row from its sum: s / H to one rounding (the remainder of s * (1 / H) is added
// back), so that a constant row whose sum is exact has an exact mean.
__device__ __forceinline__ float mean_of(float s, float H, float inv_H) {
  const float q = s * inv_H;
  return fmaf(fmaf(-q, H, s), inv_H, q);
}
// Factors for rows whose variance (with eps) is above float32's range or below 2^-120.  LARGE on the row
// as it came: values below 2^48, squares whose sum stays below 2^112, and as long as the row is not
// constant a variance above 2^-60.  SMALL on the centred values, which are below 2^-53 then: their
// squares are normal numbers down to the smallest subnormal value's.
constexpr float LARGE = 0x1p-80f, SMALL = 0x1p100f;
__device__ __forceinline__ bool in_range(float var) { return var >= 0x1p-120f && var <= FLT_MAX; }

// The rows of this thread's row group whose variance (with eps) is above float32's range or below 2^-120,
// once more, on times a power of two.  A loop of its own behind the kernel's: with these rows' work in
// that loop, in line or called, all others took 3 to 13% longer.  Everything is read again from memory.
// Where h has taken the place of x or the residual by then, the row is h as stored; in bf16 its variance
// is not quite the sum's, so that rows near the bounds are taken along.
template <typename T, int VEC, int NV>
__device__ __noinline__ void norm_fwd_rescaled(const NormArgs& a, int tpr, float* buf0, float* buf1, float* buf2) {
  const Place<VEC, NV, 2, 0> at(tpr, nullptr);
  const float inv_H = 1.f / float(a.H);
  const bool summed = a.h != nullptr && (a.h == a.x || a.h == a.residual);
  const T* x = static_cast<const T*>(summed ? a.h : a.x);
  const T* res = static_cast<const T*>(summed ? nullptr : a.residual);
  float h[NV][VEC], w[VEC], sum[VEC];
  const auto total = [&](float* buf) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += sum[j];
    row_sum<1>(s, tpr, at.group, buf);
    return s[0];
  };
  // h = the row times f, and its sum per thread
  const auto load = [&](int64_t row, float f) {
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
      v_add<VEC>(sum, h[i]);
    }
  };
  // h = (h - mu) * f, and its squares' sum per thread
  const auto centre = [&](float mu, float f) {
    v_fill<VEC>(w, f);
    v_fill<VEC>(sum, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float minus[VEC];
      v_fill<VEC>(minus, at.col(i) < a.H ? -mu : 0.f);
      v_add<VEC>(h[i], minus);
      v_mul<VEC>(h[i], w);
      v_fma<VEC>(sum, h[i], h[i]);
    }
  };
  for (int64_t row = int64_t(blockIdx.x) * at.groups + at.group; row < a.rows; row += int64_t(gridDim.x) * at.groups) {
    load(row, 1.f);
    float mean = mean_of(total(buf0), float(a.H), inv_H);
    centre(mean, 1.f);
    const float var = total(buf1) * inv_H + a.eps;
    if (summed ? var >= 0x1p-119f && var <= 0x1p127f : in_range(var)) continue;
    float f = SMALL;
    if (!(var < 1.f)) {
      f = LARGE;
      load(row, LARGE);
      const float s = total(buf2), mu = fabsf(s) <= FLT_MAX ? mean_of(s, float(a.H), inv_H) : s;
      mean = mu * (1.f / LARGE);
      centre(mu, 1.f);
    } else {
      centre(0.f, SMALL);
    }
    const float squares = total(f == LARGE ? buf1 : buf2);
    float rstd = inv_sqrt(squares * inv_H + a.eps * f * f);        // of the row as it is held
    if (at.t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = squares == 0.f ? inv_sqrt(a.eps) : rstd * f;
    }
    if (squares == 0.f && a.eps > 0.f) rstd = 0.f;                 // eps * f * f may have gone under
    T* y = static_cast<T*>(a.y) + row * a.ld_out + at.col0;
    uint8_t* codes = a.codes + row * a.H + at.col0;
    uint8_t* scales = a.scales + row * ((a.H + 31) >> 5) + (at.col0 >> 5);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = at.col(i) < a.H;
      v_fill<VEC>(w, rstd);
      v_mul<VEC>(h[i], w);
      if (a.codes != nullptr)
        store_act8<VEC>(h[i], in, codes + i * (32 * VEC), scales + i * VEC, (at.col0 & 31) == 0);
      if (!in) continue;
      float b[VEC];
      v_fill<VEC>(b, 0.f);
      load_weight<VEC>(a.gamma, a.w_f32, at.col(i), w);
      if (a.beta != nullptr) load_weight<VEC>(a.beta, a.w_f32, at.col(i), b);
      v_fma<VEC>(b, h[i], w);
      store_vec<VEC>(y + i * (32 * VEC), b);
    }
  }
}

// A persistent grid: block b takes the row groups b, b + grid, ...  The next groups' x (and
// residual) are on their way to shared memory while the current one is summed, so the two
// sums of a row (mean, then the variance of the centred values) cost no memory time.
// 32768 x 2048 bf16 with residual and checkpoint: 100 us, 6.1 TB/s.  Single columns are bound by their
// narrow loads (8192 x 5001: 2.0 TB/s).
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(max_block(VEC), 1) norm_fwd_kernel(const __grid_constant__ NormArgs a, int tpr) {
  constexpr int STG = ring_stages(VEC, 2 * NV);
  __shared__ float sums[3][32];
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
  if constexpr (VEC > 1) at.clear();
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * at.groups + at.group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  const Weight<VEC, NV> gamma(a.gamma, a.w_f32, at.col0, a.H), beta(a.beta, a.w_f32, at.col0, a.H);
  int st = 0;
  bool odd = false;                               // the same in all of a row group's threads
  for (; row < a.rows; row += step) {             // the rows' groups go on independently of one another
    if constexpr (VEC > 1) {
      fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
      cp_async_wait<STG - 1>();
    }
    float h[NV][VEC], sum[VEC];
    v_fill<VEC>(sum, 0.f);
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
        // unconditional loads (column 0 past the row's end), so that a row's are all in flight at once
        const bool in = at.col(i) < a.H;
        const int64_t off = row * a.ld_in + (in ? at.col(i) : 0);
        Raw<T, 1> x, r;
        x.load(static_cast<const T*>(a.x) + off);
        r.zero();
        if (has_res) r.load(static_cast<const T*>(a.residual) + off);
        x.get(h[i]);
        r.get(v);
        h[i][0] = in ? h[i][0] + v[0] : 0.f;
      }
      v_add<VEC>(sum, h[i]);
    }
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += sum[j];
    row_sum<1>(s, tpr, at.group, sums[0]);
    const float mu = mean_of(s[0], float(a.H), inv_H);
    if (a.h != nullptr) {
      T* ho = static_cast<T*>(a.h) + row * a.ld_out + at.col0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (at.col(i) < a.H) store_vec<VEC>(ho + i * (32 * VEC), h[i]);
    }
    float minus[VEC], sq[VEC];
    v_fill<VEC>(sq, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v_fill<VEC>(minus, at.col(i) < a.H ? -mu : 0.f);
      v_add<VEC>(h[i], minus);
      v_fma<VEC>(sq, h[i], h[i]);
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += sq[j];
    row_sum<1>(s, tpr, at.group, sums[1]);
    const float var = s[0] * inv_H + a.eps, rstd = inv_sqrt(var);
    odd |= !in_range(var);
    if (at.t == 0) {
      if (a.mean != nullptr) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ld_out + at.col0;
    uint8_t* codes = a.codes + row * a.H + at.col0;
    uint8_t* scales = a.scales + row * ((a.H + 31) >> 5) + (at.col0 >> 5);
    float rs[VEC];
    v_fill<VEC>(rs, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = at.col(i) < a.H;
      v_mul<VEC>(h[i], rs);
      if (a.codes != nullptr)
        store_act8<VEC>(h[i], in, codes + i * (32 * VEC), scales + i * VEC, (at.col0 & 31) == 0);
      if (in) {
        float g[VEC], b[VEC];
        gamma.get(i, g);
        beta.get(i, b);
        v_fma<VEC>(b, h[i], g);
        store_vec<VEC>(y + i * (32 * VEC), b);
      }
    }
  }
  if (odd) norm_fwd_rescaled<T, VEC, NV>(a, tpr, sums[0], sums[1], sums[2]);
}

// A persistent grid and a ring as in the forward pass.  A thread keeps its columns' sums of
// dgamma and dbeta in registers; at the end the block's groups are added in order and written
// as one partial sum per block, which norm_weight_grad_kernel adds in block order.  The second
// pass over a row finds it in registers where a thread has up to 16 columns (single columns always),
// and reads the ring again where it has more.  32768 x 2048 bf16 from the checkpoint, with dres,
// weights' gradients included: 99 us, 4.8 TB/s, bound by 219 instructions a vector at half the issue
// rate (single columns, 8192 x 5001: 0.7 TB/s).
template <typename T, int VEC, int NV, bool Q8>
__global__ void __launch_bounds__(max_block(VEC), 1) norm_bwd_kernel(const NormArgs a, int tpr, float* partial) {
  constexpr int STG = ring_stages(VEC, 3 * NV);
  constexpr bool HOLD = VEC * NV <= 16;
  __shared__ float sums[2][64];
  extern __shared__ __align__(16) uint8_t ring[]; // operands dy, dres, kept rows
  const Place<VEC, NV, 3, STG> at(tpr, ring);
  const int nb = (a.H + 31) >> 5;
  const int64_t step = int64_t(gridDim.x) * at.groups;
  const bool has_res = a.dres != nullptr;
  const auto fetch = [&](int64_t row, int st) {
    if constexpr (VEC > 1) {
      if (row < a.rows) {
        const int64_t off = row * a.ld_in + at.col0;
        const T* dy = static_cast<const T*>(a.dy) + off;
        const T* res = static_cast<const T*>(a.dres) + off;
        const T* x = static_cast<const T*>(a.x) + off;
        const uint8_t* codes = a.codes + row * a.H + at.col0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (at.col(i) < a.H) {
            const int d = i * (32 * VEC);
            ring_copy<16>(at.piece(st, 0, i), dy + d);
            if constexpr (Q8) ring_copy<VEC>(at.piece(st, 2, i), codes + d);
            else ring_copy<16>(at.piece(st, 2, i), x + d);
            if (has_res) ring_copy<16>(at.piece(st, 1, i), res + d);
          }
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
    for (int i = 0; i < NV; ++i) m.c[i] = Q8 && live && at.col(i) < a.H ? a.scales[row * nb + (at.col(i) >> 5)] : 0;
    return m;
  };
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v_fill<VEC>(dg[i], 0.f);
    v_fill<VEC>(db[i], 0.f);
  }
  const float inv_H = 1.f / float(a.H);
  int flip = 0, st = 0;
  if constexpr (VEC > 1) at.clear();
  pdl_wait();
  int64_t row = int64_t(blockIdx.x) * at.groups + at.group;
#pragma unroll
  for (int k = 0; k + 1 < STG; ++k) fetch(row + k * step, k);
  const Weight<VEC, NV> gamma(a.gamma, a.w_f32, at.col0, a.H);
  Small next = fetch_small(row);
  for (; row < a.rows; row += step, flip ^= 1) {
    const Small m = next;
    if constexpr (VEC > 1) fetch(row + (STG - 1) * step, st == 0 ? STG - 1 : st - 1);
    next = fetch_small(row + step);
    // n from halves where x - mean could overflow (x is below 2^128, and a mean up to 2^100 does not move it)
    const bool halve = !Q8 && fabsf(m.mu) > 0x1p100f;
    const float minus_mu = halve ? -0.5f * m.mu : -m.mu, scale = halve ? 2.f * m.rstd : m.rstd;
    if constexpr (VEC > 1) cp_async_wait<STG - 1>();
    // dy and the normalised values (0 past the row's end) of vector i
    const auto get = [&](int i, float* d, float* n) {
      const bool in = at.col(i) < a.H;
      if constexpr (VEC > 1) {
        ring_get<T>(at.piece(st, 0, i), d);
        if constexpr (Q8) {
          Act8<VEC> q;
          const uint32_t* p = reinterpret_cast<const uint32_t*>(at.piece(st, 2, i));
          q.q[0] = p[0];
          if constexpr (VEC == 8) q.q[1] = p[1];
          q.c = m.c[i];
          q.get(n);
        } else {
          ring_get<T>(at.piece(st, 2, i), n);
        }
      } else {
        // unconditional loads, as in the forward pass
        const int col = in ? at.col(i) : 0;
        Raw<T, 1> r;
        r.load(static_cast<const T*>(a.dy) + row * a.ld_in + col);
        r.get(d);
        if constexpr (Q8) {
          Act8<1> q;
          q.q[0] = a.codes[row * a.H + col];
          q.c = m.c[i];
          q.get(n);
        } else {
          r.load(static_cast<const T*>(a.x) + row * a.ld_in + col);
          r.get(n);
        }
        d[0] = in ? d[0] : 0.f;
        n[0] = in ? n[0] : 0.f;
      }
      if constexpr (!Q8) {
        float minus[VEC], rs[VEC];
        if (halve) {
          v_fill<VEC>(rs, 0.5f);
          v_mul<VEC>(n, rs);
        }
        v_fill<VEC>(minus, in ? minus_mu : 0.f);
        v_fill<VEC>(rs, scale);
        v_add<VEC>(n, minus);
        v_mul<VEC>(n, rs);
      }
    };
    float s1[VEC], s2[VEC];
    float kn[HOLD ? NV : 1][VEC], kd[HOLD ? NV : 1][VEC];         // n and d * gamma, for the second pass
    v_fill<VEC>(s1, 0.f);
    v_fill<VEC>(s2, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&n)[VEC] = kn[HOLD ? i : 0], (&d)[VEC] = kd[HOLD ? i : 0], g[VEC];
      get(i, d, n);
      v_fill<VEC>(g, 0.f);
      if (at.col(i) < a.H) gamma.get(i, g);
      v_fma<VEC>(dg[i], d, n);
      v_add<VEC>(db[i], d);
      v_mul<VEC>(d, g);
      v_add<VEC>(s1, d);
      v_fma<VEC>(s2, d, n);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      s[0] += s1[j];
      s[1] += s2[j];
    }
    row_sum<2>(s, tpr, at.group, sums[flip]);
    // dx = rstd (d - m1 - n m2) + dres
    float m1[VEC], m2[VEC], rs[VEC];
    v_fill<VEC>(m1, -(s[0] * inv_H));
    v_fill<VEC>(m2, -(s[1] * inv_H));
    v_fill<VEC>(rs, m.rstd);
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
        } else {
          Raw<T, 1> r;
          r.load(static_cast<const T*>(a.dres) + row * a.ld_in + at.col0 + i * 32);
          r.get(v);
        }
      }
      v_add<VEC>(d, m1);
      v_fma<VEC>(d, n, m2);
      v_fma<VEC>(v, d, rs);
      store_vec<VEC>(dx + i * (32 * VEC), v);
    }
    if constexpr (VEC > 1) st = st + 1 == STG ? 0 : st + 1;
  }
  // The block's row groups, added in order: every group's sums to shared memory (the ring is
  // free by now), then all threads add columns.
  float* fold = reinterpret_cast<float*>(ring);   // [group][2][H]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = at.col(i);
    if (col >= a.H) continue;
    float* f = fold + size_t(at.group) * 2 * a.H + col;
#pragma unroll
    for (int j = 0; j < VEC; j += VEC > 1 ? 4 : 1) {
      if constexpr (VEC > 1) {
        *reinterpret_cast<float4*>(f + j) = make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
        *reinterpret_cast<float4*>(f + a.H + j) = make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
      } else {
        f[0] = dg[i][0];
        f[a.H] = db[i][0];
      }
    }
  }
  __syncthreads();
  pdl_launch_dependents();
  for (int c = threadIdx.x; c < 2 * a.H; c += blockDim.x) {
    float sum = fold[c];
    for (int g = 1; g < at.groups; ++g) sum += fold[size_t(g) * 2 * a.H + c];
    partial[int64_t(blockIdx.x) * 2 * a.H + c] = sum;
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
#pragma unroll 5
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

template <typename T, int VEC, int NV>
cudaError_t norm_fwd_shape(const NormArgs& a, const RowShape& s, cudaStream_t st) {
  static Resident known;
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  const size_t smem = size_t(ring_stages(VEC, 2 * NV)) * 2 * NV * 16 * s.block;
  int64_t most = 0;
  if (const cudaError_t e = resident_blocks(norm_fwd_kernel<T, VEC, NV>, s, smem, known, &most); e != cudaSuccess) return e;
  return launch_pdl(norm_fwd_kernel<T, VEC, NV>, dim3(unsigned(need < most ? need : most)), dim3(unsigned(s.block)),
                    smem, st, a, s.tpr);
}

template <typename T, int VEC, int NV, bool Q8>
cudaError_t norm_bwd_shape(const NormArgs& a, const RowShape& s, float* partial, int* parts, cudaStream_t st) {
  static Resident known;
  const int64_t rpb = s.block / s.tpr, need = (a.rows + rpb - 1) / rpb;
  const size_t ring = size_t(ring_stages(VEC, 3 * NV)) * 3 * NV * 16 * s.block;
  const size_t fold = size_t(rpb) * 2 * a.H * sizeof(float);      // H <= tpr * VEC * NV: at most 128 KB
  const size_t smem = ring > fold ? ring : fold;
  int64_t grid = 0;
  if (const cudaError_t e = resident_blocks(norm_bwd_kernel<T, VEC, NV, Q8>, s, smem, known, &grid); e != cudaSuccess) return e;
  grid = grid < kNormMaxParts ? grid : kNormMaxParts;
  grid = grid < need ? grid : need;
  *parts = int(grid);
  return launch_pdl(norm_bwd_kernel<T, VEC, NV, Q8>, dim3(unsigned(grid)), dim3(unsigned(s.block)), smem, st, a, s.tpr,
                    partial);
}

template <typename T>
RowShape shape_of(const NormArgs& a, int wide_nv) {
  return row_shape(a.H, a.H % 8 == 0 && a.ld_in % 8 == 0 && a.ld_out % 8 == 0 ? kWide<T> : 1, wide_nv);
}

template <typename T>
cudaError_t norm_fwd_t(const NormArgs& a, cudaStream_t st) {
  const RowShape s = shape_of<T>(a, 4);
  return with_shape<T>(s, [&](auto vec, auto nv) { return norm_fwd_shape<T, vec.value, nv.value>(a, s, st); });
}

template <typename T, bool Q8>
cudaError_t norm_bwd_t(const NormArgs& a, float* partial, int* parts, cudaStream_t st) {
  const RowShape s = shape_of<T>(a, sizeof(T) == 2 ? 2 : 4);
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
