// The router's balance loss with the experts' counts, its z loss, and their gradient.
//
// Page "英伟达开源MoE加速神器", section "三板斧" (tokens are routed to a few experts; a router that is not
// held to even loads leaves experts idle; the loss itself is an interface addition).  Over the n tokens that
// the mask leaves, with s = softmax(logits), c_e the choices of expert e and P_e the mean of s_e:
//   balance = E / (k n) * sum_e c_e P_e,   z = mean (log sum exp logits)^2,   loss = alpha balance + beta z
//   dlogits = (alpha s_e (f_e - sum_j f_j s_j) + 2 beta lse s_e) / n,   f_e = E c_e / (k n) - 1
// (the counts are constants; since the softmax sums to one, f may be counted from 1, where even loads do not
// cancel).  Small and bound by latency: one launch each way.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int BAL_THREADS = 512;
constexpr int BAL_WARPS = BAL_THREADS / 32;
constexpr int BAL_GROUP = 32;                    // blocks whose sums one of them adds
constexpr int BAL_UN = 4;                        // tokens a lane group has on their way at once

// Four neighbouring experts' logits from column c on; -Inf past the last.
template <bool WIDE>
__device__ __forceinline__ void load4(const float* row, int c, int E, float* x) {
  if constexpr (WIDE) {
    float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (c < E) q = __ldg(reinterpret_cast<const float4*>(row + c));
    x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = c + j < E ? __ldg(row + c + j) : -INFINITY;
  }
}

// A token's G lanes, each with 4 V of its logits: x -> the softmax, and log sum exp as the result.  A token
// all of whose logits are -Inf has no softmax: zeros, and 0.
template <int G, int V>
__device__ __forceinline__ float softmax(float (*x)[4]) {
  float m = x[0][0];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, x[v][j]);
#pragma unroll
  for (int off = 1; off < G; off *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  const bool none = m == -INFINITY;
  float z = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[v][j] = none && x[v][j] == -INFINITY ? 0.f : expf(x[v][j] - m);
      z += x[v][j];
    }
#pragma unroll
  for (int off = 1; off < G; off *= 2) z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
  if (z == 0.f) return 0.f;
  const float inv = __fdiv_rn(1.f, z);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[v][j] *= inv;
  return m + logf(z);
}

// A block's sums of the softmax, of the squared lse and its counts go to a row of `partial`
// [E sums | sum of squares | E counts | tokens].  Rows are added in order: where there are more than 32, by the block of
// every 32 that finishes last, then their sums by the last of those.  (Both measured, that one first, then all rows by the
// last block of all: 16384 tokens, 256 experts 17.2 and 23.6 us; 32768 tokens, 64 experts 11.7 and 12.2.)
// 32768 tokens, 64 experts, forward and backward in turn: 19 us both ways, by 15 and 9 us a cold launch.
template <int G, int V, bool WIDE>
__global__ void __launch_bounds__(BAL_THREADS) balance_fwd_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ uint32_t sh[];               // [warps][E + 1] f32, then [E + 1] counts
  __shared__ bool last_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & (G - 1);
  const int E = a.E, W = 2 * (E + 1);
  float* wsum = reinterpret_cast<float*>(sh);
  int* hist = reinterpret_cast<int*>(sh + BAL_WARPS * (E + 1));
  for (int e = tid; e <= E; e += BAL_THREADS) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  float acc[V][4], zz = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[v][j] = 0.f;
  int tokens = 0;
  constexpr int PER = 32 / G;                    // tokens a warp works on side by side
  const int64_t step = int64_t(gridDim.x) * BAL_WARPS * PER * BAL_UN;
  // whole warps go round together: a lane past the last token, or at a masked one, adds nothing
  for (int64_t t0 = (int64_t(blockIdx.x) * BAL_WARPS + warp) * PER * BAL_UN + lane / G; t0 - lane / G < a.T; t0 += step) {
    float x[BAL_UN][V][4];
    bool live[BAL_UN];
    int choice[BAL_UN];
#pragma unroll
    for (int u = 0; u < BAL_UN; ++u) {
      const int64_t t = t0 + u * PER;
      const bool in = t < a.T;
      live[u] = in && (a.mask == nullptr || a.mask[t] != 0);
      choice[u] = in && sub < a.k ? a.idx[t * a.k + sub] : 0;
#pragma unroll
      for (int v = 0; v < V; ++v) load4<WIDE>(a.logits + (in ? t : 0) * E, in ? (v * G + sub) * 4 : E, E, x[u][v]);
    }
#pragma unroll
    for (int u = 0; u < BAL_UN; ++u) {
      const float lse = softmax<G, V>(x[u]);
      if (!live[u]) continue;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[v][j] += x[u][v][j];
      for (int j = sub; j < a.k; j += G) {
        const int e = j == sub ? choice[u] : a.idx[(t0 + u * PER) * a.k + j];
        if (e < 0 || e >= E) report_error(a.err, MOE_ERR_DEVICE_BOUNDS, SITE_BALANCE);
        else atomicAdd(hist + e, 1);
      }
      if (sub == 0) {
        zz = fmaf(lse, lse, zz);
        ++tokens;
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int off = G; off < 32; off *= 2) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[v][j] += __shfl_xor_sync(0xFFFFFFFFu, acc[v][j], off);
    zz += __shfl_xor_sync(0xFFFFFFFFu, zz, off);
  }
  if (lane < G) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((v * G + sub) * 4 + j < E) wsum[warp * (E + 1) + (v * G + sub) * 4 + j] = acc[v][j];
  }
  if (lane == 0) wsum[warp * (E + 1) + E] = zz;
  if (tokens != 0) atomicAdd(hist + E, tokens);
  __syncthreads();
  const auto block_sum = [&](int e) {
    float v = 0.f;
    for (int w = 0; w < BAL_WARPS; ++w) v += wsum[w * (E + 1) + e];
    return v;
  };
  if (gridDim.x == 1) {                          // few tokens: all sums are at hand
    for (int e = tid; e <= E; e += BAL_THREADS) {
      wsum[e] = block_sum(e);                    // (column e of warp 0's, which nobody else reads)
      a.counts[e] = hist[e];
    }
  } else {
    // whether this block is the last of n; the ticket is back at zero for the next call
    const auto last_of = [&](unsigned* ticket, unsigned n) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        last_s = atomicAdd(ticket, 1u) + 1 == n;
        if (last_s) *ticket = 0;
      }
      __syncthreads();
      if (last_s) __threadfence();
      return last_s;
    };
    // n rows' columns, each `stride` rows behind the one before
    const auto add_rows = [&](int first, int n, int stride, auto done) {
      for (int c = tid; c < W; c += BAL_THREADS) {
        const uint32_t* p = a.partial + int64_t(first) * W + c;
        float sum = 0.f;
        int count = 0;
#pragma unroll 2
        for (int r0 = 0; r0 < n; r0 += 8) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = r0 + i < n ? __ldcg(p + int64_t(r0 + i) * stride * W) : 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (c <= E) sum += __uint_as_float(v[i]);
            else count += int(v[i]);
          }
        }
        done(c, sum, count);
      }
    };
    uint32_t* mine = a.partial + int64_t(blockIdx.x) * W;
    for (int e = tid; e <= E; e += BAL_THREADS) {
      __stcg(mine + e, __float_as_uint(block_sum(e)));
      __stcg(mine + E + 1 + e, uint32_t(hist[e]));
    }
    int rows = int(gridDim.x), stride = 1;
    if (rows > BAL_GROUP) {
      const int group = int(blockIdx.x) / BAL_GROUP, first = group * BAL_GROUP, n = min(BAL_GROUP, rows - first);
      if (!last_of(a.ticket + 1 + group, unsigned(n))) return;
      uint32_t* sum_of = a.partial + int64_t(first) * W;         // in the place of its first block's
      add_rows(first, n, 1, [&](int c, float v, int k) { __stcg(sum_of + c, c <= E ? __float_as_uint(v) : uint32_t(k)); });
      rows = (rows + BAL_GROUP - 1) / BAL_GROUP;
      stride = BAL_GROUP;
    }
    if (!last_of(a.ticket, unsigned(rows))) return;
    add_rows(0, rows, stride, [&](int c, float v, int k) {
      if (c <= E) {
        wsum[c] = v;
      } else {
        hist[c - E - 1] = k;
        a.counts[c - E - 1] = k;
      }
    });
  }
  __syncthreads();
  if (warp != 0) return;
  const float n = float(hist[E] > 0 ? hist[E] : 1);
  float dot = 0.f;
  for (int e = lane; e < E; e += 32) {
    const float p = __fdiv_rn(wsum[e], n);
    a.prob[e] = p;
    dot = fmaf(float(hist[e]), p, dot);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
  if (lane == 0) {
    const float balance = __fdiv_rn(dot * float(E), float(a.k) * n), z = __fdiv_rn(wsum[E], n);
    a.loss[0] = fmaf(a.alpha, balance, a.beta * z);
    a.loss[1] = balance;
    a.loss[2] = z;
  }
}

template <int G, int V, bool WIDE>
__global__ void __launch_bounds__(BAL_THREADS) balance_bwd_kernel(const __grid_constant__ BalanceArgs a) {
  __shared__ float load_s[4 * 32 * 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (G - 1);
  const int E = a.E;
  pdl_wait();
  const int64_t n = a.counts[E] > 0 ? a.counts[E] : 1;
  // alpha f, from whole numbers: E c - k n has no rounding that even loads would be left with
  for (int e = threadIdx.x; e < 4 * 32 * 2; e += BAL_THREADS)
    load_s[e] = e < E ? a.alpha * __fdiv_rn(float(int64_t(E) * a.counts[e] - a.k * n), float(a.k * n)) : 0.f;
  __syncthreads();
  float f[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) f[v][j] = load_s[(v * G + sub) * 4 + j];
  const float g = __fdiv_rn(a.grad != nullptr ? *a.grad : 1.f, float(n));
  constexpr int PER = 32 / G;
  const int64_t step = int64_t(gridDim.x) * BAL_WARPS * PER * BAL_UN;
  for (int64_t t0 = (int64_t(blockIdx.x) * BAL_WARPS + warp) * PER * BAL_UN + lane / G; t0 - lane / G < a.T; t0 += step) {
    float x[BAL_UN][V][4];
    bool live[BAL_UN];
#pragma unroll
    for (int u = 0; u < BAL_UN; ++u) {
      const int64_t t = t0 + u * PER;
      const bool in = t < a.T;
      live[u] = in && (a.mask == nullptr || a.mask[t] != 0);
#pragma unroll
      for (int v = 0; v < V; ++v) load4<WIDE>(a.logits + (in ? t : 0) * E, in ? (v * G + sub) * 4 : E, E, x[u][v]);
    }
#pragma unroll
    for (int u = 0; u < BAL_UN; ++u) {
      const int64_t t = t0 + u * PER;
      const float lse = softmax<G, V>(x[u]);
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(f[v][j], x[u][v][j], dot);
#pragma unroll
      for (int off = 1; off < G; off *= 2) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
      if (t >= a.T) continue;
      const float base = 2.f * a.beta * lse - dot;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * G + sub) * 4;
        float d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = live[u] ? g * x[u][v][j] * (f[v][j] + base) : 0.f;
        float* o = a.dlogits + t * E + c;
        if constexpr (WIDE) {
          if (c < E) *reinterpret_cast<float4*>(o) = make_float4(d[0], d[1], d[2], d[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < E) o[j] = d[j];
        }
      }
    }
  }
}

template <int G, int V, bool WIDE>
cudaError_t balance_run(const BalanceArgs& a, bool backward, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  constexpr int64_t TOKENS = BAL_WARPS * (32 / G) * BAL_UN;       // of a block's round
  const int64_t need = (a.T + TOKENS - 1) / TOKENS;
  if (backward) {
    const int64_t most = int64_t(sms) * 4;
    return launch_pdl(balance_bwd_kernel<G, V, WIDE>, dim3(unsigned(need < most ? need : most)), dim3(BAL_THREADS), 0, st, a);
  }
  static_assert(1 + (kBalanceMaxParts + BAL_GROUP - 1) / BAL_GROUP <= 56, "tickets lie in the workspace's first 256 bytes, from word 8 on");
  const int64_t most = 2 * sms < kBalanceMaxParts ? 2 * sms : kBalanceMaxParts;     // two blocks an SM
  const size_t smem = size_t(BAL_WARPS + 1) * (a.E + 1) * 4;                 // at most 18 KB
  return launch_pdl(balance_fwd_kernel<G, V, WIDE>, dim3(unsigned(need < most ? need : most)), dim3(BAL_THREADS), smem, st, a);
}

template <bool WIDE>
cudaError_t balance_lanes(const BalanceArgs& a, bool backward, cudaStream_t st) {
  const int fours = (a.E + 3) / 4;               // as few lanes a token as hold its logits, four each
  if (fours <= 1) return balance_run<1, 1, WIDE>(a, backward, st);
  if (fours <= 2) return balance_run<2, 1, WIDE>(a, backward, st);
  if (fours <= 4) return balance_run<4, 1, WIDE>(a, backward, st);
  if (fours <= 8) return balance_run<8, 1, WIDE>(a, backward, st);
  if (fours <= 16) return balance_run<16, 1, WIDE>(a, backward, st);
  if (fours <= 32) return balance_run<32, 1, WIDE>(a, backward, st);
  return balance_run<32, 2, WIDE>(a, backward, st);
}

}  // namespace

size_t balance_ws_bytes(int E) { return 256 + size_t(kBalanceMaxParts) * 2 * (E + 1) * 4; }

cudaError_t launch_balance(const BalanceArgs& a, bool backward, cudaStream_t st) {
  return a.E % 4 == 0 ? balance_lanes<true>(a, backward, st) : balance_lanes<false>(a, backward, st);
}

}  // namespace moe
