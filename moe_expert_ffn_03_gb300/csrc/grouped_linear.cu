// Linear layers grouped by expert on dense ragged rows: forward, input gradient and weight
// gradient, bf16 operands on the tensor cores (tcgen05 kind::f16, f32 accumulation).
//
// Page "Efficient MoE Training for Biological Foundation Models", section "GroupedLinear：把
// 逐专家循环改成一次分组GEMM": the tokens collected per expert and split_sizes, one grouped
// call instead of a loop over the experts.  The rows of expert e follow those of expert e - 1
// without padding; split_sizes stays on the device.
//
//   forward   y[r]  = W_e x[r]               D[m][n]: m output features, n rows,     sum over K
//   dgrad     dx[r] = W_e^T dy[r]            D[m][n]: m input features,  n rows,     sum over N
//   wgrad     dW_e  = sum_r dy[r] x[r]^T     D[m][n]: m input features,  n outputs,  sum over rows
//
// The weights (and, in wgrad, x) are the M side of the MMA and the ragged rows the N side,
// whose extent an instruction can choose in steps of 32: a tile of s rows costs roundup(s, 32)
// columns instead of 128 or 256 rows, so one token per expert costs little more than reading
// the weights.  All three read their operands where they lie: K-major tiles where the sum runs
// along memory, MN-major tiles where it does not, so nothing is transposed or padded first.
// In every mode m is the contiguous index of the output.
//
// A stage of an operand is 128 x 128 values: K-major as two 64-deep steps of 128 rows, MN-major as
// two 64-wide blocks of 128 deep, each row 128 swizzled bytes.  Where the row lengths are
// multiples of 64 (ATOMS) one TMA box fetches it whole: what TMA delivers to an SM grows with the
// bytes of a copy.  Other lengths take two boxes, whose ends TMA fills with zeros.
//
// Persistent CTA pairs (clusters of two, one CTA per SM): a pair computes a 256 x 256 tile
// with tcgen05.mma.cta_group::2; each CTA stages its 128 m and its half of the n columns.
//   warp 0       TMA producer: stages of two 64-deep steps (64 KB of operands per CTA);
//   warp 1       TMEM allocation; in the leader, the MMAs; two 256-column accumulators;
//   warps 2..17  epilogue, four per TMEM lane quarter, 64 accumulator columns each;
//   warp 18      wgrad: clears the rows of a tile's last step that belong to the next expert.
// Every wait is bounded.
#include <atomic>
#include <cstdio>

#include "kernels.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int LG_M = 256, LG_N = 256;            // the pair's tile
constexpr int LG_KT = 64;                        // contraction per step: 128 bytes of a K-major row
constexpr int LG_PER = 2;                        // steps per barrier stage
constexpr int LG_NSTG = 3;                       // barrier stages
constexpr int LG_TILE = 128 * LG_KT * 2;         // bytes of one operand's step in one CTA
constexpr int LG_OPERAND = LG_PER * LG_TILE;     // of one operand's stage: 32 KB
constexpr int LG_STAGE = 2 * LG_OPERAND;
constexpr int LG_EPI_WARPS = 16;
constexpr int LG_THREADS = 32 * (3 + LG_EPI_WARPS);
constexpr int LG_MAX_E = 256;
constexpr int LG_GROUP = 8;                      // row tiles that share the sweep over the weights
constexpr int LG_SMALL = 32;                     // rows of the small row box

constexpr int LG_OFF_BAR = LG_NSTG * LG_STAGE;
// full[3], empty[3], tail[3], cleared[3], tmem_full[2], tmem_empty[2], drain
constexpr int LG_BARS = 4 * LG_NSTG + 5;
constexpr int LG_OFF_MISC = LG_OFF_BAR + LG_BARS * 8;
constexpr int LG_OFF_SEG = (LG_OFF_MISC + 16 + 15) & ~15;   // row0[E+1], tile0[E+1], order[E]
// Epilogue: per warp eight column pairs of 32 m, as words {column 2p, column 2p + 1} at a pitch of
// 36 words, so that both the writes (a word per lane) and the reads (16 bytes) are conflict-free.
constexpr int LG_TR_PITCH = 36;
constexpr int LG_OFF_TR = (LG_OFF_SEG + 3 * (LG_MAX_E + 1) * 4 + 15) & ~15;
constexpr int LG_TR_WARP = 8 * LG_TR_PITCH * 4;
constexpr int LG_SMEM = LG_OFF_TR + LG_EPI_WARPS * LG_TR_WARP + 1024;
static_assert(LG_SMEM <= 232448, "shared memory budget");

// kind::f16 instruction descriptor: bf16 x bf16 -> f32, M = 256, N columns; a_mn, b_mn: the
// operand is MN-major.
__device__ __forceinline__ uint32_t lg_idesc(bool a_mn, bool b_mn, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(LG_M >> 4) << 24);
}

// Arrival on an mbarrier of the cluster that makes this thread's earlier writes visible to the
// waiter, and the wait that observes it.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t caddr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_phase_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                                int site) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1; !mbar_try_wait_cluster(bar, parity); ++n) {
    if ((n & 31u) != 0) continue;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      report_error(err, MOE_ERR_DEVICE_TIMEOUT, site);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

struct LinTile {
  int e;
  int m0;          // first m of the pair's tile
  int n0, cnt;     // first n (row, or output feature in wgrad) and how many the tile has
  int n;           // MMA columns: cnt rounded up to 32 (wgrad: 128)
  int c0, c_cnt;   // contraction: first index and length
  int steps;       // ceil(c_cnt / 64)
};

template <int MODE>
__device__ __forceinline__ int lin_m(const LinearArgs& a) { return MODE == LIN_FWD ? a.N : a.K; }

template <int MODE>
__device__ __forceinline__ int lin_tiles(const LinearArgs& a, const int* tile0) {
  const int mt = (lin_m<MODE>(a) + LG_M - 1) / LG_M;
  if (MODE == LIN_WGRAD) return a.E * mt * ((a.N + LG_N - 1) / LG_N);
  return tile0[a.E] * mt;
}

template <int MODE>
__device__ __forceinline__ void lin_decode(const LinearArgs& a, const int* row0, const int* tile0, const int* order,
                                           int t, LinTile& tl) {
  const int mt = (lin_m<MODE>(a) + LG_M - 1) / LG_M;
  if (MODE == LIN_WGRAD) {
    // experts with the most rows first; inside an expert the m tiles of a few n tiles in turn
    const int nt = (a.N + LG_N - 1) / LG_N;
    const int slot = t / (mt * nt), rem = t - slot * (mt * nt);
    const int per = LG_GROUP * mt;
    const int g = rem / per, first = g * LG_GROUP, gs = min(LG_GROUP, nt - first);
    const int local = rem - g * per;
    tl.e = order[slot];
    tl.m0 = (local / gs) * LG_M;
    tl.n0 = (first + local % gs) * LG_N;
    tl.cnt = min(LG_N, a.N - tl.n0);
    tl.c0 = row0[tl.e];
    tl.c_cnt = row0[tl.e + 1] - tl.c0;
  } else {
    const int total = tile0[a.E];
    const int per = LG_GROUP * mt;
    const int g = t / per, first = g * LG_GROUP, gs = min(LG_GROUP, total - first);
    const int local = t - g * per;
    const int tt = first + local % gs;
    int lo = 0, hi = a.E - 1;                    // largest e with tile0[e] <= tt
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] <= tt) lo = mid; else hi = mid - 1;
    }
    tl.e = lo;
    tl.m0 = (local / gs) * LG_M;
    tl.n0 = row0[lo] + (tt - tile0[lo]) * LG_N;
    tl.cnt = min(LG_N, row0[lo + 1] - tl.n0);
    tl.c0 = 0;
    tl.c_cnt = MODE == LIN_FWD ? a.K : a.N;
  }
  // wgrad's columns come in 64-wide swizzle atoms per CTA, the rows of the others in 16s
  tl.n = MODE == LIN_WGRAD ? (tl.cnt + 127) & ~127 : (tl.cnt + 31) & ~31;
  tl.steps = (tl.c_cnt + LG_KT - 1) / LG_KT;
}

// A wgrad tile whose contraction does not end on a multiple of 16 rows: its last stage is
// cleared past the end by warp 18 of both CTAs before the MMAs read it.
template <int MODE>
__device__ __forceinline__ bool lin_tail(const LinTile& tl) { return MODE == LIN_WGRAD && (tl.c_cnt & 15) != 0; }

template <int MODE, bool ATOMS>
__global__ void __launch_bounds__(LG_THREADS, 1)
    grouped_linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmBs, const LinearArgs args) {
  constexpr bool A_MN = MODE != LIN_FWD, B_MN = MODE == LIN_WGRAD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LG_OFF_BAR);
  uint64_t* empty = full + LG_NSTG;
  uint64_t* tail = empty + LG_NSTG;              // this CTA's copies of a tail stage have landed
  uint64_t* cleared = tail + LG_NSTG;            // leader: both CTAs have cleared a tail stage
  uint64_t* tmem_full = cleared + LG_NSTG;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* drain = tmem_empty + 2;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + LG_OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + LG_OFF_MISC + 4);
  volatile int* bad_s = reinterpret_cast<volatile int*>(smem + LG_OFF_MISC + 8);
  int* row0 = reinterpret_cast<int*>(smem + LG_OFF_SEG);
  int* tile0 = row0 + LG_MAX_E + 1;
  int* order = tile0 + LG_MAX_E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();       // 0: leader (issues the MMAs), 1: peer
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < LG_NSTG; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&cleared[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], 2 * LG_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmBs);
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_s, 512);                // collectively with the peer CTA
    tmem_relinquish();
  }
  // Up to here the kernel touches only its own shared memory, TMEM and parameters.
  pdl_wait();
  if (warp == 2) {
    // prefix sums of the experts' rows and row tiles, eight experts per lane
    int rows[8], sum = 0, tiles = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      const int s = e < args.E ? args.split_sizes[e] : 0;
      bad |= s < 0 || s > args.rows;
      rows[i] = s < 0 || s > args.rows ? 0 : s;
    }
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += rows[i];
      all += rows[i];
      tiles += (rows[i] + LG_N - 1) / LG_N;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
    bad = __any_sync(0xFFFFFFFFu, bad) || all > args.rows;
    if (lane == 0) {
      *bad_s = bad;
      if (bad) report_error(args.err, MOE_ERR_DEVICE_BOUNDS, SITE_LINEAR + 9);
    }
    int rs = sum, ts = tiles;                    // inclusive scans over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int r = __shfl_up_sync(0xFFFFFFFFu, rs, off), q = __shfl_up_sync(0xFFFFFFFFu, ts, off);
      if (lane >= off) {
        rs += r;
        ts += q;
      }
    }
    rs -= sum;
    ts -= tiles;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      if (e <= args.E) {
        row0[e] = rs;
        tile0[e] = ts;
      }
      rs += rows[i];
      ts += (rows[i] + LG_N - 1) / LG_N;
    }
    if (lane == 31 && args.E == LG_MAX_E) {
      row0[LG_MAX_E] = rs;
      tile0[LG_MAX_E] = ts;
    }
    __syncwarp();
    if (MODE == LIN_WGRAD) {
      for (int e = lane; e < args.E; e += 32) {
        const int me = row0[e + 1] - row0[e];
        int r = 0;
        for (int f = 0; f < args.E; ++f) {
          const int other = row0[f + 1] - row0[f];
          r += (other > me) || (other == me && f < e);
        }
        order[r] = e;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                // the pair's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  // inconsistent split_sizes: nothing is computed (the error word says so)
  const int total = *bad_s ? 0 : lin_tiles<MODE>(args, tile0);

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      const uint32_t full_c0 = mapa_shared(smem_u32(full), 0);
      int it = 0;
      bool ok = true;
      int last_round[LG_NSTG];
#pragma unroll
      for (int s = 0; s < LG_NSTG; ++s) last_round[s] = -1;
      bool issued = false;
      for (int t = pair; t < total && ok; t += num_pairs) {
        LinTile tl;
        lin_decode<MODE>(args, row0, tile0, order, t, tl);
        const int half = tl.n >> 1;
        const int m = tl.m0 + int(rank) * 128;
        const int nr = tl.n0 + int(rank) * half;
        const bool small = !B_MN && half <= LG_SMALL;
        const uint32_t b_step = small ? LG_SMALL * 128u : uint32_t(LG_TILE);
        for (int kt0 = 0; kt0 < tl.steps; kt0 += LG_PER, ++it) {
          const int st = it % LG_NSTG, round = it / LG_NSTG;
          if (!wait_phase(&empty[st], (round & 1) ^ 1, abort_s, args.err, SITE_LINEAR, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const int nk = min(LG_PER, tl.steps - kt0);
          // both CTAs' copies complete on the leader's full barrier; those of a tail stage on each
          // CTA's tail barrier, since each clears its own rows (full then only advances its phase)
          const bool tl_stage = lin_tail<MODE>(tl) && kt0 + LG_PER >= tl.steps;
          uint32_t bar_c = full_c0 + uint32_t(st) * 8u;
          // K-major operands without ATOMS are fetched step by step, everything else whole
          const uint32_t bytes = (ATOMS || A_MN ? uint32_t(LG_OPERAND) : uint32_t(nk * LG_TILE)) +
                                 (ATOMS || B_MN ? LG_PER * b_step : uint32_t(nk) * b_step);
          if (tl_stage) {
            if (rank == 0) mbar_arrive_expect_tx(&full[st], 0);
            mbar_arrive_expect_tx(&tail[st], bytes);
            bar_c = mapa_shared(smem_u32(&tail[st]), rank);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(&full[st], 2u * bytes);
          }
          last_round[st] = round;
          issued = true;
          uint8_t* pa = smem + st * LG_STAGE;
          uint8_t* pb = pa + LG_OPERAND;
          const int c = tl.c0 + kt0 * LG_KT;
          if (ATOMS) {
            // {64 columns, 128 rows, 2 blocks of 64 columns(, expert)}
            if (MODE == LIN_FWD) tma_load_4d(pa, &tmA, 0, m, c >> 6, tl.e, bar_c);
            else if (MODE == LIN_DGRAD) tma_load_4d(pa, &tmA, 0, c, m >> 6, tl.e, bar_c);
            else tma_load_3d(pa, &tmA, 0, c, m >> 6, bar_c);
            if (B_MN) tma_load_3d(pb, &tmB, 0, c, nr >> 6, bar_c);
            else tma_load_3d(pb, small ? &tmBs : &tmB, 0, nr, c >> 6, bar_c);
          } else {
            if (MODE == LIN_FWD) {
              for (int s = 0; s < nk; ++s) tma_load_3d(pa + s * LG_TILE, &tmA, c + s * LG_KT, m, tl.e, bar_c);
            } else if (MODE == LIN_DGRAD) {
              for (int h = 0; h < 2; ++h) tma_load_3d(pa + h * LG_TILE, &tmA, m + h * 64, c, tl.e, bar_c);
            } else {
              for (int h = 0; h < 2; ++h) tma_load_2d(pa + h * LG_TILE, &tmA, m + h * 64, c, bar_c);
            }
            if (B_MN) {
              for (int h = 0; h < 2; ++h) tma_load_2d(pb + h * LG_TILE, &tmB, nr + h * 64, c, bar_c);
            } else {
              for (int s = 0; s < nk; ++s)
                tma_load_2d(pb + s * b_step, small ? &tmBs : &tmB, c + s * LG_KT, nr, bar_c);
            }
          }
        }
      }
      pdl_launch_dependents();
      if (!ok && issued) {
        // let copies already issued land before the CTA exits: the leader watches the full
        // barriers, then a fixed grace period for copies that signal elsewhere
        if (rank == 0) {
          for (int s = 0; s < LG_NSTG; ++s) {
            if (last_round[s] < 0) continue;
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&full[s], last_round[s] & 1) && globaltimer_ns() - t0 < 20000000ull) {
            }
          }
        }
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (leader) ----------------
      int it = 0, tcount = 0;
      uint32_t cleared_par = 0;                  // bit s: parity of the next tail phase of stage s
      bool ok = true, issued = false;
      for (int t = pair; t < total && ok; t += num_pairs, ++tcount) {
        LinTile tl;
        lin_decode<MODE>(args, row0, tile0, order, t, tl);
        const uint32_t idesc = lg_idesc(A_MN, B_MN, tl.n);
        const int ab = tcount & 1, use = tcount >> 1;
        const uint32_t acc = tmem + uint32_t(ab) * 256u;
        if (!wait_phase(&tmem_empty[ab], (use & 1) ^ 1, abort_s, args.err, SITE_LINEAR + 1, kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kt0 = 0; kt0 < tl.steps; kt0 += LG_PER, ++it) {
          const int st = it % LG_NSTG, round = it / LG_NSTG;
          const int nk = min(LG_PER, tl.steps - kt0);
          if (!wait_phase(&full[st], round & 1, abort_s, args.err, SITE_LINEAR + 2, kWaitLimitNs)) {
            ok = false;
            break;
          }
          if (lin_tail<MODE>(tl) && kt0 + LG_PER >= tl.steps) {
            if (!wait_phase_cluster(&cleared[st], (cleared_par >> st) & 1u, abort_s, args.err, SITE_LINEAR + 3)) {
              ok = false;
              break;
            }
            cleared_par ^= 1u << st;
          }
          tc_fence_after();
          const uint32_t pa = smem_u32(smem + st * LG_STAGE), pb = pa + LG_OPERAND;
          const uint64_t ad = A_MN ? desc_sw128_mn(pa, LG_TILE) : desc_sw128(pa);
          const uint64_t bd = B_MN ? desc_sw128_mn(pb, LG_TILE) : desc_sw128(pb);
          const uint32_t b_step = !B_MN && tl.n <= 2 * LG_SMALL ? LG_SMALL * 128u : uint32_t(LG_TILE);
          for (int s = 0; s < nk; ++s) {
            // 16 of the contraction, in the descriptors' 16-byte units: 32 bytes of a K-major row,
            // two 8-row groups (2 KB) of an MN-major block
            const uint64_t a0 = ad + uint64_t(s * ((A_MN ? 64 * 128 : LG_TILE) >> 4));
            const uint64_t b0 = bd + uint64_t(s * ((B_MN ? 64 * 128 : int(b_step)) >> 4));
            const int left = tl.c_cnt - (kt0 + s) * LG_KT;
            const int kk_n = left >= LG_KT ? LG_KT / 16 : (left + 15) / 16;
            for (int kk = 0; kk < kk_n; ++kk)
              tc_mma_bf16(acc, a0 + uint64_t((A_MN ? 128 : 2) * kk), b0 + uint64_t((B_MN ? 128 : 2) * kk), idesc,
                          (kt0 | s | kk) != 0);
          }
          issued = true;
          tc_commit(&empty[st]);                 // frees the stage in both CTAs
        }
        if (!ok) break;
        tc_commit(&tmem_full[ab]);
      }
      if (!ok && issued) {
        tc_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp < 2 + LG_EPI_WARPS) {
    // ---------------- epilogue warps (both CTAs) ----------------
    const int q = warp & 3;                      // TMEM lane quarter this warp may access
    const int cg = (warp - 2) >> 2;              // column group 0..3
    const uint32_t tmem_row = tmem + (uint32_t(q * 32) << 16) + uint32_t(cg * 64);
    const uint32_t tmem_empty_c0 = mapa_shared(smem_u32(tmem_empty), 0);
    const int M = lin_m<MODE>(args);
    uint32_t* tr = reinterpret_cast<uint32_t*>(smem + LG_OFF_TR + (warp - 2) * LG_TR_WARP);
    int tcount = 0;
    for (int t = pair; t < total; t += num_pairs, ++tcount) {
      LinTile tl;
      lin_decode<MODE>(args, row0, tile0, order, t, tl);
      const int ab = tcount & 1, use = tcount >> 1;
      if (!wait_phase(&tmem_full[ab], use & 1, abort_s, args.err, SITE_LINEAR + 4, kWaitLimitNs)) break;
      tc_fence_after();
      uint32_t r[64];
      if (cg * 64 < tl.cnt) {
        tmem_ld32_async(tmem_row + uint32_t(ab) * 256u, r);
        if (cg * 64 + 32 < tl.cnt) tmem_ld32_async(tmem_row + uint32_t(ab) * 256u + 32u, r + 32);
        tmem_wait_ld<64>(r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tmem_empty_c0 + uint32_t(ab) * 8u);
      // Lane l holds m = l of 64 columns.  Through shared memory, 16 columns at a time, a lane
      // gets eight m of two columns, p and p + 1: 16-byte stores, 64 bytes per column and warp.
      const int p = lane >> 2, m = tl.m0 + int(rank) * 128 + q * 32 + (lane & 3) * 8;
      const int64_t first = (MODE == LIN_WGRAD ? int64_t(tl.e) * args.N : 0) + tl.n0 + cg * 64;
      __nv_bfloat16* o = args.out + (first + 2 * p) * args.ldo + m;
      const bool zero = tl.steps == 0;           // wgrad of an expert without rows
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 16) {
        if (cg * 64 + c0 >= tl.cnt) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = pack_bf16x2(__uint_as_float(r[c0 + 2 * i]), __uint_as_float(r[c0 + 2 * i + 1]));
          tr[i * LG_TR_PITCH + lane] = zero ? 0u : w;
        }
        __syncwarp();
        const uint4* src = reinterpret_cast<const uint4*>(tr + p * LG_TR_PITCH + (lane & 3) * 8);
        const uint4 u = src[0], v = src[1];
        __syncwarp();
        const int left = tl.cnt - (cg * 64 + c0 + 2 * p);        // columns of the tile from this pair on
        __nv_bfloat16* oc = o + int64_t(c0) * args.ldo;
        if (m < M && left > 0)
          *reinterpret_cast<uint4*>(oc) = make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410),
                                                     __byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410));
        if (m < M && left > 1)
          *reinterpret_cast<uint4*>(oc + args.ldo) =
              make_uint4(__byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x7632), __byte_perm(v.x, v.y, 0x7632),
                         __byte_perm(v.z, v.w, 0x7632));
      }
    }
  } else if (MODE == LIN_WGRAD) {
    // ---------------- warp 18: rows of a tail stage past the expert's end (both CTAs) ----------------
    const uint32_t cleared_c0 = mapa_shared(smem_u32(cleared), 0);
    uint32_t par = 0;
    int it = 0;
    bool ok = true;
    for (int t = pair; t < total && ok; t += num_pairs) {
      LinTile tl;
      lin_decode<MODE>(args, row0, tile0, order, t, tl);
      const int stages = (tl.steps + LG_PER - 1) / LG_PER;
      if (lin_tail<MODE>(tl)) {
        // (a barrier is waited on in every one of its phases or not at all: skipping phases, this
        // warp would take an older phase of the same parity for the one it wants; so tail stages
        // have barriers of their own)
        const int st = (it + stages - 1) % LG_NSTG;
        ok = wait_phase(&tail[st], (par >> st) & 1u, abort_s, args.err, SITE_LINEAR + 5, kWaitLimitNs);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        par ^= 1u << st;
        const int valid = tl.c_cnt - (stages - 1) * LG_PER * LG_KT;   // the stage's rows
        const int upto = (valid + 15) & ~15;
        // 4 blocks (A's two of 64 columns, B's two) x rows x eight 16-byte chunks
        const int n = (upto - valid) * 8;
        for (int i = lane; i < 4 * n; i += 32) {
          const int block = i / n, j = i - block * n;
          const int row = valid + (j >> 3);
          *reinterpret_cast<uint4*>(smem + st * LG_STAGE + block * LG_TILE + row * 128 + (j & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async;" ::: "memory");          // visible to the MMAs' reads
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_release(cleared_c0 + uint32_t(st) * 8u);
      }
      it += stages;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                // no CTA leaves while the pair's MMAs or arrivals may touch it
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// bf16 map over row-major [batch][rows][inner] (batch 0: no such dimension) with 128-byte swizzle.
// atoms: the columns as {64, inner / 64} and a box of {64, box_rows, 2(, 1)}; else {64, box_rows(, 1)}.
bool lin_map(CUtensorMap* m, bool atoms, const void* base, int64_t inner, int64_t rows, int64_t ld, int64_t batch,
             int box_rows) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {cuuint64_t(atoms ? 64 : inner), cuuint64_t(rows)}, strides[3] = {cuuint64_t(ld) * 2};
  cuuint32_t box[4] = {64, cuuint32_t(box_rows), 1, 1}, estr[4] = {1, 1, 1, 1};
  int rank = 2;
  if (atoms) {
    strides[rank - 1] = 128;
    box[rank] = 2;
    dims[rank++] = cuuint64_t(inner / 64);
  }
  if (batch > 0) {
    strides[rank - 1] = cuuint64_t(ld) * cuuint64_t(rows) * 2;
    dims[rank++] = cuuint64_t(batch);
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool ATOMS>
cudaError_t lin_launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mbs, const LinearArgs& a,
                       int grid, cudaStream_t st) {
  // the shared-memory attribute is per device: set it once on each device this process uses
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(grouped_linear_kernel<MODE, ATOMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, LG_SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(LG_THREADS);
  cfg.dynamicSmemBytes = LG_SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // the kernel calls pdl_wait()
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_linear_kernel<MODE, ATOMS>, ma, mb, mbs, a);
}

}  // namespace

cudaError_t launch_grouped_linear(int mode, const LinearArgs& a, const void* x, int64_t ldx, const void* dy,
                                  int64_t lddy, const void* w, cudaStream_t st, char* msg, size_t msg_len) {
  CUtensorMap ma, mb, mbs;
  bool ok;
  const bool at = a.K % 64 == 0 && a.N % 64 == 0;
  if (mode == LIN_FWD) {
    ok = lin_map(&ma, at, w, a.K, a.N, a.K, a.E, 128) && lin_map(&mb, at, x, a.K, a.rows, ldx, 0, 128) &&
         lin_map(&mbs, at, x, a.K, a.rows, ldx, 0, LG_SMALL);
  } else if (mode == LIN_DGRAD) {
    ok = lin_map(&ma, at, w, a.K, a.N, a.K, a.E, 128) && lin_map(&mb, at, dy, a.N, a.rows, lddy, 0, 128) &&
         lin_map(&mbs, at, dy, a.N, a.rows, lddy, 0, LG_SMALL);
  } else {
    ok = lin_map(&ma, at, x, a.K, a.rows, ldx, 0, 128) && lin_map(&mb, at, dy, a.N, a.rows, lddy, 0, 128);
    mbs = mb;                                    // not used
  }
  if (!ok) {
    snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (rows %lld, K %d, N %d, E %d)", (long long)a.rows, a.K, a.N,
             a.E);
    return cudaErrorInvalidValue;
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // no more pairs than tiles there can be
  const int64_t mt = ((mode == LIN_FWD ? a.N : a.K) + LG_M - 1) / LG_M;
  const int64_t nt = mode == LIN_WGRAD ? int64_t(a.E) * ((a.N + LG_N - 1) / LG_N)
                                       : (a.rows < a.E ? a.rows : a.E) + a.rows / LG_N;
  const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
  const int grid = 2 * int(mt * nt < pairs ? mt * nt : pairs);
  switch (mode * 2 + int(at)) {
    case LIN_FWD * 2: return lin_launch<LIN_FWD, false>(ma, mb, mbs, a, grid, st);
    case LIN_FWD * 2 + 1: return lin_launch<LIN_FWD, true>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 2: return lin_launch<LIN_DGRAD, false>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 2 + 1: return lin_launch<LIN_DGRAD, true>(ma, mb, mbs, a, grid, st);
    case LIN_WGRAD * 2: return lin_launch<LIN_WGRAD, false>(ma, mb, mbs, a, grid, st);
    default: return lin_launch<LIN_WGRAD, true>(ma, mb, mbs, a, grid, st);
  }
}

}  // namespace moe
