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
// Persistent CTA pairs (clusters of two, one CTA per SM): a pair computes a tile of 256 m and up to
// tn n (64, 128, 256 or 512) with tcgen05.mma.cta_group::2; each CTA stages its 128 m and its half
// of the n.  What bounds the main loop of large tiles is the bytes a step needs against the ring's
// bytes in flight: 512 columns need 48 B per clock and SM at the full MMA rate, 256 columns 64 B,
// and TMA delivers about 50.  The 512 columns of TMEM are two accumulators of 256, handed out in
// turn: a wide tile takes both, a narrow one leaves the other to the next tile.  A wide tile
// starts on its first accumulator while the epilogue still reads the second.
//   warp 0       TMA producer of the M side, warp 19 of the N side: one 64-deep step per stage, as
//                many stages as 192 KB hold (9 of 64 columns, 8 of 128, 6 of 256, 4 of 512);
//   warp 1       TMEM allocation; in the leader, the MMAs;
//   warps 2..17  epilogue, four per TMEM lane quarter, a quarter of the columns each;
//   warp 18      wgrad: clears the rows of a tile's last step that belong to the next expert.
// A stage's operands are blocks of 128 bytes per row, swizzled: K-major 128 (m or n) rows of 64
// deep, MN-major 64 deep rows of 64 (m or n).  MN-major operands whose rows are multiples of 64
// (ATOMS) come two blocks to a TMA box, others one by one so that TMA fills the end with zeros.
// Few rows and few tiles (CUT): the call is bound by reading the weights, and the last round of
// whole tiles would leave pairs idle.  Where twice its tiles or more fit the pairs, its tiles are
// cut along the contraction into as many equal pieces as fit.  The pieces of one place in the
// contraction run side by side, so that the weights are still read in long stretches (shares cut
// without regard to that read them 12% slower, measured).  The warp that finishes a tile's last
// piece adds the f32 partial sums from the workspace in the order of the contraction, so
// results do not depend on timing; nobody waits for anybody.  A kernel of its own: the code that
// puts pieces together costs the others' main loops 2 to 5% by being there.
// Every wait is bounded.  The epilogue's wait for an accumulator lasts as long as a tile's contraction,
// warp 18's for a tail stage as long as all tiles without one before it, and in wgrad both have no upper
// limit but the number of rows (2^30 rows on one pair take seconds).  So their limit starts anew with
// every stage that the producer finds free again: they give up when nothing moves.
//
// Many rows are bound by the tensor pipe under the power limit: 32768 rows, K = 4096, N = 28672, E = 8,
// forward 4573 us, dgrad 4595, wgrad 4495 (1.68, 1.67, 1.71 PFLOP/s); 196608 rows, 2048 -> 2816, E = 64:
// 1383, 1392, 1578 us (1.64, 1.63, 1.44); other cards take up to 9% longer.  Few rows are bound by the
// weights: 16 rows, 4096 -> 28672, six of eight experts used, 247 us, 5.7 TB/s.
#include <atomic>
#include <cstdio>

#include "kernels.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int LG_M = 256;                        // the pair's tile: m
constexpr int LG_ACC = 256;                      // columns of an accumulator
constexpr int LG_KT = 64;                        // contraction per stage
constexpr int LG_MAX_STG = 9;
constexpr int LG_TILE = 128 * LG_KT * 2;         // 128 m or n of a stage: 16 KB
constexpr int LG_BLOCK = LG_TILE / 2;            // one MN-major block
constexpr int LG_RING = 192 * 1024;
constexpr int LG_LEAD = 3;                       // stages a wide tile's first accumulator may run ahead
constexpr int LG_EPI_WARPS = 16;
constexpr int LG_THREADS = 32 * (4 + LG_EPI_WARPS);
constexpr int LG_MAX_E = 256;
constexpr int LG_GROUP = 8;                      // row tiles that share the sweep over the weights
constexpr int LG_SMALL = 32;                     // rows of the small box of rows
constexpr int LG_MIN_PIECE = 8;                  // steps a piece of a tile has at least
constexpr int LG_PIECE = 16 * 32;                // f32 of a warp's partial sums: 16 columns of 32 m
constexpr int LG_PLACES = 32;                    // warps that share a tile of 64 columns: 2 CTAs x 16

constexpr int LG_OFF_BAR = LG_RING;
// full, empty, tail, cleared [LG_MAX_STG] each, tmem_full[2], tmem_empty[2], drain
constexpr int LG_BARS = 4 * LG_MAX_STG + 5;

// Bytes of a stage's N side in one CTA, and the stages of a ring, for tiles of tn columns.
__host__ __device__ __forceinline__ int lin_b_bytes(int tn) { return tn / 2 * 128; }
__host__ __device__ __forceinline__ int lin_stages(int tn) { return LG_RING / (LG_TILE + lin_b_bytes(tn)); }
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
                                                int site, uint64_t limit_ns) {
  uint64_t t0 = 0;                               // as wait_phase
  for (uint32_t n = 1; !mbar_try_wait_cluster(bar, parity); ++n) {
    if ((n & 255u) != 0) continue;
    if (*abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit_ns) {
      report_error(err, MOE_ERR_DEVICE_TIMEOUT, site);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// wait_phase_warp for waits across many stages: limit_ns without a change of *stages_used.  In line, since
// the epilogue's wait is on a short call's path (wgrad of 64 rows over 64 experts 102.8 -> 99.6 us).
__device__ __forceinline__ bool wait_phase_warp_moving(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                       int* err, int site, uint64_t limit_ns,
                                                       const volatile uint32_t* stages_used) {
  uint64_t t0 = 0;
  uint32_t seen = 0;
  bool ok = true;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if ((n & 255u) != 0) continue;
    if (*abort_flag) {
      ok = false;
      break;
    }
    const uint64_t now = globaltimer_ns();
    const uint32_t used = *stages_used;
    if (t0 == 0 || used != seen) {
      t0 = now;
      seen = used;
    } else if (now - t0 > limit_ns) {
      report_error(err, MOE_ERR_DEVICE_TIMEOUT, site);
      *abort_flag = 1;
      ok = false;
      break;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A place in the ring: stage and the parity of its current phase.
struct Cursor {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// One tcgen05.mma (bf16, f32 accumulation) from descriptors given as their two halves: all
// descriptors of a kernel differ in the low half only.
__device__ __forceinline__ void lg_mma(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}"
      ::"r"(d), "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct LinTile {
  int e;
  int m0;          // first m of the pair's tile
  int n0, cnt;     // first n (row, or output feature in wgrad) and how many the tile has
  int n;           // MMA columns: cnt rounded up to 32 (wgrad: 128); CTA r holds n0 + r * n/2 ..
  int c0, c_cnt;   // contraction: first index and length
  int all;         // its 64-deep steps: ceil(c_cnt / 64)
  int k0, steps;   // those of this piece of the tile: first, number
  int part, parts; // the piece's place among the tile's pieces
  int cut;         // the tile's place among those cut
  // accumulators of the tile, and columns of accumulator h: each CTA's first 128 n, then the rest
  __device__ __forceinline__ int accs() const { return n > LG_ACC ? 2 : 1; }
  __device__ __forceinline__ int cols(int h) const { return h == 0 ? (n > LG_ACC ? LG_ACC : n) : n - LG_ACC; }
};

template <int MODE>
__device__ __forceinline__ int lin_m(const LinearArgs& a) { return MODE == LIN_FWD ? a.N : a.K; }

template <int MODE>
__device__ __forceinline__ int lin_tiles(const LinearArgs& a, const int* tile0) {
  const int mt = (lin_m<MODE>(a) + LG_M - 1) / LG_M;
  if (MODE == LIN_WGRAD) return a.E * mt * ((a.N + a.tn - 1) / a.tn);
  return tile0[a.E] * mt;
}

template <int MODE>
__device__ __forceinline__ void lin_decode(const LinearArgs& a, const int* row0, const int* tile0, const int* order,
                                           int t, LinTile& tl) {
  const int mt = (lin_m<MODE>(a) + LG_M - 1) / LG_M;
  if (MODE == LIN_WGRAD) {
    // experts with the most rows first; inside an expert the m tiles of a few n tiles in turn
    const int nt = (a.N + a.tn - 1) / a.tn;
    const int slot = t / (mt * nt), rem = t - slot * (mt * nt);
    const int per = LG_GROUP * mt;
    const int g = rem / per, first = g * LG_GROUP, gs = min(LG_GROUP, nt - first);
    const int local = rem - g * per;
    tl.e = order[slot];
    tl.m0 = (local / gs) * LG_M;
    tl.n0 = (first + local % gs) * a.tn;
    tl.cnt = min(a.tn, a.N - tl.n0);
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
    tl.n0 = row0[lo] + (tt - tile0[lo]) * a.tn;
    tl.cnt = min(a.tn, row0[lo + 1] - tl.n0);
    tl.c0 = 0;
    tl.c_cnt = MODE == LIN_FWD ? a.K : a.N;
  }
  // wgrad's columns come in 64-wide swizzle atoms per CTA, the rows of the others in 16s
  tl.n = MODE == LIN_WGRAD ? (tl.cnt + 127) & ~127 : (tl.cnt + 31) & ~31;
  tl.all = (tl.c_cnt + LG_KT - 1) / LG_KT;
  tl.k0 = 0;
  tl.steps = tl.all;
  tl.part = 0;
  tl.parts = 1;
  tl.cut = 0;
}

// The pieces of work of a pair: every num_pairs-th of the tiles taken whole, then at most one
// piece of the `rest` tiles that are cut into `parts` each.
struct Plan {
  int whole, rest, parts;
};
template <int MODE, bool CUT>
__device__ __forceinline__ Plan lin_plan(const LinearArgs& a, int total, int num_pairs) {
  Plan p{total, 0, 1};
  if (!CUT) return p;
  const int all = ((MODE == LIN_FWD ? a.K : a.N) + LG_KT - 1) / LG_KT;
  const int rest = total % num_pairs;
  const int parts = rest == 0 ? 1 : min(num_pairs / rest, all / LG_MIN_PIECE);
  if (parts < 2) return p;
  return Plan{total - rest, rest, parts};
}
// The next of the pair's pieces; t: its next tile, from pair on.
template <int MODE, bool CUT>
__device__ __forceinline__ bool lin_next(const LinearArgs& a, const int* row0, const int* tile0, const int* order,
                                         const Plan& p, int pair, int num_pairs, int& t, LinTile& tl) {
  if (t < p.whole) {
    lin_decode<MODE>(a, row0, tile0, order, t, tl);
    if (MODE == LIN_WGRAD) {
      // there and back: tiles come longest first, so the pair that got the longest of one round gets
      // the shortest of the next
      const int at = t % num_pairs;
      t += 2 * (num_pairs - 1 - at) + 1;
    } else {
      t += num_pairs;
    }
    return true;
  }
  if (!CUT || t >= p.whole + num_pairs || pair >= p.rest * p.parts) return false;
  t += num_pairs;
  const int cut = pair % p.rest, part = pair / p.rest;
  lin_decode<MODE>(a, row0, tile0, order, p.whole + cut, tl);
  tl.cut = cut;
  tl.part = part;
  tl.parts = p.parts;
  tl.k0 = part * tl.all / p.parts;
  tl.steps = (part + 1) * tl.all / p.parts - tl.k0;
  return true;
}

// A wgrad tile whose contraction does not end on a multiple of 16 rows: its last stage is
// cleared past the end by warp 18 of both CTAs before the MMAs read it.
template <int MODE>
__device__ __forceinline__ bool lin_tail(const LinTile& tl) { return MODE == LIN_WGRAD && (tl.c_cnt & 15) != 0; }

// A warp's 32 m x 16 columns of a piece of a tile (tn = 64): written to the workspace, unless this
// is the last of the tile's pieces to arrive here; then r becomes the sum of all of them, in the
// order of the contraction, and the caller stores it (true).  place: the warp's among the tile's
// 32 (CTA, lane quarter, column group).
__device__ __forceinline__ bool join_pieces(const LinearArgs& a, const LinTile& tl, int rest, int place, int lane,
                                            uint32_t* r) {
  const auto slot = [&](int part) {              // piece `part` of cut tile c is pair part * rest + c's
    return a.pieces + (int64_t(part * rest + tl.cut) * LG_PLACES + place) * LG_PIECE + lane;
  };
  float* mine = slot(tl.part);
#pragma unroll
  for (int c = 0; c < 16; ++c) __stcg(mine + c * 32, __uint_as_float(r[c]));
  __threadfence();
  __syncwarp();
  unsigned* arrived = a.arrived + tl.cut * LG_PLACES + place;
  unsigned before = 0;
  if (lane == 0) before = atomicAdd(arrived, 1u);
  before = __shfl_sync(0xFFFFFFFFu, before, 0);
  if (before + 1 != unsigned(tl.parts)) return false;
  __threadfence();
  if (lane == 0) *arrived = 0;                   // for the next call
  const float* first = slot(0);
#pragma unroll
  for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__ldcg(first + c * 32));
  for (int p = 1; p < tl.parts; ++p) {
    const float* s = slot(p);
#pragma unroll
    for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) + __ldcg(s + c * 32));
  }
  return true;
}

template <int MODE, bool ATOMS, bool CUT>
__global__ void __launch_bounds__(LG_THREADS, 1)
    grouped_linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmBs, const LinearArgs args) {
  constexpr bool A_MN = MODE != LIN_FWD, B_MN = MODE == LIN_WGRAD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LG_OFF_BAR);
  uint64_t* empty = full + LG_MAX_STG;
  uint64_t* tail = empty + LG_MAX_STG;              // this CTA's copies of a tail stage have landed
  uint64_t* cleared = tail + LG_MAX_STG;            // leader: both CTAs have cleared a tail stage
  uint64_t* tmem_full = cleared + LG_MAX_STG;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* drain = tmem_empty + 2;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + LG_OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + LG_OFF_MISC + 4);
  volatile int* bad_s = reinterpret_cast<volatile int*>(smem + LG_OFF_MISC + 8);
  volatile uint32_t* stages_used = reinterpret_cast<volatile uint32_t*>(smem + LG_OFF_MISC + 12);
  int* row0 = reinterpret_cast<int*>(smem + LG_OFF_SEG);
  int* tile0 = row0 + LG_MAX_E + 1;
  int* order = tile0 + LG_MAX_E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();       // 0: leader (issues the MMAs), 1: peer
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const int stages = lin_stages(args.tn), stage_bytes = LG_TILE + lin_b_bytes(args.tn);

  if (threadIdx.x == 0) {
    for (int s = 0; s < LG_MAX_STG; ++s) {
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
    *stages_used = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmBs);
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_s, 512);                // collectively with the peer CTA
    tmem_relinquish();
  }
  cluster_arrive();                              // this CTA's barriers are initialised
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
      tiles += (rows[i] + args.tn - 1) / args.tn;
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
      ts += (rows[i] + args.tn - 1) / args.tn;
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
  cluster_wait();                                // and the other's, before anything arrives there
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  // inconsistent split_sizes: nothing is computed (the error word says so)
  const int total = *bad_s ? 0 : lin_tiles<MODE>(args, tile0);
  const Plan plan = lin_plan<MODE, CUT>(args, total, num_pairs);
  const uint64_t lim = args.wait_limit_ns;

  if (warp == 0 || warp == 19) {
    if (lane == 0 && !args.selftest_no_loads) {
      // ---------------- TMA producers (both CTAs): warp 0 the M side, warp 19 the N side ----------------
      const bool m_side = warp == 0;
      const uint32_t full_c0 = mapa_shared(smem_u32(full), 0);
      Cursor cur;
      uint32_t used = 0;
      bool ok = true;
      int next = pair;
      for (LinTile tl; ok && lin_next<MODE, CUT>(args, row0, tile0, order, plan, pair, num_pairs, next, tl);) {
        const int half = tl.n >> 1;
        const int m = tl.m0 + int(rank) * 128;
        const int nr = tl.n0 + int(rank) * half;
        const bool small = half <= (B_MN ? 64 : LG_SMALL);       // one MN-major block, or few rows
        const int nb = half > 128 ? 2 : 1;       // 128-wide parts of the N side
        const uint32_t bytes = LG_TILE + (small ? uint32_t(B_MN ? LG_BLOCK : LG_SMALL * 128) : uint32_t(nb * LG_TILE));
        for (int kt = 0; kt < tl.steps; ++kt, cur.next(stages)) {
          if (!wait_phase(&empty[cur.st], cur.ph ^ 1u, abort_s, args.err, SITE_LINEAR, lim)) {
            ok = false;
            break;
          }
          if (MODE == LIN_WGRAD && m_side) *stages_used = ++used;
          // both CTAs' copies complete on the leader's full barrier; those of a tail stage on each
          // CTA's tail barrier, since each clears its own rows (full then only advances its phase)
          uint32_t bar_c = full_c0 + uint32_t(cur.st) * 8u;
          if (lin_tail<MODE>(tl) && kt + 1 == tl.steps) {
            bar_c = mapa_shared(smem_u32(&tail[cur.st]), rank);
            if (m_side) {
              if (rank == 0) mbar_arrive_expect_tx(&full[cur.st], 0);
              mbar_arrive_expect_tx(&tail[cur.st], bytes);
            }
          } else if (m_side && rank == 0) {
            mbar_arrive_expect_tx(&full[cur.st], 2u * bytes);
          }
          uint8_t* pa = smem + cur.st * stage_bytes;
          uint8_t* pb = pa + LG_TILE;
          const int c = tl.c0 + (tl.k0 + kt) * LG_KT;
          if (m_side) {
            if (MODE == LIN_FWD) {
              tma_load_3d(pa, &tmA, c, m, tl.e, bar_c);
            } else if (ATOMS) {
              if (MODE == LIN_DGRAD) tma_load_4d(pa, &tmA, 0, c, m >> 6, tl.e, bar_c);
              else tma_load_3d(pa, &tmA, 0, c, m >> 6, bar_c);
            } else {
              for (int k = 0; k < 2; ++k) {
                if (MODE == LIN_DGRAD) tma_load_3d(pa + k * LG_BLOCK, &tmA, m + k * 64, c, tl.e, bar_c);
                else tma_load_2d(pa + k * LG_BLOCK, &tmA, m + k * 64, c, bar_c);
              }
            }
          } else if (small) {
            tma_load_2d(pb, &tmBs, B_MN ? nr : c, B_MN ? c : nr, bar_c);
          } else {
            for (int h = 0; h < nb; ++h) {
              if (!B_MN) tma_load_2d(pb + h * LG_TILE, &tmB, c, nr + h * 128, bar_c);
              else if (ATOMS) tma_load_3d(pb + h * LG_TILE, &tmB, 0, c, (nr + h * 128) >> 6, bar_c);
              else
                for (int k = 0; k < 2; ++k)
                  tma_load_2d(pb + h * LG_TILE + k * LG_BLOCK, &tmB, nr + h * 128 + k * 64, c, bar_c);
            }
          }
        }
      }
      pdl_launch_dependents();
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (leader) ----------------
      // The thread's own time per stage counts: the tensor pipe takes a few MMAs ahead, and what
      // the thread does between the last of a stage and the first of the next is idle time once
      // they have run out.  So the descriptors are kept as offsets, whole steps are unrolled, and
      // the next stage's barrier is looked at before this stage's MMAs.
      const uint64_t a_desc = A_MN ? desc_sw128_mn(smem_u32(smem), LG_BLOCK) : desc_sw128(smem_u32(smem));
      const uint64_t b_desc = B_MN ? desc_sw128_mn(smem_u32(smem + LG_TILE), LG_BLOCK) : desc_sw128(smem_u32(smem + LG_TILE));
      const uint32_t alo0 = uint32_t(a_desc), ahi = uint32_t(a_desc >> 32), blo0 = uint32_t(b_desc), bhi = uint32_t(b_desc >> 32);
      // 16 of the contraction, in the descriptors' 16-byte units: 32 bytes of a K-major row, two
      // 8-row groups (2 KB) of an MN-major block
      constexpr uint32_t A_K = A_MN ? 128 : 2, B_K = B_MN ? 128 : 2;
      // the MMAs of one stage into accumulator half h
      const auto mma = [&](int st, bool first, int groups, int h, uint32_t acc, uint32_t idesc) {
        const uint32_t off = uint32_t(st * (stage_bytes >> 4));
        const uint32_t a0 = alo0 + off, b0 = blo0 + off + uint32_t(h * (LG_TILE >> 4));
        if (groups == LG_KT / 16) {
#pragma unroll
          for (uint32_t kk = 0; kk < LG_KT / 16; ++kk)
            lg_mma(acc, a0 + A_K * kk, ahi, b0 + B_K * kk, bhi, idesc, kk == 0 ? uint32_t(!first) : 1u);
        } else {
          for (uint32_t kk = 0; kk < uint32_t(groups); ++kk)
            lg_mma(acc, a0 + A_K * kk, ahi, b0 + B_K * kk, bhi, idesc, uint32_t(!first) | kk);
        }
      };
      Cursor cur;
      int ac = 0;                                // accumulators used so far
      uint32_t cleared_par = 0;                  // bit s: parity of the next tail phase of stage s
      bool ok = true, issued = false, ready = false;
      int next = pair;
      for (LinTile tl; ok && lin_next<MODE, CUT>(args, row0, tile0, order, plan, pair, num_pairs, next, tl);) {
        if (MODE == LIN_WGRAD && tl.steps == 0) continue;        // the epilogue writes zeros
        const int accs = tl.accs();
        const int b0 = ac & 1, b1 = (ac + 1) & 1;
        const uint32_t acc0 = tmem + uint32_t(b0 * LG_ACC), acc1 = tmem + uint32_t(b1 * LG_ACC);
        const uint32_t id0 = lg_idesc(A_MN, B_MN, tl.cols(0)), id1 = lg_idesc(A_MN, B_MN, tl.cols(1));
        const uint32_t par1 = (((ac + 1) >> 1) & 1) ^ 1;
        const int last_groups = min(LG_KT, tl.c_cnt - (tl.k0 + tl.steps - 1) * LG_KT) + 15 >> 4;
        if (!wait_phase(&tmem_empty[b0], ((ac >> 1) & 1) ^ 1, abort_s, args.err, SITE_LINEAR + 1, lim)) {
          ok = false;
          break;
        }
        // steps to run ahead on the first accumulator while the epilogue reads the second
        const int lead = accs == 1 || mbar_test(&tmem_empty[b1], par1) ? 0 : min(LG_LEAD, tl.steps);
        Cursor behind = cur;
        tc_fence_after();
        for (int kt = 0; kt < tl.steps; ++kt) {
          if (!ready && !wait_phase(&full[cur.st], cur.ph, abort_s, args.err, SITE_LINEAR + 2, lim)) {
            ok = false;
            break;
          }
          const int st = cur.st;
          if (lin_tail<MODE>(tl) && kt + 1 == tl.steps) {
            if (!wait_phase_cluster(&cleared[st], (cleared_par >> st) & 1u, abort_s, args.err, SITE_LINEAR + 3, lim)) {
              ok = false;
              break;
            }
            cleared_par ^= 1u << st;
          }
          cur.next(stages);
          ready = mbar_test(&full[cur.st], cur.ph);
          tc_fence_after();
          const int groups = kt + 1 == tl.steps ? last_groups : LG_KT / 16;
          mma(st, kt == 0, groups, 0, acc0, id0);
          issued = true;
          if (kt < lead) {
            if (kt + 1 < lead) continue;
            if (!wait_phase(&tmem_empty[b1], par1, abort_s, args.err, SITE_LINEAR + 1, lim)) {
              ok = false;
              break;
            }
            tc_fence_after();
            for (int j = 0; j <= kt; ++j, behind.next(stages)) {
              mma(behind.st, j == 0, j == kt ? groups : LG_KT / 16, 1, acc1, id1);
              tc_commit(&empty[behind.st]);
            }
            continue;
          }
          if (accs == 2) mma(st, kt == 0, groups, 1, acc1, id1);
          tc_commit(&empty[st]);                 // frees the stage in both CTAs
        }
        if (!ok) break;
        tc_commit(&tmem_full[b0]);
        if (accs == 2) tc_commit(&tmem_full[b1]);
        ac += accs;
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
    const int width = min(64, args.tn >> 2), col0 = cg * width;  // this warp's columns of an accumulator
    const uint32_t tmem_row = tmem + (uint32_t(q * 32) << 16) + uint32_t(col0);
    const uint32_t tmem_empty_c0 = mapa_shared(smem_u32(tmem_empty), 0);
    const int M = lin_m<MODE>(args);
    uint32_t* tr = reinterpret_cast<uint32_t*>(smem + LG_OFF_TR + (warp - 2) * LG_TR_WARP);
    int ac = 0;
    bool ok = true;
    int next = pair;
    for (LinTile tl; ok && lin_next<MODE, CUT>(args, row0, tile0, order, plan, pair, num_pairs, next, tl);) {
      if (MODE == LIN_WGRAD && tl.steps == 0) {
        // the weight gradient of an expert without rows: zeros, 256 bytes of an output row per 16 lanes
        const int m = tl.m0 + int(rank) * 128 + (lane & 15) * 8;
        if (m < M)
          for (int c = (warp - 2) * 2 + (lane >> 4); c < tl.cnt; c += 2 * LG_EPI_WARPS)
            *reinterpret_cast<uint4*>(args.out + (int64_t(tl.e) * args.N + tl.n0 + c) * args.ldo + m) = make_uint4(0, 0, 0, 0);
        continue;
      }
      const int accs = tl.accs();
      for (int h = 0; h < accs; ++h, ++ac) {
        const int ab = ac & 1;
        if (!wait_phase_warp_moving(&tmem_full[ab], (ac >> 1) & 1, abort_s, args.err, SITE_LINEAR + 4, lim, stages_used)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int cols = tl.cols(h), part = cols >> 1;           // the first `part` columns are the leader's n
        uint32_t r[64];
        if (width == 16) {
          tmem_ld16_async(tmem_row + uint32_t(ab * LG_ACC), r);  // (past cols: columns that nobody stores)
          tmem_wait_ld<16>(r);
        } else if (col0 < cols) {
          tmem_ld32_async(tmem_row + uint32_t(ab * LG_ACC), r);
          if (width == 64 && col0 + 32 < cols) tmem_ld32_async(tmem_row + uint32_t(ab * LG_ACC) + 32u, r + 32);
          tmem_wait_ld<64>(r);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tmem_empty_c0 + uint32_t(ab) * 8u);
        // Lane l holds m = l of its warp's columns.  Through shared memory, 16 columns at a time, a lane
        // gets eight m of two columns, p and p + 1: 16-byte stores, 64 bytes per column and warp.
        const int p = lane >> 2, m = tl.m0 + int(rank) * 128 + q * 32 + (lane & 3) * 8;
        if (CUT && tl.parts > 1 && !join_pieces(args, tl, plan.rest, (int(rank) * 4 + q) * 4 + cg, lane, r)) continue;
        __nv_bfloat16* o = args.out + ((MODE == LIN_WGRAD ? int64_t(tl.e) * args.N : 0) + tl.n0 + 2 * p) * args.ldo + m;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 16) {
          const int j = col0 + c0;
          if (j >= cols || c0 >= width) break;
          const int off = (j >= part ? (tl.n >> 1) + j - part : j) + h * 128;    // n - n0 of column j
          if (off >= tl.cnt) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w = pack_bf16x2(__uint_as_float(r[c0 + 2 * i]), __uint_as_float(r[c0 + 2 * i + 1]));
            tr[i * LG_TR_PITCH + lane] = w;
          }
          __syncwarp();
          const uint4* src = reinterpret_cast<const uint4*>(tr + p * LG_TR_PITCH + (lane & 3) * 8);
          const uint4 u = src[0], v = src[1];
          __syncwarp();
          const int left = tl.cnt - (off + 2 * p);               // columns of the tile from this pair on
          __nv_bfloat16* oc = o + int64_t(off) * args.ldo;
          if (m < M && left > 0)
            *reinterpret_cast<uint4*>(oc) = make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410),
                                                       __byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410));
          if (m < M && left > 1)
            *reinterpret_cast<uint4*>(oc + args.ldo) =
                make_uint4(__byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x7632),
                           __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x7632));
        }
      }
    }
  } else if (warp == 18 && MODE == LIN_WGRAD) {
    // ---------------- rows of a tail stage past the expert's end (both CTAs) ----------------
    const uint32_t cleared_c0 = mapa_shared(smem_u32(cleared), 0);
    uint32_t par = 0;                            // bit s: parity of the next tail phase of stage s
    int at = 0;                                  // stages used so far
    bool ok = true;
    int next = pair;
    for (LinTile tl; ok && lin_next<MODE, CUT>(args, row0, tile0, order, plan, pair, num_pairs, next, tl);) {
      at += tl.steps;
      if (!lin_tail<MODE>(tl)) continue;
      // (a barrier is waited on in every one of its phases or not at all: skipping phases, this
      // warp would take an older phase of the same parity for the one it wants; so tail stages
      // have barriers of their own)
      const int st = (at - 1) % stages;
      ok = wait_phase_warp_moving(&tail[st], (par >> st) & 1u, abort_s, args.err, SITE_LINEAR + 5, lim, stages_used);
      if (!ok) break;
      par ^= 1u << st;
      const int valid = tl.c_cnt - (tl.steps - 1) * LG_KT;       // the stage's rows
      const int n = (((valid + 15) & ~15) - valid) * 8;          // 16-byte chunks to clear in each block
      const int blocks = 2 + (tl.n >> 7);                        // of 64 columns: M's two, N's one to four
      for (int i = lane; i < blocks * n; i += 32) {
        const int block = i / n, j = i - block * n;
        *reinterpret_cast<uint4*>(smem + st * stage_bytes + block * LG_BLOCK + (valid + (j >> 3)) * 128 + (j & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async;" ::: "memory");            // visible to the MMAs' reads
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_release(cleared_c0 + uint32_t(st) * 8u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && *abort_s) {
    // A wait gave up in this CTA, of whichever warp: copies issued before, by producers that may have
    // finished since, land before the shared memory goes (they take microseconds; bounded).  The others
    // wait for this warp at the cluster's barrier.
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
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

template <int MODE, bool ATOMS, bool CUT>
cudaError_t lin_launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mbs, const LinearArgs& a,
                       int grid, cudaStream_t st) {
  // the shared-memory attribute is per device: set it once on each device this process uses
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(grouped_linear_kernel<MODE, ATOMS, CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, LG_SMEM);
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
  return cudaLaunchKernelEx(&cfg, grouped_linear_kernel<MODE, ATOMS, CUT>, ma, mb, mbs, a);
}

}  // namespace

size_t linear_ws_bytes() {
  return 256 + size_t(kLinearMaxPairs) * LG_PLACES * (sizeof(unsigned) + LG_PIECE * sizeof(float));
}

cudaError_t launch_grouped_linear(int mode, const LinearArgs& args, const void* x, int64_t ldx, const void* dy,
                                  int64_t lddy, const void* w, cudaStream_t st, char* msg, size_t msg_len) {
  LinearArgs a = args;
  // the workspace: error word, arrival counts, pieces
  a.arrived = reinterpret_cast<unsigned*>(reinterpret_cast<uint8_t*>(a.err) + 256);
  a.pieces = reinterpret_cast<float*>(a.arrived + kLinearMaxPairs * LG_PLACES);
  CUtensorMap ma, mb, mbs;
  bool ok;
  const bool at = a.K % 64 == 0 && (mode == LIN_DGRAD || a.N % 64 == 0);   // rows of the MN-major operands
  if (mode == LIN_FWD) {
    ok = lin_map(&ma, false, w, a.K, a.N, a.K, a.E, 128) && lin_map(&mb, false, x, a.K, a.rows, ldx, 0, 128) &&
         lin_map(&mbs, false, x, a.K, a.rows, ldx, 0, LG_SMALL);
  } else if (mode == LIN_DGRAD) {
    ok = lin_map(&ma, at, w, a.K, a.N, a.K, a.E, 64) && lin_map(&mb, false, dy, a.N, a.rows, lddy, 0, 128) &&
         lin_map(&mbs, false, dy, a.N, a.rows, lddy, 0, LG_SMALL);
  } else {
    ok = lin_map(&ma, at, x, a.K, a.rows, ldx, 0, 64) && lin_map(&mb, at, dy, a.N, a.rows, lddy, 0, 64) &&
         lin_map(&mbs, false, dy, a.N, a.rows, lddy, 0, 64);
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
  // Columns of a tile.  64 (wgrad 128) where an expert has few rows, so that the call reads the
  // weights and little else: their stages are small and nine are in flight; and where 256 would
  // leave half the pairs without a tile (777 rows, K = 200, N = 136, E = 5: 8.6 -> 6.6 us a call).  512
  // where they still make four tiles a pair, else 256 (fewer, larger tiles leave pairs idle at the end).
  const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
  const int64_t mt = ((mode == LIN_FWD ? a.N : a.K) + LG_M - 1) / LG_M;
  const auto n_tiles = [&](int tn) {
    return mode == LIN_WGRAD ? int64_t(a.E) * ((a.N + tn - 1) / tn) : (a.rows < a.E ? a.rows : a.E) + a.rows / tn;
  };
  const int64_t wide = mode == LIN_WGRAD ? n_tiles(512) : a.rows / 512;
  const bool few_rows = mode != LIN_WGRAD && (a.rows <= 64 || a.rows <= int64_t(32) * a.E);
  if (few_rows || 2 * mt * n_tiles(256) <= pairs) a.tn = mode == LIN_WGRAD ? 128 : 64;
  else a.tn = mt * wide >= 4 * pairs ? 512 : 256;
  const int64_t nt = n_tiles(a.tn);
  // Tiles are cut where at most half the pairs have one, or where there is a second round at most
  // (16 rows, K = 14336, N = 4096: 165 -> 143 us; 2 rows, N = 14336, K = 4096, dgrad: 79 -> 57 us).  One
  // round of more than half the pairs cannot be cut, and the plain kernel is 2 us faster there.
  const int64_t tiles = mt * nt;
  const int steps = ((mode == LIN_FWD ? a.K : a.N) + LG_KT - 1) / LG_KT;
  const bool cut = a.tn == 64 && steps >= 2 * LG_MIN_PIECE && pairs <= kLinearMaxPairs &&
                   (2 * tiles <= pairs || (tiles > pairs && tiles <= 2 * pairs));
  // else no more pairs than tiles there can be
  const int grid = 2 * int(tiles < pairs && !cut ? tiles : pairs);
  switch (mode * 4 + int(at) * 2 + int(cut)) {
    case LIN_FWD * 4:
    case LIN_FWD * 4 + 2: return lin_launch<LIN_FWD, false, false>(ma, mb, mbs, a, grid, st);   // both K-major
    case LIN_FWD * 4 + 1:
    case LIN_FWD * 4 + 3: return lin_launch<LIN_FWD, false, true>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 4: return lin_launch<LIN_DGRAD, false, false>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 4 + 1: return lin_launch<LIN_DGRAD, false, true>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 4 + 2: return lin_launch<LIN_DGRAD, true, false>(ma, mb, mbs, a, grid, st);
    case LIN_DGRAD * 4 + 3: return lin_launch<LIN_DGRAD, true, true>(ma, mb, mbs, a, grid, st);
    case LIN_WGRAD * 4: return lin_launch<LIN_WGRAD, false, false>(ma, mb, mbs, a, grid, st);
    default: return lin_launch<LIN_WGRAD, true, false>(ma, mb, mbs, a, grid, st);
  }
}

}  // namespace moe
