// Forward and input gradient of the grouped linear layers on 8-bit operands for few rows an expert (tokens of
// a served model): bound by reading the weights.
//
// The sums are those of grouped_linear_fp8.cu, with the sides exchanged: the weights are the M side of the MMA
// and the rows the N side, whose extent an instruction can choose, so that a tile of 128 output values x up
// to 64 rows costs little more than its weights.  m is an output feature (forward) or an input feature (dgrad).  A
// CTA's 128 m share one scale a block, a row has its own, read from shared memory: with so few columns that is
// no load.  What decides the speed is how many weights are on their way: eight stages of 16 KB an SM, each
// with 64 columns of tensor memory of its own, so that nothing that a block's sums wait for holds up the
// loads.  (The pairs of the other kernel have two buffers, and hand them back across two SMs: 16 rows,
// 4096 -> 28672, six of eight experts, 155 us there.)
//   warp 0      TMA producer: 128 m and up to 64 rows of a block
//   warps 1, 2  the MMAs; warp 1 tensor memory too
//   warp 3      the experts' prefix sums
//   warps 4..7  sums, 32 m each
// Where the tiles do not fill the SMs evenly, they are cut along the contraction into equal pieces; the warp that
// finishes a tile's last piece adds the f32 partial sums from the workspace in the order of the contraction,
// so results do not depend on timing; nobody waits for anybody.
#include <atomic>
#include <cstdio>
#include <type_traits>

#include "linear8.cuh"

namespace moe {
namespace {

constexpr int F8_M = 128, F8_ROWS = 64;          // a CTA's tile
constexpr int F8_STAGES = 8;                     // as many as buffers of 64 columns in tensor memory
constexpr int F8_A = F8_M * L8_KT, F8_STAGE = F8_A + F8_ROWS * L8_KT;
constexpr int F8_SMALL = 16;                     // rows of the small box of rows
constexpr int F8_THREADS = 256;
constexpr int F8_AHEAD = 8;                      // blocks whose scales are on their way
constexpr int F8_SLOT = F8_ROWS + 4;             // a block's: the rows', then the weights'
static_assert(F8_PIECE == F8_M * F8_ROWS, "f32 of a piece");
constexpr int F8_MIN_PIECE = 4;                  // blocks a piece has at least

constexpr int F8_OFF_BAR = F8_STAGES * F8_STAGE;
constexpr int F8_OFF_MISC = F8_OFF_BAR + (2 * F8_STAGES + 2) * 8;            // full, done, drain[2]
constexpr int F8_OFF_SEG = (F8_OFF_MISC + 16 + 15) & ~15;        // row0[E+1], tile0[E+1]
constexpr int F8_OFF_SCALE = (F8_OFF_SEG + 2 * (L8_MAX_E + 1) * 4 + 15) & ~15;       // [warp][F8_AHEAD][F8_SLOT]
constexpr int F8_SMEM = F8_OFF_SCALE + 4 * F8_AHEAD * F8_SLOT * 4 + 1024;
static_assert(F8_SMEM <= 232448, "shared memory budget");

// The PTX of single CTAs (tcgen05.cuh has that of pairs).
__device__ __forceinline__ void f8_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void f8_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void f8_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One tcgen05.mma (E4M3, f32 accumulation) from descriptors given as their two halves.
__device__ __forceinline__ void f8_mma(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}"
      ::"r"(d), "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct Unit8 {
  int e, m0;       // expert, first m
  int r0, cnt;     // first row, and how many the tile has
  int tile, part;
  int k0, blocks;  // blocks of the contraction: first, number
};

// Piece u of the call's tiles * parts; the pieces of one place in the contraction run side by side, so that
// the weights are still read in long stretches.
template <int MODE>
__device__ __forceinline__ void f8_decode(const Linear8Args& a, const int* row0, const int* tile0, int tiles, int parts, int u,
                                          Unit8& w) {
  const int mt = ((MODE == LIN_FWD ? a.N : a.K) + F8_M - 1) / F8_M;
  const int all = ((MODE == LIN_FWD ? a.K : a.N) + L8_KT - 1) / L8_KT;
  w.part = u / tiles;
  w.tile = u - w.part * tiles;
  const int tt = w.tile / mt;
  w.m0 = (w.tile - tt * mt) * F8_M;
  int lo = 0, hi = a.E - 1;                      // largest e with tile0[e] <= tt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile0[mid] <= tt) lo = mid; else hi = mid - 1;
  }
  w.e = lo;
  w.r0 = row0[lo] + (tt - tile0[lo]) * F8_ROWS;
  w.cnt = min(F8_ROWS, row0[lo + 1] - w.r0);
  w.k0 = int(uint32_t(w.part) * uint32_t(all) / uint32_t(parts));            // below 608 * 2^13
  w.blocks = int(uint32_t(w.part + 1) * uint32_t(all) / uint32_t(parts)) - w.k0;
}

// Pieces of a tile: what makes the SMs' last round the fullest, each piece at least F8_MIN_PIECE blocks; a
// piece's own cost (its sums through memory, behind a fence) is taken as eight blocks (as two: 64 rows, 2048 -> 2816,
// E = 8: 22.1 us, 17.6; 100 rows, 1024 -> 1024, E = 8: 9.2, 7.8).  One warp, a number of pieces per lane.
__device__ __forceinline__ int f8_parts(int tiles, int all, int ctas, int lane) {
  const int most = min(all / F8_MIN_PIECE, tiles > 0 ? F8_MAX_PIECES / tiles : 1);
  uint32_t best = 0xFFFFFFFFu;                   // blocks of the longest SM, then pieces (fewest win)
  for (int p = lane + 1; p <= max(most, 1); p += 32) {
    // below 2^32: tiles * p is at most F8_MAX_PIECES, or p is 1 and tiles below 2^22
    const uint32_t rounds = (uint32_t(tiles) * p + ctas - 1) / uint32_t(ctas), cost = rounds * ((uint32_t(all) + p - 1) / p + (p > 1 ? 8 : 0));
    const uint32_t key = (cost < (1u << 21) ? cost : (1u << 21) - 1) << 10 | uint32_t(p);
    best = min(best, key);
  }
  return int(__reduce_min_sync(0xFFFFFFFFu, best) & 1023u);
}

template <int MODE>
__global__ void __launch_bounds__(F8_THREADS, 1)
    grouped_linear_fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                                  const __grid_constant__ CUtensorMap tmXs, const Linear8Args args) {
  constexpr bool A_MN = MODE == LIN_DGRAD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F8_OFF_BAR);
  uint64_t* done = full + F8_STAGES;
  uint64_t* drain = done + F8_STAGES;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + F8_OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + F8_OFF_MISC + 4);
  volatile int* bad_s = reinterpret_cast<volatile int*>(smem + F8_OFF_MISC + 8);
  volatile int* parts_s = reinterpret_cast<volatile int*>(smem + F8_OFF_MISC + 12);
  int* row0 = reinterpret_cast<int*>(smem + F8_OFF_SEG);
  int* tile0 = row0 + L8_MAX_E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = MODE == LIN_FWD ? args.N : args.K, mt = (M + F8_M - 1) / F8_M;
  const int all = ((MODE == LIN_FWD ? args.K : args.N) + L8_KT - 1) / L8_KT;
  if (threadIdx.x == 0) {
    for (int s = 0; s < F8_STAGES; ++s) {
      mbar_init(&full[s], 1 + 4);                // the operands, and the buffer from the four warps that add
      mbar_init(&done[s], 1);                    // the block's sums are there, and its stage is free
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmXs);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_base_s)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // Up to here the kernel touches only its own shared memory, tensor memory and parameters.
  pdl_wait();
  if (warp == 3) {
    const bool bad = l8_prefix<F8_ROWS>(args, lane, row0, tile0);
    __syncwarp();
    const int parts = f8_parts(tile0[args.E] * mt, all, int(gridDim.x), lane);
    if (lane == 0) {
      *bad_s = bad;
      *parts_s = parts;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const int parts = *parts_s;
  // inconsistent split_sizes: nothing is computed (the error word says so)
  const int tiles = *bad_s ? 0 : tile0[args.E] * mt;
  const int units = tiles * parts;
  const uint64_t lim = args.wait_limit_ns;

  if (warp == 0) {
    if (lane == 0 && !args.selftest_no_loads) {
      // ---------------- TMA producer ----------------
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      Unit8 w;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        f8_decode<MODE>(args, row0, tile0, tiles, parts, u, w);
        const bool small = w.cnt <= F8_SMALL;
        for (int kt = 0; kt < w.blocks; ++kt) {
          if (!wait_phase_inline(&done[st], ph ^ 1u, abort_s, args.err, SITE_LINEAR8, lim)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[st], uint32_t(F8_A + (small ? F8_SMALL : F8_ROWS) * L8_KT));
          uint8_t* pa = smem + st * F8_STAGE;
          const int c = (w.k0 + kt) * L8_KT;
          f8_load_3d(pa, &tmW, A_MN ? w.m0 : c, A_MN ? c : w.m0, w.e, &full[st]);
          f8_load_2d(pa + F8_A, small ? &tmXs : &tmX, c, w.r0, &full[st]);
          if (++st == F8_STAGES) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      pdl_launch_dependents();
    }
  } else if (warp == 1 || warp == 2) {
    if (lane == 0) {
      // ---------------- MMA issuers: warp 1 the even stages, warp 2 the odd ones ----------------
      // A block's wait, four MMAs and commit take a thread about 740 clocks, as long as its weights take at the
      // memory's rate; two threads at it are out of the way.
      const uint64_t a_desc = A_MN ? desc_sw128_mn(smem_u32(smem), F8_A) : desc_sw128(smem_u32(smem));
      const uint64_t b_desc = desc_sw128(smem_u32(smem + F8_A));
      constexpr uint32_t A_K = A_MN ? 256 : 2, B_K = 2;            // 32 of the contraction, in 16-byte units
      const int last = (MODE == LIN_FWD ? args.K : args.N) - (all - 1) * L8_KT;
      const int odd = warp - 1;
      bool ok = true, issued = false;
      uint32_t ph = 0;
      int st = odd, before = 0;                  // before: blocks of all pieces so far
      Unit8 w;
#pragma unroll 1
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        f8_decode<MODE>(args, row0, tile0, tiles, parts, u, w);
        const uint32_t idesc = (1u << 4) | (uint32_t(A_MN) << 15) | (uint32_t(((w.cnt + 15) & ~15) >> 3) << 17) |
                               (uint32_t(F8_M >> 4) << 24);
        const int ends = w.k0 + w.blocks == all ? w.blocks - 1 : -1;         // the block that may be a short one
#pragma unroll 1
        for (int kt = (before ^ odd) & 1; kt < w.blocks; kt += 2) {
          ok = wait_phase_inline(&full[st], ph, abort_s, args.err, SITE_LINEAR8 + 1, lim);
          if (!ok) break;
          tc_fence_after();
          const uint32_t acc = tmem + st * F8_ROWS, off = uint32_t(st * (F8_STAGE >> 4));
          const uint32_t alo = uint32_t(a_desc) + off, blo = uint32_t(b_desc) + off;
          const int groups = kt == ends ? (last + 31) >> 5 : 4;
          f8_mma(acc, alo, uint32_t(a_desc >> 32), blo, uint32_t(b_desc >> 32), idesc, 0);
#pragma unroll
          for (uint32_t kk = 1; kk < 4; ++kk)
            if (int(kk) < groups)
              f8_mma(acc, alo + A_K * kk, uint32_t(a_desc >> 32), blo + B_K * kk, uint32_t(b_desc >> 32), idesc, 1);
          issued = true;
          f8_commit(&done[st]);
          st += 2;
          if (st >= F8_STAGES) {
            st = odd;
            ph ^= 1u;
          }
        }
        before += w.blocks;
      }
      if (!ok && issued) {
        f8_commit(&drain[odd]);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&drain[odd], 0) && globaltimer_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- sums ----------------
    const int q = warp & 3;                      // lane quarter this warp may access
    const uint32_t tmem_row = tmem + (uint32_t(q * 32) << 16);
    const int kbs = (args.K + 127) / 128, nbs = (args.N + 127) / 128;
    const int64_t sb_step = MODE == LIN_FWD ? 1 : kbs;
    // the warp's ring of scales: lane l copies rows l and l + 32, lane 0 the weights' too
    float* const ring = reinterpret_cast<float*>(smem + F8_OFF_SCALE) + q * F8_AHEAD * F8_SLOT;
    for (int s = 0; s < F8_STAGES; ++s)
      if (lane == 0) mbar_arrive(&full[s]);      // all buffers are free at first
    int st = 0, slot = 0, coming = 0, cnt = 0;
    uint32_t ph = 0;
    const float *sa = nullptr, *sb = nullptr;
    const auto ask = [&]() {
      if (coming > 0) {
        float* to = ring + slot * F8_SLOT;
        if (lane < cnt) cp_async4(to + lane, sa + lane);
        if (lane + 32 < cnt) cp_async4(to + lane + 32, sa + lane + 32);
        if (lane == 0) cp_async4(to + F8_ROWS, sb);
        sa += args.rows;
        sb += sb_step;
        --coming;
      }
      cp_async_group();
      slot = slot + 1 == F8_AHEAD ? 0 : slot + 1;
    };
    bool ok = true;
    Unit8 w;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      f8_decode<MODE>(args, row0, tile0, tiles, parts, u, w);
      cnt = w.cnt;
      coming = w.blocks;
      sa = args.sa + w.k0 * args.rows + w.r0;
      const int mb = w.m0 / 128;
      sb = args.sb + int64_t(w.e) * nbs * kbs + (MODE == LIN_FWD ? int64_t(mb) * kbs + w.k0 : int64_t(w.k0) * kbs + mb);
#pragma unroll 1
      for (int i = 0; i < F8_AHEAD; ++i) ask();
      float acc[F8_ROWS];
#pragma unroll
      for (int i = 0; i < F8_ROWS; ++i) acc[i] = 0.f;
      for (int left = w.blocks; left > 0; --left) {
        cp_async_left<F8_AHEAD - 1>();
        __syncwarp();                            // the other lanes' copies too
        const float* sc = ring + slot * F8_SLOT;
        const float sw = sc[F8_ROWS];
        ok = wait_phase_warp_inline(&done[st], ph, abort_s, args.err, SITE_LINEAR8 + 4, lim);
        if (!ok) break;
        tc_fence_after();
        uint32_t p[F8_ROWS];
        const uint32_t src = tmem_row + uint32_t(st * F8_ROWS);
        // 16 rows at a time, as many as the tile has
        tmem_ld16_async(src, p);
        if (cnt > 16) tmem_ld16_async(src + 16, p + 16);
        if (cnt > 32) tmem_ld32_async(src + 32, p + 32);
        tmem_wait_ld<F8_ROWS>(p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
#pragma unroll
        for (int c = 0; c < F8_ROWS; c += 4) {
          if (c >= cnt) break;
          const float4 s4 = *reinterpret_cast<const float4*>(sc + c);
          acc[c] = fmaf(__uint_as_float(p[c]), s4.x * sw, acc[c]);
          acc[c + 1] = fmaf(__uint_as_float(p[c + 1]), s4.y * sw, acc[c + 1]);
          acc[c + 2] = fmaf(__uint_as_float(p[c + 2]), s4.z * sw, acc[c + 2]);
          acc[c + 3] = fmaf(__uint_as_float(p[c + 3]), s4.w * sw, acc[c + 3]);
        }
        __syncwarp();                            // all lanes have read the slot
        ask();
        if (++st == F8_STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (parts > 1) {
        // the warp's share of the piece, [row][32 m], and its tile's arrivals
        const auto piece = [&](int part) { return args.pieces + (int64_t(part) * tiles + w.tile) * F8_PIECE + q * (F8_ROWS * 32) + lane; };
        float* mine = piece(w.part);
#pragma unroll
        for (int c = 0; c < F8_ROWS; ++c)
          if (c < cnt) __stcg(mine + c * 32, acc[c]);
        __threadfence();
        __syncwarp();
        unsigned before = 0;
        if (lane == 0) before = atomicAdd(args.arrived + w.tile * 4 + q, 1u);
        before = __shfl_sync(0xFFFFFFFFu, before, 0);
        if (before + 1 != unsigned(parts)) continue;
        __threadfence();
        if (lane == 0) args.arrived[w.tile * 4 + q] = 0;           // for the next call
        // few rows: four pieces at a time are on their way
        const auto join = [&](auto most) {
          constexpr int ROWS = decltype(most)::value, BATCH = F8_ROWS / ROWS;
#pragma unroll
          for (int c = 0; c < ROWS; ++c) acc[c] = 0.f;
          for (int p = 0; p < parts; p += BATCH) {
            float v[BATCH][ROWS];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
              for (int c = 0; c < ROWS; ++c) v[i][c] = c < cnt && p + i < parts ? __ldcg(piece(p + i) + c * 32) : 0.f;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
              for (int c = 0; c < ROWS; ++c) acc[c] += v[i][c];
          }
        };
        if (cnt <= F8_SMALL) join(std::integral_constant<int, F8_SMALL>{});
        else join(std::integral_constant<int, F8_ROWS>{});
      }
      // lanes hold neighbouring m of a row: 64 bytes a warp and row
      const int m = w.m0 + q * 32 + lane;
      if (m < M) {
        __nv_bfloat16* o = args.out + int64_t(w.r0) * args.ldo + m;
#pragma unroll
        for (int c = 0; c < F8_ROWS; ++c)
          if (c < cnt) o[c * args.ldo] = __float2bfloat16_rn(acc[c]);
      }
    }
    cp_async_left<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && *abort_s) {
    // A wait gave up: copies issued before land before the shared memory goes (they take microseconds; bounded).
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int MODE>
cudaError_t f8_launch(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& mxs, const Linear8Args& a, int grid,
                      cudaStream_t st) {
  // the shared-memory attribute is per device: set it once on each device this process uses
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(grouped_linear_fp8_few_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, F8_SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) ready[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(grouped_linear_fp8_few_kernel<MODE>, dim3(unsigned(grid)), dim3(F8_THREADS), F8_SMEM, st, mw, mx, mxs, a);
}

}  // namespace

cudaError_t launch_grouped_linear_fp8_few(int mode, const Linear8Args& args, const uint8_t* rows_codes, const uint8_t* w_codes,
                                          int sms, cudaStream_t st, char* msg, size_t msg_len) {
  const Linear8Args& a = args;
  CUtensorMap mw, mx, mxs;
  const int64_t inner = mode == LIN_FWD ? a.K : a.N;
  if (!l8_map(&mw, w_codes, a.K, a.N, a.E, 128) || !l8_map(&mx, rows_codes, inner, a.rows, 0, F8_ROWS) ||
      !l8_map(&mxs, rows_codes, inner, a.rows, 0, F8_SMALL)) {
    snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (rows %lld, K %d, N %d, E %d)", (long long)a.rows, a.K, a.N,
             a.E);
    return cudaErrorInvalidValue;
  }
  return mode == LIN_FWD ? f8_launch<LIN_FWD>(mw, mx, mxs, a, sms, st) : f8_launch<LIN_DGRAD>(mw, mx, mxs, a, sms, st);
}

}  // namespace moe
