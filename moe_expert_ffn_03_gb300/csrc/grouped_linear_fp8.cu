// Linear layers grouped by expert on dense ragged rows with 8-bit operands: E4M3 codes and one f32
// scale per block of 128, forward, input gradient and weight gradient on the tensor cores (tcgen05
// kind::f8f6f4).
//
// Page "Efficient MoE Training for Biological Foundation Models", sections "GroupedLinear：把逐专家
// 循环改成一次分组GEMM" (one grouped call over the experts' rows) and "MoE训练的瓶颈与TE的对应能力"
// (8-bit operands; the blocks of 128 with f32 scales are an interface addition).
//
//   D[m][n] = sum over blocks b of 128 of  sa[b][m] * sb[b][n / 128] * (sum over the block of A * B)
//   forward   m rows,      n output features, sum over K:      A = x codes,  B = w codes
//   dgrad     m rows,      n input features,  sum over N:      A = dy codes, B = w codes, MN-major
//   wgrad     m out. feat. n input features,  sum over tokens: A = dy codes, B = x codes, both MN-major
//
// The tensor cores sum codes, so every block of 128 is a product of its own, whose f32 sums are scaled and
// added to f32 sums in registers.  What that costs decides the layout: with m in the lanes and n in the
// columns of tensor memory, a thread's row has one scale and its 128 columns (aligned to a block of the B
// side) another, so a partial sum takes one multiply-add with one factor per thread.  (A scale per
// column would have to come out of shared memory, 32 bits for every multiply-add.)  256 x 256 x 128 takes
// the pair's tensor pipes 512 clocks, an SM's quarter 256 of packed multiply-adds and 136 of reads.
//
// Persistent CTA pairs (clusters of two, one CTA per SM), tiles of 256 m x 256 n with cta_group::2: each
// CTA stages its 128 m and its 128 n of a block, 32 KB a stage, four stages.  The 512 columns of tensor
// memory are two buffers of 256: the tensor pipe fills one with a block's sums while the other is added.
//   warp 0       TMA producer of the A side, warp 2 of the B side
//   warp 1       tensor memory; in the leader, the MMAs
//   warp 3       the experts' prefix sums, then the tiles, laid out ahead for the others
//   warps 4..11  sums: two per lane quarter, 128 columns each, with 232 registers a thread (the other
//                four warps give up theirs: 128 x 40 + 256 x 232 = 384 x 168)
// Waits are bounded as everywhere; each lasts as long as a block or a tile's output at most, warp 3's as long as a
// tile.
//
// What holds the tensor pipe up is the way round of a buffer: sums there, seen, read, added, handed back, seen,
// filled again, with single threads and two warps a quarter on it: 750 clocks a block, 613 without any sums.  So a
// block has one wait and one commit for the MMA's thread, constant descriptors, scales asked for two
// blocks ahead (8192 rows, 4096 -> 16384, before the steps below: one ahead 490 us, two 414; from a ring in shared
// memory 412, but 32768 rows 5% longer), and goes back before its last half is added (416 -> 404); measured the
// same or worse: sixteen warps of 64 columns (494 against 490), halves of 128 columns with four buffers (558; an
// MMA of 128 columns takes 104 clocks, not 64), single CTAs of 128 x 256 (490), a second thread that issues
// (478), test_wait in place of try_wait where the sums are waited for (425 against 396).  All of these on one card with
// even splits, random codes and a memory fill between calls, and so: 32768 rows, 4096 -> 28672, E = 8, forward
// 2.78 ms (2.77 PFLOP/s; on other cards 2.89 to 3.12); 8192 rows, 4096 -> 16384, E = 2: 396 us (2.78; 451 to 463);
// 65536 rows, 2048 -> 2816, E = 16: 304 us forward (2.49: a tile's output is a tenth of its time there; 316 to 359), 300
// input gradient (302 to 306), 278 weight gradient (2.72; 287 to 297).  Calls in a row meet the power limit, and loads that
// are uneven leave pairs without work: the first with such loads 3.12 to 3.32 ms (2.4).
#include <atomic>
#include <cstdio>
#include <type_traits>

#include "linear8.cuh"

namespace moe {
namespace {

struct alignas(16) Tile8 {
  int e;
  int m0, cnt;     // first m (a row of all experts', or an output feature of e) and how many the tile has
  int n0;          // first n
  int n;           // the MMA's columns: those left rounded up to 32; CTA r holds n0 + r * n/2 ..
  int c0;          // contraction: first index (wgrad: row of the layout on blocks)
  int blocks;      // its blocks of 128; -1 behind the last tile
  int last;        // indices in the last block
  const float *sa, *sb[2];  // scales of the first block: m0's, and those of n0 and n0 + 128
  int piece;       // of a tile that is cut: where its partial sums go; else -1
  int unused;
};

constexpr int L8_M = 256, L8_N = 256;            // the pair's tile
constexpr int L8_SIDE = 128 * L8_KT;             // bytes of a CTA's A or B in a stage
constexpr int L8_STAGE = 2 * L8_SIDE;
constexpr int L8_STAGES = 4;                     // an even number: a block's buffer is its stage's parity
constexpr int L8_EPI_WARPS = 8;
constexpr int L8_THREADS = 32 * (4 + L8_EPI_WARPS);
constexpr int L8_REGS = 168, L8_REGS_FEW = 40, L8_REGS_MANY = 232;
static_assert(128 * L8_REGS_FEW + 32 * L8_EPI_WARPS * L8_REGS_MANY == L8_THREADS * L8_REGS, "register split");
constexpr int L8_GROUP = 8;                      // row tiles that share the sweep over the weights
constexpr int L8_SMALL = 32;                     // rows of the small box of rows
constexpr int L8_SHARES = 2 * L8_EPI_WARPS;      // of a tile: 32 m x 128 n each
constexpr int L8_MIN_CUT = 8;                    // blocks up to which a tile is not cut

// a warp's output on its way: two boxes of 32 rows of 64 bf16, swizzled in 128 bytes
constexpr int L8_BOX = 32 * 128;
constexpr int L8_OFF_OUT = L8_STAGES * L8_STAGE;
constexpr int L8_OFF_BAR = L8_OFF_OUT + L8_EPI_WARPS * 2 * L8_BOX;
constexpr int L8_TILES = 4;                      // tiles laid out ahead
constexpr int L8_BARS = 2 * L8_STAGES + 1 + 2 * L8_TILES;        // full, empty, drain, laid, taken
constexpr int L8_OFF_MISC = L8_OFF_BAR + L8_BARS * 8;
constexpr int L8_OFF_SEG = (L8_OFF_MISC + 16 + 15) & ~15;        // row0[E+1], tile0[E+1], order[E], unit0[E+1]
constexpr int L8_OFF_TILES = (L8_OFF_SEG + 4 * (L8_MAX_E + 1) * 4 + 15) & ~15;
constexpr int L8_SMEM = L8_OFF_TILES + L8_TILES * int(sizeof(Tile8)) + 1024;
static_assert(L8_SMEM <= 232448, "shared memory budget");

// kind::f8f6f4 instruction descriptor: E4M3 x E4M3 -> f32, M = 256, N columns; a_mn, b_mn: the operand
// is MN-major.
__device__ __forceinline__ uint32_t l8_idesc(bool a_mn, bool b_mn, int N) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(L8_M >> 4) << 24);
}
// One tcgen05.mma (E4M3, f32 accumulation).  All descriptors of a kernel differ in the low half only, by a
// constant from the ring's first, and are made here: as values of their own, all stages' would be kept in
// registers at once, and there are none for them.
template <uint32_t A_OFF, uint32_t B_OFF, bool ACCUMULATE>
__device__ __forceinline__ void l8_mma(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 la, lb;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "add.u32 la, %1, %6;\n\t"
      "add.u32 lb, %3, %7;\n\t"
      "mov.b64 da, {la, %2};\n\t"
      "mov.b64 db, {lb, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %5, p;\n\t}"
      ::"r"(d), "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "n"(A_OFF), "n"(B_OFF), "n"(int(ACCUMULATE))
      : "memory");
}

struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == L8_STAGES) {
      st = 0;
      ph ^= 1u;
    }
  }
};


template <int MODE>
__device__ __forceinline__ int l8_cols(const Linear8Args& a) { return MODE == LIN_FWD ? a.N : a.K; }

template <int MODE>
__device__ __forceinline__ int l8_tiles(const Linear8Args& a, const int* tile0) {
  const int nt = (l8_cols<MODE>(a) + L8_N - 1) / L8_N;
  return MODE == LIN_WGRAD ? a.E * ((a.N + L8_M - 1) / L8_M) * nt : tile0[a.E] * nt;
}

// An expert's tile i of the weight gradient: the n tiles of a few m tiles in turn.
__device__ __forceinline__ void l8_wgrad_tile(const Linear8Args& a, int i, int& m0, int& n0) {
  const int mt = (a.N + L8_M - 1) / L8_M, nt = (a.K + L8_N - 1) / L8_N, per = L8_GROUP * nt;
  const int g = i / per, first = g * L8_GROUP, gs = min(L8_GROUP, mt - first);
  const int local = i - g * per;
  m0 = (first + local % gs) * L8_M;
  n0 = local / gs * L8_N;
}

// Warps (their logarithm) that share a cut tile's sums: with few pieces they are quick for one.
__device__ __forceinline__ int l8_team(int parts) { return parts <= 4 ? 0 : parts <= 8 ? 1 : parts <= 16 ? 2 : 3; }

// One warp: into how many pieces the weight gradient's tiles are cut along their rows, where an expert's are few and
// long.  unit0: of every expert in `order` (most rows first) the first of its tiles' pieces, those of one
// place side by side.  A piece has `len` blocks at most: of 31 lengths from an even share of the pairs up, and
// of the longest tile's, the one that is done first by this measure in blocks (400 ns): the pairs' rounds, or an even
// share and one piece more if that is less; four for an output; if anything is cut, 8 for the second launch
// and a fifth for writing and reading each piece.  Cut tiles are longer than a share, so that their pieces are less than
// twice as many as the pairs.  The cut experts are written to `plan`.
__device__ __forceinline__ void l8_cut(const Linear8Args& a, const int* row0, const int* order, int* unit0, int pairs, int lane,
                                       bool writes) {
  const int tiles = ((a.N + L8_M - 1) / L8_M) * ((a.K + L8_N - 1) / L8_N);            // an expert's
  const auto blocks_of = [&](int slot) { return (row0[order[slot] + 1] - row0[order[slot]] + L8_KT - 1) / L8_KT; };
  int64_t sum = 0;
  for (int s = lane; s < a.E; s += 32) sum += blocks_of(s);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  const int share = int((sum * tiles + pairs - 1) / pairs), longest = blocks_of(0);
  const int base = max(L8_MIN_CUT, share);
  int len = lane < 31 ? base + int(int64_t(base) * lane / 8) : max(base, longest);
  const float per = 1.f / float(len);
  float units = 0.f, cut = 0.f;
  int s = 0;
  for (; s < a.E; ++s) {
    const int b = blocks_of(s);
    if (b <= base) break;                        // nor are those behind it cut
    const float parts = b <= len ? 1.f : ceilf(float(b) * per);
    units += parts;
    cut += b <= len ? 0.f : parts;
  }
  units = (units + float(a.E - s)) * float(tiles);
  const float piece = float(min(len, longest));
  const float cost = fminf(ceilf(units / float(pairs)) * piece, float(share) + piece) + 4.f +
                     (cut > 0.f ? 8.f + 0.2f * cut * float(tiles) : 0.f);
  const uint32_t best = __reduce_min_sync(0xFFFFFFFFu, __float_as_uint(cost));        // not negative: ordered as integers
  len = __shfl_sync(0xFFFFFFFFu, len, __ffs(__ballot_sync(0xFFFFFFFFu, __float_as_uint(cost) == best)) - 1);
  // eight experts a lane
  for (;;) {
    int mine[8], all = 0, cut = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = lane * 8 + i;
      const int parts = slot < a.E ? max(1, (blocks_of(slot) + len - 1) / len) : 0;
      mine[i] = parts * tiles;
      all += mine[i];
      cut += parts > 1 ? mine[i] : 0;
    }
    int before = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, before, off);
      if (lane >= off) before += u;
    }
    before -= all;
    if (__reduce_add_sync(0xFFFFFFFFu, unsigned(cut)) > unsigned(L8_MAX_PIECES)) {
      len += len;
      continue;
    }
    int joins = 0;                               // units of the second launch
#pragma unroll
    for (int i = 0; i < 8; ++i) joins += mine[i] > tiles ? tiles * L8_SHARES << l8_team(mine[i] / tiles) : 0;
    int join0 = joins;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, join0, off);
      if (lane >= off) join0 += u;
    }
    const int all_joins = __shfl_sync(0xFFFFFFFFu, join0, 31);
    join0 -= joins;
    int cuts = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = lane * 8 + i;
      if (slot <= a.E) unit0[slot] = before;
      if (mine[i] > tiles) {
        const int parts = mine[i] / tiles;
        ++cuts;
        if (writes) reinterpret_cast<int4*>(a.plan)[1 + slot] = make_int4(order[slot], before, parts, join0);
        join0 += tiles * L8_SHARES << l8_team(parts);
      }
      before += mine[i];
    }
    if (lane == 31 && a.E == L8_MAX_E) unit0[L8_MAX_E] = before;
    cuts = int(__reduce_add_sync(0xFFFFFFFFu, unsigned(cuts)));
    if (writes && lane == 0) reinterpret_cast<int4*>(a.plan)[0] = make_int4(cuts, all_joins, 0, 0);
    __syncwarp();
    return;
  }
}

// tile0: the experts' first row tiles; wgrad: their first blocks of 128 rows.
template <int MODE, bool CUT>
__device__ __forceinline__ void l8_decode(const Linear8Args& a, const int* row0, const int* tile0, const int* order,
                                          const int* unit0, int t, Tile8& tl) {
  const int cols = l8_cols<MODE>(a), nt = (cols + L8_N - 1) / L8_N;
  tl.piece = -1;
  if (MODE == LIN_WGRAD) {
    // experts with the most rows first
    const int tiles = (a.N + L8_M - 1) / L8_M * nt;
    int slot, rem, part = 0, parts = 1;
    if constexpr (CUT) {
      int lo = 0, hi = a.E - 1;                  // largest slot with unit0[slot] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit0[mid] <= t) lo = mid; else hi = mid - 1;
      }
      slot = lo;
      rem = t - unit0[slot];
      parts = (unit0[slot + 1] - unit0[slot]) / tiles;
      part = rem / tiles;
      rem -= part * tiles;
      if (parts > 1) tl.piece = t;
    } else {
      slot = t / tiles;
      rem = t - slot * tiles;
    }
    tl.e = order[slot];
    l8_wgrad_tile(a, rem, tl.m0, tl.n0);
    tl.cnt = min(L8_M, a.N - tl.m0);
    const int rows = row0[tl.e + 1] - row0[tl.e], all = (rows + L8_KT - 1) / L8_KT;
    const int from = CUT ? int(int64_t(part) * all / parts) : 0, to = CUT ? int(int64_t(part + 1) * all / parts) : all;
    tl.c0 = (tile0[tl.e] + from) * L8_KT;
    tl.blocks = to - from;
    tl.last = to == all ? rows - (all - 1) * L8_KT : L8_KT;
  } else {
    const int total = tile0[a.E];
    const int per = L8_GROUP * nt;
    const int g = t / per, first = g * L8_GROUP, gs = min(L8_GROUP, total - first);
    const int local = t - g * per;
    const int tt = first + local % gs;
    int lo = 0, hi = a.E - 1;                    // largest e with tile0[e] <= tt
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] <= tt) lo = mid; else hi = mid - 1;
    }
    tl.e = lo;
    tl.n0 = local / gs * L8_N;
    tl.m0 = row0[lo] + (tt - tile0[lo]) * L8_M;
    tl.cnt = min(L8_M, row0[lo + 1] - tl.m0);
    const int c = MODE == LIN_FWD ? a.K : a.N;
    tl.c0 = 0;
    tl.blocks = (c + L8_KT - 1) / L8_KT;
    tl.last = c - (tl.blocks - 1) * L8_KT;
  }
  tl.n = (min(L8_N, cols - tl.n0) + 31) & ~31;
  const int64_t kbs = (a.K + 127) / 128, nbs = (a.N + 127) / 128, nb = tl.n0 / 128, blk = tl.c0 / L8_KT;
  tl.sa = a.sa + (MODE == LIN_WGRAD ? blk * a.N : 0) + tl.m0;
  tl.sb[0] = a.sb + (MODE == LIN_FWD ? (tl.e * nbs + nb) * kbs : (MODE == LIN_DGRAD ? tl.e * nbs : blk) * kbs + nb);
  tl.sb[1] = tl.sb[0] + (MODE == LIN_FWD ? kbs : 1);
}

// The pair's tile after t.  wgrad: there and back, since tiles come longest first: the pair that got the
// longest of one round gets the shortest of the next.
template <int MODE>
__device__ __forceinline__ int l8_after(int t, int num_pairs) {
  return t + (MODE == LIN_WGRAD ? 2 * (num_pairs - 1 - t % num_pairs) + 1 : num_pairs);
}

// The pair's tiles in turn, as warp 3 of each CTA lays them out in a small ring of shared memory: finding a tile (a
// search among the experts, divisions) took the warps that add 4000 clocks, a quarter of a tile of 2048.
struct Tiles8 {
  const Tile8* ring;
  uint64_t *laid, *taken;
  int slot = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ Tiles8(const Tile8* r, uint64_t* l, uint64_t* t) : ring(r), laid(l), taken(t) {}
  __device__ __forceinline__ void advance() {
    if (++slot == L8_TILES) {
      slot = 0;
      ph ^= 1u;
    }
  }
};

// acc += part * f, two at a time
__device__ __forceinline__ void l8_add(float* acc, const uint32_t* part, float2 f) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(part[i]), __uint_as_float(part[i + 1])), f,
                                make_float2(acc[i], acc[i + 1]));
    acc[i] = r.x;
    acc[i + 1] = r.y;
  }
}

// A warp's arrival on the leader's barrier of a buffer that it has read (mbar_arrive_cluster_relaxed by lane 0,
// without a branch).
__device__ __forceinline__ void l8_hand_back(uint32_t caddr, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}"
      ::"r"(caddr), "r"(lane)
      : "memory");
}

// A box of the output from shared memory; what is past the output's end is left out.
template <int MODE>
__device__ __forceinline__ void l8_store(const CUtensorMap* map, const void* src, int n, int m, int e) {
  if constexpr (MODE == LIN_WGRAD)
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(n), "r"(m), "r"(e) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(n), "r"(m) : "memory");
}

template <int MODE, bool CUT>
__global__ void __launch_bounds__(L8_THREADS, 1)
    grouped_linear_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAs,
                              const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmO,
                              const Linear8Args args) {
  constexpr bool A_MN = MODE == LIN_WGRAD, B_MN = MODE != LIN_FWD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L8_OFF_BAR);
  uint64_t* empty = full + L8_STAGES;
  uint64_t* drain = empty + L8_STAGES;
  uint64_t* laid = drain + 1;
  uint64_t* taken = laid + L8_TILES;
  Tile8* const tile_ring = reinterpret_cast<Tile8*>(smem + L8_OFF_TILES);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + L8_OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + L8_OFF_MISC + 4);
  volatile int* bad_s = reinterpret_cast<volatile int*>(smem + L8_OFF_MISC + 8);
  int* row0 = reinterpret_cast<int*>(smem + L8_OFF_SEG);
  int* tile0 = row0 + L8_MAX_E + 1;
  int* order = tile0 + L8_MAX_E + 1;
  int* unit0 = order + L8_MAX_E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();       // 0: leader (issues the MMAs), 1: peer
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L8_STAGES; ++s) {
      mbar_init(&full[s], 1 + 2 * L8_EPI_WARPS); // the operands, and the buffer from both CTAs' warps
      mbar_init(&empty[s], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < L8_TILES; ++i) {
      mbar_init(&laid[i], 1);
      // by the warps that add, the producers and, in the leader, the MMA issuer
      mbar_init(&taken[i], L8_EPI_WARPS + (args.selftest_no_loads ? 0 : 2) + (rank == 0 ? 1 : 0));
    }
    *abort_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmAs);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmO);
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_s, 512);                // collectively with the peer CTA
    tmem_relinquish();
  }
  cluster_arrive();                              // this CTA's barriers are initialised
  // Up to here the kernel touches only its own shared memory, tensor memory and parameters.
  pdl_wait();
  if (warp == 3) {
    const bool bad = l8_prefix<MODE == LIN_WGRAD ? L8_KT : L8_M>(args, lane, row0, tile0);
    if (lane == 0) *bad_s = bad;
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
      __syncwarp();
      if constexpr (CUT) l8_cut(args, row0, order, unit0, num_pairs, lane, blockIdx.x == 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();                                // and the other's, before anything arrives there
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  // inconsistent split_sizes: nothing is computed (the error word says so)
  const int total = *bad_s ? 0 : CUT ? unit0[args.E] : l8_tiles<MODE>(args, tile0);
  const uint64_t lim = args.wait_limit_ns;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L8_REGS_FEW));
    if (lane == 0 && (warp == 0 || warp == 2) && !args.selftest_no_loads) {
      // ---------------- TMA producers (both CTAs): warp 0 the A side, warp 2 the B side ----------------
      const bool a_side = warp == 0;
      const uint32_t full_c0 = mapa_shared(smem_u32(full), 0);
      Ring cur;
      Tiles8 tiles(tile_ring, laid, taken);
      bool ok = true;
      for (;;) {
        ok = ok && wait_phase_inline(&laid[tiles.slot], tiles.ph, abort_s, args.err, SITE_LINEAR8 + 6, lim);
        if (!ok) break;
        const Tile8 tl = tile_ring[tiles.slot];
        mbar_arrive(&taken[tiles.slot]);
        tiles.advance();
        if (tl.blocks < 0) break;
        // A boxes of 128 m, or 32 rows where the CTA has no more; none where it has no m at all (what the
        // stage holds there instead only meets lanes that nobody stores)
        const auto a_bytes = [&](int r) {
          const int left = tl.cnt - r * 128;
          return left <= 0 ? 0 : !A_MN && left <= L8_SMALL ? L8_SMALL * L8_KT : L8_SIDE;
        };
        const int mine = a_bytes(int(rank)), m = tl.m0 + int(rank) * 128, nr = tl.n0 + int(rank) * (tl.n >> 1);
        for (int kt = 0; kt < tl.blocks; ++kt, cur.next()) {
          if (!wait_phase_inline(&empty[cur.st], cur.ph ^ 1u, abort_s, args.err, SITE_LINEAR8, lim)) {
            ok = false;
            break;
          }
          const uint32_t bar_c = full_c0 + uint32_t(cur.st) * 8u;
          uint8_t* pa = smem + cur.st * L8_STAGE;
          const int c = tl.c0 + kt * L8_KT;
          if (a_side) {
            if (rank == 0) mbar_arrive_expect_tx(&full[cur.st], uint32_t(a_bytes(0) + a_bytes(1) + 2 * L8_SIDE));
            if (mine != 0) tma_load_2d(pa, mine == L8_SIDE ? &tmA : &tmAs, A_MN ? m : c, A_MN ? c : m, bar_c);
          } else if (MODE == LIN_WGRAD) {
            tma_load_2d(pa + L8_SIDE, &tmB, nr, c, bar_c);
          } else {
            tma_load_3d(pa + L8_SIDE, &tmB, B_MN ? nr : c, B_MN ? c : nr, tl.e, bar_c);
          }
        }
      }
      pdl_launch_dependents();
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        // ---------------- MMA issuer (leader) ----------------
        // An MMA takes its pipe 128 clocks.  Issuing one took this thread 84 with operands computed on the way, and
        // 50 with constant ones, so the loop is unrolled over the ring's stages (the buffer is the stage's
        // parity).  A block has one wait (its operands and its buffer share a barrier) and one commit
        // (the stage is free when the sums are there).
        const uint64_t a_desc = A_MN ? desc_sw128_mn(smem_u32(smem), L8_SIDE) : desc_sw128(smem_u32(smem));
        const uint64_t b_desc = B_MN ? desc_sw128_mn(smem_u32(smem + L8_SIDE), L8_SIDE) : desc_sw128(smem_u32(smem + L8_SIDE));
        const uint32_t alo = uint32_t(a_desc), ahi = uint32_t(a_desc >> 32), blo = uint32_t(b_desc), bhi = uint32_t(b_desc >> 32);
        // 32 of the contraction, in the descriptors' 16-byte units: 32 bytes of a K-major row, four
        // 8-row groups (4 KB) of an MN-major block
        constexpr uint32_t A_K = A_MN ? 256 : 2, B_K = B_MN ? 256 : 2;
        bool ok = true, issued = false;
        uint32_t ph = 0;
        int at = 0;                              // the next block's stage
        Tiles8 tiles(tile_ring, laid, taken);
        for (;;) {
          ok = ok && wait_phase_inline(&laid[tiles.slot], tiles.ph, abort_s, args.err, SITE_LINEAR8 + 7, lim);
          if (!ok) break;
          int left = tile_ring[tiles.slot].blocks;
          const int last = tile_ring[tiles.slot].last;
          const uint32_t idesc = l8_idesc(A_MN, B_MN, tile_ring[tiles.slot].n);
          mbar_arrive(&taken[tiles.slot]);
          tiles.advance();
          if (left < 0) break;
          // the block in stage ST; false: the tile ends, or a wait gave up
          const auto block = [&](auto stage) {
            constexpr uint32_t ST = decltype(stage)::value, OFF = ST * (L8_STAGE >> 4);
            if (left == 0) return false;
            if (!wait_phase_inline(&full[ST], ph, abort_s, args.err, SITE_LINEAR8 + 1, lim)) {
              ok = false;
              return false;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (ST & 1) * L8_N;
            const int groups = left > 1 ? 4 : (last + 31) >> 5;           // of 32: all but the last are full blocks
            l8_mma<OFF, OFF, false>(acc, alo, ahi, blo, bhi, idesc);
            if (groups > 1) l8_mma<OFF + A_K, OFF + B_K, true>(acc, alo, ahi, blo, bhi, idesc);
            if (groups > 2) l8_mma<OFF + 2 * A_K, OFF + 2 * B_K, true>(acc, alo, ahi, blo, bhi, idesc);
            if (groups > 3) l8_mma<OFF + 3 * A_K, OFF + 3 * B_K, true>(acc, alo, ahi, blo, bhi, idesc);
            issued = true;
            tc_commit(&empty[ST]);
            --left;
            at = ST + 1 < L8_STAGES ? int(ST) + 1 : 0;
            ph ^= uint32_t(at == 0);
            return true;
          };
          while (ok && left > 0) {
            switch (at) {
              case 0: if (!block(std::integral_constant<uint32_t, 0>{})) break; [[fallthrough]];
              case 1: if (!block(std::integral_constant<uint32_t, 1>{})) break; [[fallthrough]];
              case 2: if (!block(std::integral_constant<uint32_t, 2>{})) break; [[fallthrough]];
              default: block(std::integral_constant<uint32_t, 3>{});
            }
          }
        }
        if (!ok && issued) {
          tc_commit(drain);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < 20000000ull) {
          }
        }
      }
    } else if (warp == 3) {
      if (lane == 0) {
        // ---------------- the pair's tiles, laid out for the others ----------------
        // A slot comes free when the tile before is done.  In the weight gradient that is below the limit, too: what
        // l8_cut weighs leaves no piece longer than two even shares, which is tiles / 38 of all rows on 76 pairs, and
        // tiles enough for that to be long want K + N above 2500, so that memory has room for some 110 million
        // rows: 0.3 s a tile (750 clocks a block of 128).
        Tiles8 tiles(tile_ring, laid, taken);
        for (int t = pair;; t = l8_after<MODE>(t, num_pairs)) {
          if (!wait_phase_inline(&taken[tiles.slot], tiles.ph ^ 1u, abort_s, args.err, SITE_LINEAR8 + 8, lim)) break;
          Tile8 tl;
          if (t < total) l8_decode<MODE, CUT>(args, row0, tile0, order, unit0, t, tl);
          else tl.blocks = -1;
          tile_ring[tiles.slot] = tl;
          mbar_arrive(&laid[tiles.slot]);
          tiles.advance();
          if (t >= total) break;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L8_REGS_MANY));
    // ---------------- sums (both CTAs) ----------------
    const int q = warp & 3;                      // lane quarter this warp may access
    const int col0 = ((warp - 4) >> 2) * 128;    // its columns of a buffer: one block of the B side
    const uint32_t tmem_row = tmem + (uint32_t(q * 32) << 16) + uint32_t(col0);
    // a block's buffer is handed back on the barrier of the block after the next, which takes it again
    const uint32_t full_c0 = mapa_shared(smem_u32(full), 0);
    const auto back = [&](int st) { l8_hand_back(full_c0 + uint32_t(st + 2 < L8_STAGES ? st + 2 : st + 2 - L8_STAGES) * 8u, lane); };
    l8_hand_back(full_c0, lane);                 // both buffers are free at first
    l8_hand_back(full_c0 + 8u, lane);
    const int cols = l8_cols<MODE>(args);
    const int64_t sa_step = MODE == LIN_WGRAD ? args.N : args.rows;
    const int64_t kbs = (args.K + 127) / 128, sb_step = MODE == LIN_FWD ? 1 : kbs;
    const float *sa = nullptr, *sb = nullptr;    // scales of the next block's: the lane's m, the warp's columns
    float fa0 = 0.f, fb0 = 0.f, fa1 = 0.f, fb1 = 0.f;        // asked for two blocks ahead, by turns
    int coming = 0;                              // blocks of the tile not yet asked for
    const auto ask = [&](float& fa, float& fb) {
      if (coming > 0) {
        fa = __ldg(sa);
        fb = __ldg(sb);
        sa += sa_step;
        sb += sb_step;
        --coming;
      }
    };
    Ring cur;                                    // a block's sums are there when its stage is free
    bool ok = true, live = false, end = false;
    Tiles8 tiles(tile_ring, laid, taken);
    const int at = int(rank) * 128 + q * 32;     // this warp's first of a tile's m
    int blocks = 0, e = 0, m = 0, n = 0, m_left = 0;         // the tile's, m and n from the warp's first on
    int piece = -1;
    // takes the next tile up, and asks for its first blocks' scales
    const auto take = [&]() {
      ok = wait_phase_warp_inline(&laid[tiles.slot], tiles.ph, abort_s, args.err, SITE_LINEAR8 + 6, lim);
      if (!ok) return;
      const Tile8* tl = &tile_ring[tiles.slot];
      blocks = tl->blocks;
      if (MODE == LIN_WGRAD) e = tl->e;
      if (CUT) piece = tl->piece;
      m = tl->m0 + at;
      n = tl->n0 + col0;
      m_left = tl->cnt - at;
      sa = tl->sa + min(at + lane, tl->cnt - 1);
      sb = tl->sb[col0 >> 7];
      __syncwarp();
      if (lane == 0) mbar_arrive(&taken[tiles.slot]);
      tiles.advance();
      end = blocks < 0;
      live = m_left > 0 && n < cols && !end;
      coming = live ? blocks : 0;
      ask(fa0, fb0);
      ask(fa1, fb1);
    };
    take();
    while (ok && !end) {
      if (!live) {
        // nobody's m or n: the buffers are handed back as they come
        for (int kt = 0; ok && kt < blocks; ++kt, cur.next()) {
          ok = wait_phase_warp_inline(&empty[cur.st], cur.ph, abort_s, args.err, SITE_LINEAR8 + 5, lim);
          if (ok) back(cur.st);
        }
        if (ok) take();
        continue;
      }
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // A block's columns come 64 at a time, and its buffer is handed back before the last 64 are added: the time
      // from the sums' arrival to that is on the buffer's way round, what comes after is not.  (32 at a time, the
      // last 32 added behind the next block's first load: 8192 rows, 4096 -> 16384, 416 us; this 404.)
      uint32_t p0[32], p1[32];
      if (blocks > 0) {
        wait_phase_warp_later(&empty[cur.st], cur.ph, abort_s, args.err, SITE_LINEAR8 + 4, lim, ok);
        tc_fence_after();
        tmem_ld32_async(tmem_row + (cur.st & 1) * L8_N, p0);
        tmem_ld32_async(tmem_row + (cur.st & 1) * L8_N + 32, p1);
      }
      const auto block = [&](int left, float& fa, float& fb) {
        const uint32_t src = tmem_row + (cur.st & 1) * L8_N;
        const float f = fa * fb;
        const float2 f2 = make_float2(f, f);
        tmem_wait_ld<32>(p0);
        tmem_wait_ld<32>(p1);
        l8_add(acc, p0, f2);
        tmem_ld32_async(src + 64, p0);
        l8_add(acc + 32, p1, f2);
        tmem_ld32_async(src + 96, p1);
        ask(fa, fb);
        const int freed = cur.st;
        cur.next();
        tmem_wait_ld<32>(p0);
        tmem_wait_ld<32>(p1);
        tc_fence_before();
        back(freed);
        l8_add(acc + 64, p0, f2);
        l8_add(acc + 96, p1, f2);
        if (left > 1) {
          wait_phase_warp_later(&empty[cur.st], cur.ph, abort_s, args.err, SITE_LINEAR8 + 4, lim, ok);
          tc_fence_after();
          tmem_ld32_async(tmem_row + (cur.st & 1) * L8_N, p0);
          tmem_ld32_async(tmem_row + (cur.st & 1) * L8_N + 32, p1);
        }
      };
      for (int left = blocks; left > 0; left -= 2) {
        block(left, fa0, fb0);
        if (left == 1) break;
        block(left - 1, fa1, fb1);
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const int rows = min(m_left, 32), columns = cols - n, e_out = e, m_out = m, n_out = n;
      if constexpr (CUT) {
        if (piece >= 0) {
          // partial sums, [n][the warp's 32 m]
          float* mine = args.pieces + int64_t(piece) * L8_PIECE + (int(rank) * L8_EPI_WARPS + warp - 4) * (32 * 128) + lane;
#pragma unroll
          for (int c = 0; c < 128; ++c) __stcg(mine + c * 32, acc[c]);
          take();
          continue;
        }
      }
      // Through the warp's own shared memory and TMA: meanwhile the tensor pipe fills the two buffers and stops, so
      // what counts is the warps' own time.  (2000 clocks a tile of it: taking the next tile up 600, these stores
      // 650, the fence 350, two boxes 420; rows read back and stored by 16 lanes each 3300, 32 bytes a lane to 32
      // rows 5000, a bulk copy a row 3300.  65536 rows, 2048 -> 2816: 316 and 334 us.)
      uint8_t* const box = smem + L8_OFF_OUT + (warp - 4) * 2 * L8_BOX;
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");      // the last tile's has been read
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 128; c += 8)
        *reinterpret_cast<uint4*>(box + (c >> 6) * L8_BOX + lane * 128 + ((((c >> 3) & 7) ^ (lane & 7)) << 4)) =
            make_uint4(pack_bf16x2(acc[c], acc[c + 1]), pack_bf16x2(acc[c + 2], acc[c + 3]),
                       pack_bf16x2(acc[c + 4], acc[c + 5]), pack_bf16x2(acc[c + 6], acc[c + 7]));
      take();                                    // while those land; its first scales are on their way
      if (MODE == LIN_WGRAD || rows == 32) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          l8_store<MODE>(&tmO, box, n_out, m_out, e_out);
          if (columns > 64) l8_store<MODE>(&tmO, box + L8_BOX, n_out + 64, m_out, e_out);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        continue;
      }
      // the last rows of an expert (behind them are the next one's): 16 lanes store a row's 256 bytes
      __syncwarp();
      const int chunk = lane & 15;
      if (chunk * 8 < columns) {                 // columns come in multiples of 16
        const uint8_t* from = box + (chunk >> 3) * L8_BOX;
        __nv_bfloat16* to = args.out + m_out * args.ldo + n_out + chunk * 8;
#pragma unroll 4
        for (int r = lane >> 4; r < rows; r += 2)
          *reinterpret_cast<uint4*>(to + r * args.ldo) =
              *reinterpret_cast<const uint4*>(from + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && *abort_s) {
    // A wait gave up in this CTA, of whichever warp: copies issued before land before the shared memory
    // goes (they take microseconds; bounded).
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  cluster_sync();                                // no CTA leaves while the pair's MMAs or arrivals may touch it
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// bf16 map of the output [batch][rows][inner] (batch 0: no such dimension) at pitch ld, boxes of 64 x 32.
bool l8_out_map(CUtensorMap* m, void* base, int64_t inner, int64_t rows, int64_t ld, int64_t batch) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(batch)};
  cuuint64_t strides[2] = {cuuint64_t(ld) * 2, cuuint64_t(ld) * cuuint64_t(rows) * 2};
  cuuint32_t box[3] = {64, 32, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, batch > 0 ? 3 : 2, base, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cut tiles' partial sums, added in the order of the rows.  A warp takes 16 n of 32 m; where a tile has many pieces,
// two, four or eight warps share them, every second, fourth or eighth each.
__global__ void __launch_bounds__(256) grouped_linear_fp8_join_kernel(const __grid_constant__ Linear8Args a) {
  __shared__ float red[8][16][33];
  __shared__ int4 plan[1 + L8_MAX_PIECES / 2];   // a cut tile has two pieces at least
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = ((a.N + L8_M - 1) / L8_M) * ((a.K + L8_N - 1) / L8_N);
  pdl_wait();
  if (tid <= L8_MAX_PIECES / 2) plan[tid] = __ldcg(reinterpret_cast<const int4*>(a.plan) + tid);
  __syncthreads();
  const int cuts = plan[0].x, units = plan[0].y;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int lo = 0, hi = cuts - 1;                   // largest slot whose units begin up to u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (plan[1 + mid].w <= u) lo = mid; else hi = mid - 1;
    }
    const int4 slot = plan[1 + lo];
    const int parts = slot.z, lg = l8_team(parts), team = 1 << lg, rem = u - slot.w;
    const int i = rem / (L8_SHARES << lg), share = rem & (L8_SHARES - 1), sub = (rem / L8_SHARES) & (team - 1);
    int m, n;
    l8_wgrad_tile(a, i, m, n);
    m += (share >> 3) * 128 + (share & 3) * 32;  // CTA, lane quarter
    n += ((share >> 2) & 1) * 128 + sub * (128 >> lg);
    if (m >= a.N || n >= a.K) continue;
    const int c0 = sub * (128 >> lg) + (warp >> lg) * 16;
    const float* from = a.pieces + int64_t(slot.y + i) * L8_PIECE + share * (32 * 128) + c0 * 32 + lane;
    float acc[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int p = warp & (team - 1); p < parts; p += team) {
      const float* s = from + int64_t(p) * tiles * L8_PIECE;
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[c] += __ldcg(s + c * 32);
    }
    __syncthreads();                             // the sums before have been read
#pragma unroll
    for (int c = 0; c < 16; ++c) red[warp][c][lane] = acc[c];
    __syncthreads();
    const int row = tid >> 3, c = (tid & 7) * 2;
    for (int g = 0; g < 8 >> lg; ++g) {
      float x = 0.f, y = 0.f;
      for (int w = g << lg; w < (g + 1) << lg; ++w) {
        x += red[w][c][row];
        y += red[w][c + 1][row];
      }
      if (m + row < a.N && n + g * 16 < a.K)     // K comes in multiples of 16
        *reinterpret_cast<uint32_t*>(a.out + (int64_t(slot.x) * a.N + m + row) * a.ldo + n + g * 16 + c) = pack_bf16x2(x, y);
    }
  }
}

template <int MODE, bool CUT = false>
cudaError_t l8_launch(const CUtensorMap& ma, const CUtensorMap& mas, const CUtensorMap& mb, const CUtensorMap& mo,
                      const Linear8Args& a, int grid, cudaStream_t st) {
  // attributes are per device: set and checked once on each device this process uses
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !ready[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, grouped_linear_fp8_kernel<MODE, CUT>);
    if (e != cudaSuccess) return e;
    // the warps' shares have to add up to what the block is launched with, or they would wait for ever
    if (f.numRegs != L8_REGS) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(grouped_linear_fp8_kernel<MODE, CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L8_SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(L8_THREADS);
  cfg.dynamicSmemBytes = L8_SMEM;
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
  return cudaLaunchKernelEx(&cfg, grouped_linear_fp8_kernel<MODE, CUT>, ma, mas, mb, mo, a);
}

}  // namespace

// The workspace: error word, arrivals of the four warps of the tiles of few rows, plan, pieces.
constexpr size_t kPlanBytes = 1280;
static_assert(kPlanBytes >= (1 + L8_MAX_PIECES / 2) * sizeof(int4), "a cut tile has two pieces at least");
constexpr size_t kPiecesAt = 256 + size_t(F8_MAX_PIECES) * 4 * sizeof(unsigned) + kPlanBytes;
static_assert(kPiecesAt % 256 == 0, "pieces start on whole lines");
size_t linear8_ws_bytes() {
  const size_t few = size_t(F8_MAX_PIECES) * F8_PIECE, wide = size_t(L8_MAX_PIECES) * L8_PIECE;
  return kPiecesAt + (few > wide ? few : wide) * sizeof(float);
}
void linear8_ws_parts(Linear8Args* a) {
  a->arrived = reinterpret_cast<unsigned*>(reinterpret_cast<uint8_t*>(a->err) + 256);
  a->plan = reinterpret_cast<int*>(a->arrived + F8_MAX_PIECES * 4);
  a->pieces = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a->err) + kPiecesAt);
}

cudaError_t launch_grouped_linear_fp8(int mode, const Linear8Args& args, const uint8_t* a_codes, const uint8_t* b_codes,
                                      cudaStream_t st, char* msg, size_t msg_len) {
  Linear8Args a = args;
  linear8_ws_parts(&a);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
  const int64_t nt = ((mode == LIN_FWD ? a.N : a.K) + L8_N - 1) / L8_N;
  const int64_t mt = mode == LIN_WGRAD ? int64_t(a.E) * ((a.N + L8_M - 1) / L8_M)
                                       : (a.rows < a.E ? a.rows : a.E) + a.rows / L8_M;
  const int64_t tiles = nt * mt;                 // no fewer than there are
  // The kernel for few rows: up to 16 an expert, and where a long contraction has so few tiles that cutting them
  // leaves an SM 24 blocks at most.  (Both measured, that one first.  16 rows, 4096 -> 28672, six of eight experts: 128
  // and 155 us; 32 rows, 2048 -> 1024, E = 8: 9.1 and 11.1, 128 rows 10.4 and 11.2, 256 rows 12.5 and 11.3; one row,
  // 14336 -> 4096: 26 and 55, 48 rows 33 and 55; with L2 emptied, 9 us of each: 512 rows, input gradient 8192 -> 512: 27
  // and 37, 200 rows, 4096 -> 1024, E = 4: 21 and 23, 64 rows, 4096 -> 4096: 23 and 23.  Near the rule's edge it takes
  // the slower one by a little: 4000 rows, input gradient 8192 -> 128: 37 and 35; 69 rows, 1952 -> 1584: 19 and 17; and
  // 48 rows, 3968 -> 4096 go to the other kernel, 17.7 us, where 4096 -> 4096 take 14.2 in a row.)  How the rows are split
  // only the device knows: 4096 rows, 2048 -> 2816, E = 256, all of one expert, whose weights are then read once for every 64
  // rows, take 149 us here, 16 rows more 29 in the other kernel; with 1 row to each of the other experts 353 and
  // 305; split evenly 289 and 297.
  const int64_t blocks = ((mode == LIN_FWD ? a.K : a.N) + L8_KT - 1) / L8_KT;
  const int64_t small = (((mode == LIN_FWD ? a.N : a.K) + 127) / 128) * ((a.rows < a.E ? a.rows : a.E) + a.rows / 64);
  if (mode != LIN_WGRAD && (a.rows <= int64_t(16) * a.E || (blocks >= 32 && small * blocks <= int64_t(24) * sms)))
    return launch_grouped_linear_fp8_few(mode, a, a_codes, b_codes, sms, st, msg, msg_len);
  CUtensorMap ma, mas, mb, mo;
  bool ok;
  if (mode == LIN_WGRAD) {
    const int64_t rows = (a.rows / L8_KT + a.E) * L8_KT;             // of the layout on blocks
    ok = l8_map(&ma, a_codes, a.N, rows, 0, 128) && l8_map(&mb, b_codes, a.K, rows, 0, 128);
    mas = ma;
  } else {
    const int64_t inner = mode == LIN_FWD ? a.K : a.N;
    ok = l8_map(&ma, a_codes, inner, a.rows, 0, 128) && l8_map(&mas, a_codes, inner, a.rows, 0, L8_SMALL) &&
         l8_map(&mb, b_codes, a.K, a.N, a.E, 128);
  }
  ok = ok && (mode == LIN_WGRAD ? l8_out_map(&mo, a.out, a.K, a.N, a.ldo, a.E)
                                : l8_out_map(&mo, a.out, mode == LIN_FWD ? a.N : a.K, a.rows, a.ldo, 0));
  if (!ok) {
    snprintf(msg, msg_len, "cuTensorMapEncodeTiled failed (rows %lld, K %d, N %d, E %d)", (long long)a.rows, a.K, a.N,
             a.E);
    return cudaErrorInvalidValue;
  }
  const int grid = 2 * int(tiles < pairs ? tiles : pairs);
  switch (mode) {
    case LIN_FWD: return l8_launch<LIN_FWD>(ma, mas, mb, mo, a, grid, st);
    case LIN_DGRAD: return l8_launch<LIN_DGRAD>(ma, mas, mb, mo, a, grid, st);
    default: break;
  }
  // Tiles may be cut where an expert has fewer than there are pairs, and rows enough to keep one busy long after the
  // others; whether they are, the kernel finds out.  (Both measured, that one first.  65000 rows, 256 -> 256, E = 1:
  // 31 and 214 us; 40000 rows, 1024 -> 512, E = 1: 40 and 134; 60000 rows, 512 -> 512, E = 4: 43 and 62; 4000 rows,
  // 256 -> 256: 22 and 25, 2048 rows 21 and 17; nothing to cut in 8000 rows, 1024 -> 2048, E = 8: 34 and 29.)
  const int64_t tiles_e = nt * ((a.N + L8_M - 1) / L8_M);
  if (tiles_e >= pairs || a.rows / L8_KT < 4 * L8_MIN_CUT) return l8_launch<LIN_WGRAD>(ma, mas, mb, mo, a, grid, st);
  e = l8_launch<LIN_WGRAD, true>(ma, mas, mb, mo, a, 2 * int(pairs), st);
  if (e != cudaSuccess) return e;
  return launch_pdl(grouped_linear_fp8_join_kernel, dim3(unsigned(sms) * 6), dim3(256), 0, st, a);
}

}  // namespace moe
