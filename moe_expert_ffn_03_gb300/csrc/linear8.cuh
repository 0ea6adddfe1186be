// What the two kernels of the grouped linear layers on 8-bit operands share: the experts' prefix sums, small
// copies on their way, 8-bit TMA maps.
#pragma once

#include "kernels.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int L8_KT = 128;                       // a block of the contraction: one stage
constexpr int L8_MAX_E = 256;
// Partial sums of tiles that are cut along the contraction: pieces of the kernel for few rows (128 x 64), and
// of the weight gradient's (256 x 256).
constexpr int F8_MAX_PIECES = 608, F8_PIECE = 128 * 64;
constexpr int L8_MAX_PIECES = 152, L8_PIECE = 256 * 256;

// One warp: the experts' first rows and first tiles of PER rows, eight experts per lane.  Sizes that do not fit
// in the rows are recorded (true) and taken as zeros.
template <int PER>
__device__ __forceinline__ bool l8_prefix(const Linear8Args& args, int lane, int* row0, int* tile0) {
  int rows[8], sum = 0, tiles = 0;
  int64_t all = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    const int s = e < args.E ? args.split_sizes[e] : 0;
    const bool wrong = s < 0 || s > args.rows;
    bad |= wrong;
    rows[i] = wrong ? 0 : s;
    all += rows[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
  bad = __any_sync(0xFFFFFFFFu, bad) || all > args.rows;
  if (lane == 0 && bad) report_error(args.err, MOE_ERR_DEVICE_BOUNDS, SITE_LINEAR8 + 9);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (bad) rows[i] = 0;
    sum += rows[i];
    tiles += (rows[i] + PER - 1) / PER;
  }
  int rs = sum, ts = tiles;                      // inclusive scans over the lanes
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
    ts += (rows[i] + PER - 1) / PER;
  }
  if (lane == 31 && args.E == L8_MAX_E) {
    row0[L8_MAX_E] = rs;
    tile0[L8_MAX_E] = ts;
  }
  return bad;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A copy of four bytes on its way to shared memory, and the wait until all but the last N groups of them are
// there.
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_left() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 8-bit map over row-major [batch][rows][inner] (batch 0: no such dimension), boxes of 128 bytes x box_rows
// with 128-byte swizzle.
bool l8_map(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t batch, int box_rows) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(batch)};
  cuuint64_t strides[2] = {cuuint64_t(inner), cuuint64_t(inner) * cuuint64_t(rows)};
  cuuint32_t box[3] = {128, cuuint32_t(box_rows), 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, batch > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe
