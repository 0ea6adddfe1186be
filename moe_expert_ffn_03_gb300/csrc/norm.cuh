// What the row norms (norm.cu, rmsnorm.cu) share: a thread's place in its row, how many threads and
// vectors a row takes, and how many blocks of a persistent grid a device holds.
#pragma once

#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "rows.cuh"

namespace moe {
namespace {

// Wide rows have at most 512 threads, and an SM holds that many (the kernels take up to 128
// registers): what keeps the memory busy is the ring below, not the number of threads.  Rows of
// single columns have no ring but 1024 threads an SM.
constexpr int MAX_TPR = 512;
constexpr int max_block(int vec) { return vec == 1 ? 1024 : MAX_TPR; }
// Rows a thread has on their way or in work at once (VEC > 1): up to three, as 512 threads' 16-byte
// pieces fit in shared memory (`pieces` per thread and row).
constexpr int ring_stages(int vec, int pieces) {
  if (vec == 1) return 0;
  const int most = 200 * 1024 / (MAX_TPR * pieces * 16);
  return most > 3 ? 3 : most;
}

// A thread's place: its row group, its first column (vector i is 32 * VEC columns further, a
// distance the compiler knows), and its slots of the ring, laid out per warp
// [stage][operand][vector][lane] of 16 bytes so that they too are constant distances apart.
template <int VEC, int NV, int OPS, int STG>
struct Place {
  int group, groups, t, col0;
  uint8_t* slot;
  __device__ __forceinline__ Place(int tpr, uint8_t* ring) {
    group = threadIdx.x / tpr;
    groups = blockDim.x / tpr;
    t = threadIdx.x - group * tpr;
    col0 = (t >> 5) * (32 * NV * VEC) + (t & 31) * VEC;
    slot = ring + (threadIdx.x >> 5) * (STG * OPS * NV * 512) + (threadIdx.x & 31) * 16;
  }
  __device__ __forceinline__ int col(int i) const { return col0 + i * (32 * VEC); }
  __device__ __forceinline__ uint8_t* piece(int st, int op, int i) const {
    return slot + st * (OPS * NV * 512) + (op * NV + i) * 512;
  }
  // zeros in every slot: vectors past a row's end are never copied and read as zeros
  __device__ __forceinline__ void clear() const {
#pragma unroll
    for (int k = 0; k < STG * OPS * NV; ++k) *reinterpret_cast<uint4*>(slot + k * 512) = make_uint4(0, 0, 0, 0);
  }
};

// 1 / sqrt(v), with a Newton step after the approximate instruction (0 gives Inf, Inf gives 0).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float n = r * fmaf(-0.5f * v * r, r, 1.5f);
  return v > 0.f && r > 0.f ? n : r;
}
constexpr int kMaxDevices = 64;

struct RowShape {
  int vec;       // columns of a vector
  int nv;        // vectors per thread
  int tpr;       // threads per row
  int block;     // threads per block
};

// Threads and vectors per row.  Wide rows, four vectors a thread in the forward pass, two in the
// backward (wide_nv): the sums over a row's threads and the addresses cost as much as a vector or
// two of arithmetic, and the kernels are bound by the instructions they issue as soon as a thread
// has only one (H = 1024: 297 instructions per vector with one, measured); with four, the
// backward's sums of the weights' gradients do not fit the registers (144 us, 106 with two, at
// T = 32768, H = 2048).  Shorter rows take fewer vectors so that a warp is not left half empty,
// longer ones more, up to 512 threads.  Single columns: four a thread up to 1024 threads, so that
// many threads' loads are in flight (H = 5001, backward: 800 us with 16 columns on 320 threads).
RowShape row_shape(int H, int vec, int wide_nv) {
  const int n = (H + vec - 1) / vec;              // vectors of a row
  const int most = max_block(vec);
  int nv = vec > 1 ? wide_nv : 4;
  while (vec > 1 && nv > 1 && 32 * (nv / 2) >= n) nv /= 2;
  while (nv * most < n) nv *= 2;
  const int tpr = (n + 32 * nv - 1) / (32 * nv) * 32;
  return RowShape{vec, nv, tpr, tpr > MAX_TPR ? tpr : MAX_TPR / tpr * tpr};
}

// How many blocks of a persistent grid each device holds at once, looked up once per row shape
// (block and shared memory follow from tpr), with the kernel's dynamic shared memory limit set.
struct Resident {
  std::atomic<int> blocks[kMaxDevices][max_block(1) / 32 + 1];
};
template <typename K>
cudaError_t resident_blocks(K* kernel, const RowShape& s, size_t smem, Resident& known, int64_t* out) {
  int dev = 0, sms = 0, per = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* slot = dev < kMaxDevices ? &known.blocks[dev][s.tpr / 32] : nullptr;
  if (slot != nullptr && (*out = slot->load(std::memory_order_acquire)) != 0) return cudaSuccess;
  // above the 48 KB (static memory included) that need no asking
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, s.block, smem);
  if (e != cudaSuccess) return e;
  if (per < 1) return cudaErrorInvalidConfiguration;
  *out = int64_t(sms) * per;
  if (slot != nullptr) slot->store(sms * per, std::memory_order_release);
  return cudaSuccess;
}

// Partial sums the backward may write: two blocks per SM (single columns; wide rows: one).
constexpr int kNormMaxParts = 304;

// Calls f with the vector width and count of a row shape as compile-time constants.
template <typename T, typename F>
cudaError_t with_shape(const RowShape& s, F f) {
  constexpr int W = kWide<T>;
  if (s.vec == 1) {
    if (s.nv == 4) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    if (s.nv == 8) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
  }
  if (s.nv == 1) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 1>{});
  if (s.nv == 2) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 2>{});
  if (s.nv == 4) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 4>{});
  if constexpr (W == 4) return f(std::integral_constant<int, W>{}, std::integral_constant<int, 8>{});
  return cudaErrorInvalidConfiguration;           // H above 16384
}

}  // namespace
}  // namespace moe
