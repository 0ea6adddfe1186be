// 8-bit tensors with one f32 scale per block of 128: quantizers of rows, of experts' rows along tokens and of
// weights, the values back, and rows packed by expert.
//
// Page "Efficient MoE Training for Biological Foundation Models", section "MoE训练的瓶颈与TE的对应能力"
// (8-bit operands with scales of blocks; the block of 128 with an f32 scale is an interface addition).
//
//   scale = amax / 448;  code = E4M3(value * (448 / amax))      amax: the block's largest magnitude
//   rows    blocks of 1 x 128,   scales [ceil(cols/128)][rows]
//   tokens  blocks of 128 x 1,   scales [blocks][cols]             rows laid out on blocks of 128 per expert
//   tiles   blocks of 128 x 128, scales [blocks][ceil(cols/128)]   the same, or rows of matrices as they are
// Scales lie along the index that the product keeps, so that its threads read neighbouring ones.
#include "fp8_block.cuh"
#include "kernels.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_MAX_E = 256;
constexpr int Q_ROWS = 8;                        // rows per thread of a tile of 128 x 128

// A thread's eight columns of a row (zeros past `left`), as floats: neighbours, or, where rows do not start on whole
// vectors, 16 apart, so that 16 lanes read and write neighbouring values.  (65536 x 2047 bf16 into rows and
// tokens: 203 us, with neighbours 400.)
template <typename T, bool WIDE>
struct Eight {
  static constexpr int STEP = WIDE ? 1 : 16;
  Raw<T, WIDE ? kWide<T> : 1> r[WIDE ? 8 / kWide<T> : 8];
  __device__ __forceinline__ void load(const T* p, int left) {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 8 / kWide<T>; ++i) {
        if (left > 0) r[i].load(p + i * kWide<T>);
        else r[i].zero();
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i * STEP < left) r[i].load(p + i * STEP);
        else r[i].zero();
      }
    }
  }
  __device__ __forceinline__ void get(float* v) const {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 8 / kWide<T>; ++i) r[i].get(v + i * kWide<T>);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i].get(v + i);
    }
  }
};
template <bool WIDE, int STEP>
__device__ __forceinline__ void put_codes(uint8_t* p, const uint32_t* q, int left) {
  if constexpr (WIDE) {
    if (left > 0) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * STEP < left) p[i * STEP] = uint8_t(q[i >> 2] >> (8 * (i & 3)));
  }
}

// The largest magnitudes (float bits) of a thread's rows over its eight columns, and of its columns over its rows.
// Of bf16 two values at a time, on the bits of their magnitudes, which order like them with NaN and Inf above
// all others.
template <typename T, bool WIDE>
__device__ __forceinline__ void maxima(const Eight<T, WIDE>* raw, uint32_t* rmax, uint32_t* cmax) {
  if constexpr (WIDE && sizeof(T) == 2) {
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Q_ROWS; ++i) {
      const uint4 q = raw[i].r[0].q;
      const uint32_t a = q.x & 0x7FFF7FFFu, b = q.y & 0x7FFF7FFFu, c = q.z & 0x7FFF7FFFu, d = q.w & 0x7FFF7FFFu;
      m[0] = __vmaxu2(m[0], a);
      m[1] = __vmaxu2(m[1], b);
      m[2] = __vmaxu2(m[2], c);
      m[3] = __vmaxu2(m[3], d);
      const uint32_t r = __vmaxu2(__vmaxu2(a, b), __vmaxu2(c, d));
      rmax[i] = max(r << 16, r & 0xFFFF0000u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cmax[2 * j] = m[j] << 16;
      cmax[2 * j + 1] = m[j] & 0xFFFF0000u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = 0;
#pragma unroll
    for (int i = 0; i < Q_ROWS; ++i) {
      float v[8];
      raw[i].get(v);
      rmax[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = abs_bits(v[j]);
        cmax[j] = max(cmax[j], a);
        rmax[i] = max(rmax[i], a);
      }
    }
  }
}

// Tiles of 128 rows x 128 columns, rows from an expert's first on (matrices of `mat_rows` rows: from the
// matrix's); 16 lanes hold a row's 128 columns, a thread eight rows in registers, so that a tile is read once
// for both of its formats.  A persistent grid, tiles of neighbouring columns one after the other.
// Memory and instructions bound it together (1000 a thread and tile): 65536 x 2048 bf16 into rows and tokens 97 us,
// 5.5 TB/s, with 32 warps an SM (24 warps and maxima by full butterflies 111; 40 warps 105, they spill; the next
// tile on its way to shared memory meanwhile 110: loads are not what it waits for).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(Q_THREADS, WIDE && sizeof(T) == 2 ? 4 : 2) block8_quantize_kernel(const __grid_constant__ Block8Args a) {
  __shared__ uint32_t colmaxes[2][Q_THREADS / 32][B8];       // by turns: the tile before may still be read
  __shared__ __align__(16) float colup[B8];
  __shared__ int row0[Q_MAX_E + 1], blk0[Q_MAX_E + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = tid >> 4;                      // rows sub, sub + 16, ... of a tile
  constexpr int STEP = Eight<T, WIDE>::STEP;     // between a thread's columns
  const int c8 = WIDE ? (tid & 15) * 8 : tid & 15;           // and the first of them
  pdl_wait();
  if (a.split_sizes != nullptr) {
    if (warp == 0) {
      // prefix sums of rows and blocks, eight experts per lane
      int rows[8], sum = 0, blocks = 0;
      int64_t all = 0;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        const int s = e < a.E ? a.split_sizes[e] : 0;
        const bool wrong = s < 0 || s > a.rows;
        bad |= wrong;
        rows[i] = wrong ? 0 : s;
        all += rows[i];
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
      bad = __any_sync(0xFFFFFFFFu, bad) || all > a.rows;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (bad) rows[i] = 0;                    // nothing is written then; the products record the error
        sum += rows[i];
        blocks += (rows[i] + B8 - 1) / B8;
      }
      int rs = sum, bs = blocks;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int r = __shfl_up_sync(0xFFFFFFFFu, rs, off), q = __shfl_up_sync(0xFFFFFFFFu, bs, off);
        if (lane >= off) {
          rs += r;
          bs += q;
        }
      }
      rs -= sum;
      bs -= blocks;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        if (e <= a.E) {
          row0[e] = rs;
          blk0[e] = bs;
        }
        rs += rows[i];
        bs += (rows[i] + B8 - 1) / B8;
      }
      if (lane == 31 && a.E == Q_MAX_E) {
        row0[Q_MAX_E] = rs;
        blk0[Q_MAX_E] = bs;
      }
    }
    __syncthreads();
  }
  const int cb = (a.cols + B8 - 1) / B8;
  const int per = a.mat_rows > 0 ? (a.mat_rows + B8 - 1) / B8 : 0;           // blocks of rows of a matrix
  const int64_t blocks = a.split_sizes != nullptr ? blk0[a.E]
                         : a.mat_rows > 0         ? int64_t(a.E) * per
                                                  : (a.rows + B8 - 1) / B8;
  // tile t is column block t % cb of row block t / cb, counted along without divisions
  int64_t blk = blockIdx.x / cb;
  int col_blk = int(blockIdx.x - blk * cb);
  const int step_blk = int(gridDim.x) / cb, step_col = int(gridDim.x) - step_blk * cb;
  const auto next = [&]() {
    blk += step_blk;
    col_blk += step_col;
    if (col_blk >= cb) {
      col_blk -= cb;
      ++blk;
    }
  };
  int turn = 0;
  for (; blk < blocks; next()) {
    const int c0 = col_blk * B8, left = a.cols - c0 - c8;
    int64_t first;                               // row of the source, and how many the tile has
    int cnt;
    if (a.split_sizes != nullptr) {
      int lo = 0, hi = a.E - 1;                  // largest e with blk0[e] <= blk
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (blk0[mid] <= blk) lo = mid; else hi = mid - 1;
      }
      const int off = int(blk - blk0[lo]) * B8;
      first = row0[lo] + off;
      cnt = min(B8, row0[lo + 1] - row0[lo] - off);
    } else if (a.mat_rows > 0) {
      const int mat = int(blk) / per, off = (int(blk) - mat * per) * B8;
      first = int64_t(mat) * a.mat_rows + off;
      cnt = min(B8, a.mat_rows - off);
    } else {
      first = blk * B8;
      cnt = int(a.rows - first < B8 ? a.rows - first : B8);
    }
    const int64_t trow = a.mat_rows > 0 ? first : blk * B8;                  // row of the second format's codes
    Eight<T, WIDE> raw[Q_ROWS];
    {
      const T* p = static_cast<const T*>(a.src) + (first + sub) * a.ld + c0 + c8;
#pragma unroll
      for (int i = 0; i < Q_ROWS; ++i) raw[i].load(p + i * 16 * a.ld, sub + 16 * i < cnt ? left : 0);
    }
    uint32_t rmax[Q_ROWS], cmax[8];
    maxima<T, WIDE>(raw, rmax, cmax);
    if (a.codes != nullptr) {
      // The row's 16 lanes share its eight pairs of divisions: lane j takes row j's, the others read it.  Maxima are
      // exchanged by halves, so that each step leaves a lane with half as many rows, in the end its own.
      uint32_t half[4], pair[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool up = lane & 4;
        const uint32_t give = __shfl_xor_sync(0xFFFFFFFFu, up ? rmax[i] : rmax[i + 4], 4);
        half[i] = max(up ? rmax[i + 4] : rmax[i], give);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool up = lane & 2;
        const uint32_t give = __shfl_xor_sync(0xFFFFFFFFu, up ? half[i] : half[i + 2], 2);
        pair[i] = max(up ? half[i + 2] : half[i], give);
      }
      uint32_t mine = max((lane & 1) ? pair[1] : pair[0], __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? pair[0] : pair[1], 1));
      mine = max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 8));
      const float my_up = Block8(mine).up;
      const int my_row = sub + 16 * (lane & 7);
      if ((lane & 8) == 0 && my_row < cnt) a.scales[int64_t(c0 / B8) * a.rows + first + my_row] = Block8::scale(mine);
      uint8_t* out = a.codes + (first + sub) * a.cols + c0 + c8;
#pragma unroll
      for (int i = 0; i < Q_ROWS; ++i) {
        const float up = __shfl_sync(0xFFFFFFFFu, my_up, (lane & 16) | i);
        float v[8];
        raw[i].get(v);
        const Block8 b(up);
        const uint32_t q[2] = {b.codes4(v), b.codes4(v + 4)};
        if (sub + 16 * i < cnt) put_codes<WIDE, STEP>(out + int64_t(i) * 16 * a.cols, q, left);
      }
    }
    if (a.tcodes == nullptr) continue;
    uint32_t (*const colmax)[B8] = colmaxes[turn];
    turn ^= 1;
    float ups[8];                                // the columns' factors
    if (a.tiles) {
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, cmax[j]);
      amax = __reduce_max_sync(0xFFFFFFFFu, amax);
      if (lane == 0) colmax[warp][0] = amax;
      __syncthreads();
      amax = 0;
#pragma unroll
      for (int w = 0; w < Q_THREADS / 32; ++w) amax = max(amax, colmax[w][0]);
      if (tid == 0) a.tscales[blk * cb + c0 / B8] = Block8::scale(amax);
      const float up = Block8(amax).up;
#pragma unroll
      for (int j = 0; j < 8; ++j) ups[j] = up;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[j] = max(cmax[j], __shfl_xor_sync(0xFFFFFFFFu, cmax[j], 16));
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) colmax[warp][c8 + j * STEP] = cmax[j];
      }
      __syncthreads();
      if (tid < B8) {
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < Q_THREADS / 32; ++w) amax = max(amax, colmax[w][tid]);
        colup[tid] = Block8(amax).up;
        if (c0 + tid < a.cols) a.tscales[blk * a.cols + c0 + tid] = Block8::scale(amax);
      }
      __syncthreads();
      if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) *reinterpret_cast<float4*>(ups + j) = *reinterpret_cast<const float4*>(colup + c8 + j);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) ups[j] = colup[c8 + j * STEP];
      }
    }
    // rows past the expert's last are zeros on its last block; a matrix has none
    const int out_rows = a.mat_rows > 0 ? cnt : B8;
    uint8_t* out = a.tcodes + (trow + sub) * a.cols + c0 + c8;
#pragma unroll
    for (int i = 0; i < Q_ROWS; ++i) {
      float v[8];
      raw[i].get(v);
      uint32_t q[2];
#pragma unroll
      for (int k = 0; k < 8; k += 4) q[k >> 2] = block8_codes4(v + k, ups + k);
      if (cnt < B8 && sub + 16 * i >= cnt) q[0] = q[1] = 0;      // (0 times a NaN factor is none)
      if (sub + 16 * i < out_rows) put_codes<WIDE, STEP>(out + int64_t(i) * 16 * a.cols, q, left);
    }
  }
}

// Values of codes: a warp takes four rows of 256 columns at a time, eight columns a lane: neighbours, or, where rows
// do not start on whole vectors, 32 apart.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(Q_THREADS) block8_dequantize_kernel(const __grid_constant__ Block8Back a) {
  constexpr int STEP = WIDE ? 1 : 32, HALVES = WIDE ? 1 : 2;     // blocks of 128 that a lane's columns lie in
  const int lane = threadIdx.x & 31, c8 = WIDE ? lane * 8 : lane;
  const int cb = (a.cols + B8 - 1) / B8;
  const int64_t fours = (a.rows + 3) / 4;
  pdl_wait();
  for (int col = blockIdx.y * 256 + c8; col - c8 < a.cols; col += gridDim.y * 256) {
    const int left = a.cols - col;
    if (left <= 0) continue;
    for (int64_t r4 = (int64_t(blockIdx.x) * Q_THREADS + threadIdx.x) >> 5; r4 < fours; r4 += (int64_t(gridDim.x) * Q_THREADS) >> 5) {
      const int64_t first = r4 * 4;
      uint32_t q[4][2];
      float s[8];                                // tokens: the columns', of all four rows (blocks begin on 128s); else [row][half]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = first + i < a.rows;
        q[i][0] = q[i][1] = 0;
        const uint8_t* p = a.codes + (first + i) * a.cols + col;
        if constexpr (WIDE) {
          if (in) {
            const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
            q[i][0] = w.x;
            q[i][1] = w.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (in && j * STEP < left) q[i][j >> 2] |= uint32_t(p[j * STEP]) << (8 * (j & 3));
        }
        if (a.format != MOE_FP8_TOKENS) {
          int64_t at = first + i, step = a.rows; // rows: of the first half, and to the second
          if (a.format == MOE_FP8_TILES) {
            int64_t rb = first / B8;
            if (a.mat_rows > 0 && in) {          // rows below 2^31
              const uint32_t row = uint32_t(first + i), mat = row / uint32_t(a.mat_rows);
              rb = int64_t(mat) * ((a.mat_rows + B8 - 1) / B8) + (row - mat * uint32_t(a.mat_rows)) / B8;
            }
            at = rb * cb;
            step = 1;
          }
          at += col / B8 * step;
#pragma unroll
          for (int h = 0; h < HALVES; ++h) s[i * HALVES + h] = in && h * B8 < left ? __ldg(a.scales + at + h * step) : 0.f;
        }
      }
      if (a.format == MOE_FP8_TOKENS) {
        const float* p = a.scales + first / B8 * a.cols + col;
        if constexpr (WIDE) {
          *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(p));
          *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(p + 4));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = j * STEP < left ? __ldg(p + j * STEP) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (first + i >= a.rows) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 f = e4m3x2_to_float2(q[i][k >> 2] >> (8 * (k & 3)));
          const float other = s[i * HALVES + (WIDE ? 0 : k >> 2)];
          v[k] = f.x * (a.format == MOE_FP8_TOKENS ? s[k] : other);
          v[k + 1] = f.y * (a.format == MOE_FP8_TOKENS ? s[k + 1] : other);
        }
        T* o = static_cast<T*>(a.dst) + (first + i) * a.ld + col;
        if constexpr (WIDE) {
          if constexpr (sizeof(T) == 2) {
            store_vec<8>(o, v);
          } else {
            store_vec<4>(o, v);
            store_vec<4>(o + 4, v + 4);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j * STEP < left) store_vec<1>(o + j * STEP, v + j);
        }
      }
    }
  }
}

// The same for rows that are dense but do not start on whole vectors: a thread takes a few times eight neighbouring
// values, whichever rows they are of.  (65536 x 2047 to bf16: rows 111 us, value by value 212; tokens, which have a
// scale a column, 187 and 232.)
template <typename T, bool TOKENS>
__global__ void __launch_bounds__(Q_THREADS) block8_dequantize_flat_kernel(const __grid_constant__ Block8Back a) {
  constexpr int UN = TOKENS ? 2 : 4, SCALES = TOKENS ? 8 : 2;
  const int64_t total = a.rows * a.cols, eights = (total + 7) / 8, step = int64_t(gridDim.x) * Q_THREADS;
  const int cb = (a.cols + B8 - 1) / B8;
  const auto scale = [&](int64_t row, int col) {
    if (a.format == MOE_FP8_ROWS) return __ldg(a.scales + int64_t(col / B8) * a.rows + row);
    int64_t rb = row / B8;
    if (a.mat_rows > 0) {                        // rows below 2^31
      const uint32_t r = uint32_t(row), mat = r / uint32_t(a.mat_rows);
      rb = int64_t(mat) * ((a.mat_rows + B8 - 1) / B8) + (r - mat * uint32_t(a.mat_rows)) / B8;
    }
    return __ldg(a.scales + rb * cb + col / B8);
  };
  pdl_wait();
  for (int64_t t = int64_t(blockIdx.x) * Q_THREADS + threadIdx.x; t < eights; t += UN * step) {
    uint2 q[UN];
    float s[UN][SCALES];                         // of every value (tokens); of the first, and from the next block or row on
    int turn[UN];                                // where that begins
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t at = (t + u * step) * 8;
      q[u] = make_uint2(0, 0);
      turn[u] = 8;
#pragma unroll
      for (int j = 0; j < SCALES; ++j) s[u][j] = 0.f;
      if (at >= total) continue;
      if (at + 8 <= total) {
        q[u] = __ldcg(reinterpret_cast<const uint2*>(a.codes + at));
      } else {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (at + j < total) w[j >> 2] |= uint32_t(a.codes[at + j]) << (8 * (j & 3));
        q[u] = make_uint2(w[0], w[1]);
      }
      const int64_t row = total < (int64_t(1) << 32) ? int64_t(uint32_t(at) / uint32_t(a.cols)) : at / a.cols;
      const int col = int(at - row * a.cols);
      if constexpr (TOKENS) {
        const float* p = a.scales + row / B8 * a.cols + col;
        const float* next = a.scales + (row + 1) / B8 * a.cols + (col - a.cols);     // the same of the next row's
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < total) s[u][j] = __ldg((col + j < a.cols ? p : next) + j);
        continue;
      }
      s[u][0] = scale(row, col);
      turn[u] = min(a.cols - col, B8 - (col & (B8 - 1)));
      if (turn[u] < 8 && at + turn[u] < total) s[u][1] = col + turn[u] < a.cols ? scale(row, col + turn[u]) : scale(row + 1, 0);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int64_t at = (t + u * step) * 8;
      if (at >= total) continue;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 f = e4m3x2_to_float2((k < 4 ? q[u].x : q[u].y) >> (8 * (k & 3)));
        v[k] = f.x * (TOKENS ? s[u][k % SCALES] : k < turn[u] ? s[u][0] : s[u][1]);
        v[k + 1] = f.y * (TOKENS ? s[u][(k + 1) % SCALES] : k + 1 < turn[u] ? s[u][0] : s[u][1]);
      }
      T* o = static_cast<T*>(a.dst) + at;
      if (at + 8 > total) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (at + j < total) store_vec<1>(o + j, v + j);
      } else if constexpr (sizeof(T) == 2) {
        store_vec<8>(o, v);
      } else {
        store_vec<4>(o, v);
        store_vec<4>(o + 4, v + 4);
      }
    }
  }
}

// Rows of tokens copied to their places by expert, dense (row_of has every expert's rows on multiples of 128).  A
// warp takes a token: its codes once from memory, k times out; then the scales of its blocks.
__global__ void __launch_bounds__(Q_THREADS) block8_pack_kernel(const __grid_constant__ Block8Pack a) {
  __shared__ int start[Q_MAX_E], pad_start[Q_MAX_E], size[Q_MAX_E];
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (threadIdx.x < 32) {
    int rows[8], sum = 0, padded = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      rows[i] = e < a.E ? a.split_sizes[e] : 0;
      sum += rows[i];
      padded += (rows[i] + B8 - 1) / B8 * B8;
    }
    int rs = sum, ps = padded;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int r = __shfl_up_sync(0xFFFFFFFFu, rs, off), q = __shfl_up_sync(0xFFFFFFFFu, ps, off);
      if (lane >= off) {
        rs += r;
        ps += q;
      }
    }
    rs -= sum;
    ps -= padded;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      start[e] = rs;
      pad_start[e] = ps;
      size[e] = rows[i];
      rs += rows[i];
      ps += (rows[i] + B8 - 1) / B8 * B8;
    }
  }
  __syncthreads();
  const int64_t rows = int64_t(a.T) * a.k;
  const int cb = (a.cols + B8 - 1) / B8;
  for (int64_t t = (int64_t(blockIdx.x) * Q_THREADS + threadIdx.x) >> 5; t < a.T; t += (int64_t(gridDim.x) * Q_THREADS) >> 5) {
    int pos = -1;
    if (lane < a.k) {
      const int64_t pair = t * a.k + lane;
      const int e = a.idx[pair], r = a.row_of[pair];
      if (e >= 0 && e < a.E && r >= pad_start[e] && r - pad_start[e] < size[e]) pos = start[e] + (r - pad_start[e]);
      if (pos < 0 || pos >= rows) {
        report_error(a.err, MOE_ERR_DEVICE_BOUNDS, SITE_FP8_BLOCK);
        pos = -1;
      } else {
        a.prob_rows[pos] = a.prob[pair];
      }
      a.pos_of[pair] = pos;
    }
    int to[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = __shfl_sync(0xFFFFFFFFu, pos, j);
    for (int c = lane * 16; c < a.cols; c += 512) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(a.codes + t * a.cols + c));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (to[j] >= 0) *reinterpret_cast<uint4*>(a.codes_out + int64_t(to[j]) * a.cols + c) = v;
    }
    for (int b = lane; b < cb; b += 32) {
      const float s = __ldg(a.scales + int64_t(b) * a.T + t);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (to[j] >= 0) a.scales_out[b * rows + to[j]] = s;
    }
  }
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

}  // namespace

cudaError_t launch_block8_quantize(const Block8Args& a, bool f32, cudaStream_t st) {
  int sms = 0;
  if (const cudaError_t e = sm_count(&sms); e != cudaSuccess) return e;
  const int64_t cb = (a.cols + B8 - 1) / B8;
  const int64_t tiles = cb * (a.mat_rows > 0 ? int64_t(a.E) * ((a.mat_rows + B8 - 1) / B8) : a.rows / B8 + (a.split_sizes ? a.E : 1));
  const int64_t most = int64_t(sms) * 8;
  const dim3 grid(unsigned(tiles < most ? tiles : most));
  const bool wide = a.cols % 8 == 0 && a.ld % 8 == 0;
  if (f32)
    return wide ? launch_pdl(block8_quantize_kernel<float, true>, grid, dim3(Q_THREADS), 0, st, a)
                : launch_pdl(block8_quantize_kernel<float, false>, grid, dim3(Q_THREADS), 0, st, a);
  return wide ? launch_pdl(block8_quantize_kernel<__nv_bfloat16, true>, grid, dim3(Q_THREADS), 0, st, a)
              : launch_pdl(block8_quantize_kernel<__nv_bfloat16, false>, grid, dim3(Q_THREADS), 0, st, a);
}

cudaError_t launch_block8_dequantize(const Block8Back& a, bool f32, cudaStream_t st) {
  int sms = 0;
  if (const cudaError_t e = sm_count(&sms); e != cudaSuccess) return e;
  const int64_t across = (a.cols + 255) / 256, gy = across < 1024 ? across : 1024;
  const int64_t need = ((a.rows + 3) / 4 + Q_THREADS / 32 - 1) / (Q_THREADS / 32);
  const int64_t most = (int64_t(sms) * 8 + gy - 1) / gy;
  const dim3 grid(unsigned(need < most ? need : most), unsigned(gy));
  const bool wide = a.cols % 8 == 0 && a.ld % 8 == 0;
  // Eight values lie in two rows at most, and in two blocks where a row's last block has eight or more.
  if (!wide && a.ld == a.cols && a.cols >= 8 && (a.format == MOE_FP8_TOKENS || (a.cols - 1) % B8 >= 7)) {
    const int64_t blocks = (a.rows * a.cols + 8 * Q_THREADS - 1) / (8 * Q_THREADS), cap = int64_t(sms) * 6;
    const dim3 flat(unsigned(blocks < cap ? blocks : cap));
    if (a.format == MOE_FP8_TOKENS)
      return f32 ? launch_pdl(block8_dequantize_flat_kernel<float, true>, flat, dim3(Q_THREADS), 0, st, a)
                 : launch_pdl(block8_dequantize_flat_kernel<__nv_bfloat16, true>, flat, dim3(Q_THREADS), 0, st, a);
    return f32 ? launch_pdl(block8_dequantize_flat_kernel<float, false>, flat, dim3(Q_THREADS), 0, st, a)
               : launch_pdl(block8_dequantize_flat_kernel<__nv_bfloat16, false>, flat, dim3(Q_THREADS), 0, st, a);
  }
  if (f32)
    return wide ? launch_pdl(block8_dequantize_kernel<float, true>, grid, dim3(Q_THREADS), 0, st, a)
                : launch_pdl(block8_dequantize_kernel<float, false>, grid, dim3(Q_THREADS), 0, st, a);
  return wide ? launch_pdl(block8_dequantize_kernel<__nv_bfloat16, true>, grid, dim3(Q_THREADS), 0, st, a)
              : launch_pdl(block8_dequantize_kernel<__nv_bfloat16, false>, grid, dim3(Q_THREADS), 0, st, a);
}

cudaError_t launch_block8_pack(const Block8Pack& a, cudaStream_t st) {
  int sms = 0;
  if (const cudaError_t e = sm_count(&sms); e != cudaSuccess) return e;
  const int64_t blocks = (int64_t(a.T) + Q_THREADS / 32 - 1) / (Q_THREADS / 32), most = int64_t(sms) * 8;
  return launch_pdl(block8_pack_kernel, dim3(unsigned(blocks < most ? blocks : most)), dim3(Q_THREADS), 0, st, a);
}

}  // namespace moe
