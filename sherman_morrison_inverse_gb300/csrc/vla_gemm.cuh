// Shared by the tensor-core products: the epilogue's arguments and its last step, bounded waits, matrix descriptors,
// operands as TMA reads them.
#pragma once

#include <cuda.h>   // CUtensorMap and the encode entry point's types (resolved at run time)

#include "vla_dense.cuh"
#include "vla_tc.cuh"

namespace vla {
namespace gemm {

// Stages that add up in tensor memory before float32 registers take the sums over: of float32 results, and of others where a
// share of Kd is longer than kWhole stages.
constexpr int kPart = 4, kLongPart = 64, kWhole = 128;

// One product of a launch.
struct GemmArgs {
  long long M, N;
  int tiles_m, tiles_n, splits, tiles;   // tiles: of all splits
  int k_iters, passes;      // stages of one pass over Kd; passes over the terms
  int part;                 // stages that add up in tensor memory
  float* partial;           // [splits][M][part_row] where splits > 1
  long long part_row;       // N, rounded up to 8
  Epilogue out;
  bool direct;                    // rows of y, pre, residual on 32-byte boundaries, N in whole pieces of 32 bytes
  bool y_vec, res_vec, pre_vec;   // four values at a time
  unsigned long long limit;       // of a wait, in ns: the handle's and 4 us for every stage of a tile; 0: the epilogue gives up
  DevStatus* status;
};

// Passes over the terms of the operands: float32 takes (a, b) = 3-1, 1-3, 2-2, 2-1, 1-2, 1-1.
constexpr int kPasses = 6;
__device__ __forceinline__ int term_a(int pass) { return (0x201100 >> (4 * (5 - pass))) & 3; }
__device__ __forceinline__ int term_b(int pass) { return (0x021010 >> (4 * (5 - pass))) & 3; }

// Stages [k, part_end) of a range that ends at k1 add up in tensor memory; parts are added to float32 registers.
__device__ __forceinline__ int part_end(const GemmArgs& g, int k, int k1) {
  const int last = (g.passes - 1) * g.k_iters, end = k < last ? last : k + g.part;
  return end < k1 ? end : k1;
}
// The first stage of a share of Kd.  (The product is below 2^32: at most 2^24 stages, 6 passes, 32 shares.)
__device__ __forceinline__ int k_begin(const GemmArgs& g, int split) {
  const uint32_t at = (uint32_t)(g.k_iters * g.passes) * (uint32_t)split;
  return (int)(g.splits == 1 ? at : at / (uint32_t)g.splits);
}

// Matrix descriptor of a 128-byte-swizzled operand: `lbo` bytes between blocks of 64 values in the adjacent dimension of
// a transposed operand, 1024 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Waits for a phase; false when the limit runs out or the CTA has failed.  The scope is the CTA's also where another CTA completes the
// phase: what these phases order are copies and products, and reads of tensor memory behind tcgen05's own fences; no thread
// reads memory here that a thread of another CTA wrote.  (With the cluster's scope every wait empties the first-level cache and
// every arrival waits for the thread's stores: 8192 x 8192 x 64 bfloat16 58 us, 46 without.)
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, unsigned long long limit, volatile uint32_t* failed) {
  const unsigned long long start = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*failed) return false;
    if (globaltimer_ns() - start > limit) {
      *failed = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, unsigned long long limit, volatile uint32_t* failed) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, limit, failed);
}
// The same for a warp whose lanes go on together to instructions that a whole warp has to execute (tcgen05.ld): each lane tries for
// itself, and one that is the last to look can see the phase where the others have given up.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, unsigned long long limit, volatile uint32_t* failed) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, limit, failed));
}

// Four adjacent values of a row, those from `left` on absent.
template <typename T>
__device__ __forceinline__ Vec<T, 4> load4(const T* p, bool vec, int left) {
  if (vec && left >= 4) return ld_vec<T, 4>(p);
  Vec<T, 4> x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = i < left ? p[i] : from_f32<T>(0.f);
  return x;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, bool vec, int left, const float (&v)[4]) {
  if (vec && left >= 4) {
    Vec<T, 4> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = from_f32<T>(v[i]);
    st_vec<T, 4>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = from_f32<T>(v[i]);
  }
}

// bias and weight scale of four columns
struct Columns {
  float bias[4], scale[4];
};
__device__ __forceinline__ Columns columns_of(const Epilogue& e, long long n, int left) {
  Columns c;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c.bias[j] = e.bias && j < left ? e.bias[n + j] : 0.f;
    c.scale[j] = e.w_scale && j < left ? e.w_scale[n + j] : 1.f;
  }
  return c;
}
// Four sums of row m to pre and y.
template <typename T>
__device__ __forceinline__ void out4(const GemmArgs& g, float (&v)[4], const Columns& c, const Vec<T, 4>& res, long long m,
                                     long long n, int left) {
  const Epilogue& e = g.out;
  const float xs = e.x_scale ? e.x_scale[m] : 1.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j] * xs, c.scale[j], c.bias[j]);
  if (e.pre) store4<T>(static_cast<T*>(e.pre) + m * e.pre_row + n, g.pre_vec, left, v);
  if (e.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) unpair(activate2<sizeof(T) == 2>(pair(v[j], v[j + 1]), e.act), v[j], v[j + 1]);
  }
  if (e.residual) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += to_f32<T>(res.v[j]);
  }
  store4<T>(static_cast<T*>(e.y) + m * e.y_row + n, g.y_vec, left, v);
}

// An operand as it lies in memory: rows of `cols` adjacent values.
struct Operand {
  const void* p;
  long long rows, cols, row;   // row: distance of rows in values
  int size;                    // bytes a value
  bool mn;                     // what is adjacent is M or N, not Kd
  bool pack;                   // TMA reads a copy
  size_t bytes;                // of the copy
  long long out_row;
};
// side: M or N.
Operand operand(const void* p, long long side, long long kd, long long row, bool mn, int size);
// The map of its tiles: box_x adjacent values x box_y rows.  base: where it lies, or its copy.
bool encode(CUtensorMap* m, const Operand& o, const void* base, int box_x, int box_y);

// Makes the copies of up to four operands.
struct Copies {
  Operand o[4];
  void* to[4];
  int count;
};
cudaError_t pack(const Copies& c, int sm_count, cudaStream_t s);

// What the epilogue needs, but for the tiles.
GemmArgs args_of(const ProductArgs& p);

// Products with w's rows in the tensor cores' long dimension (vla_gemm_tokens.cu).
struct TokensPlan {
  int rows, splits;   // tokens a tile; shares of Kd, one CTA of a cluster each
};
TokensPlan tokens_plan(long long M, long long N, long long w_values, int all_iters, int sm_count);
cudaError_t launch_tokens(const TokensPlan& t, GemmArgs g, const Operand& x, const Operand& w, const void* x_at, const void* w_at,
                          cudaStream_t s);

}  // namespace gemm

// Few rows of x, on CUDA cores (neither operand MN); no workspace.
cudaError_t launch_few_rows(const ProductArgs& p, int mat, cudaStream_t s);

}  // namespace vla
