// Shared by the matrix products with an epilogue and the layer norm: arguments, activations and what
// happens to an accumulator on its way out.
#pragma once

#include <cuda_fp8.h>

#include "vla_layer.cuh"

namespace vla {

enum Act { kActNone = 0, kActSilu = 1, kActGelu = 2 };   // vla_act_t
enum Mat { kMatF32 = 0, kMatBf16 = 1, kMatE4m3 = 2 };    // vla_mat_t

template <>
__device__ __forceinline__ float to_f32<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) { return static_cast<float>(x); }

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

// Phi(v) = erfc(-v / sqrt(2)) / 2 and e = exp(-v^2 / 2) of a pair, for results rounded to bfloat16 (approximate exponential and
// reciprocal).  With z = |v| / sqrt(2), erfc(z) = e t P(t), t = 1 / (1 + 0.44 z), P a polynomial of degree 7 fitted to the
// smallest largest relative error over z >= 0.  The coefficients here are halved: c = Phi(-|v|).  In float32 c is off by
// 6.4e-7 of itself up to |v| = 1, 8.2e-7 to 3, 1.3e-6 to 5, 3.1e-6 to 8, 7.2e-6 to 12.6 (v v is rounded before the
// exponential), and by 3.1e-7 of 1 at most: some thousandth of half a step of bfloat16.  A bias gradient is float32 and made
// from it: its terms are off by 5e-7 of theirs where |v| < 1, 1.4e-6 below 8, measured over all values of bfloat16.
__device__ __forceinline__ uint64_t gauss_cdf2(uint64_t v, uint64_t* e) {
  const uint64_t a = v & 0x7fffffff7fffffffull;
  float x, y;
  unpair(fma2(a, both(0.44f * kSqrtHalf), both(1.f)), x, y);
  const uint64_t t = pair(rcp(x), rcp(y));
  unpair(mul2(mul2(v, v), both(-0.72134752044448170f)), x, y);   // log2(e) / 2
  *e = pair(ex2(x), ex2(y));
  uint64_t p = both(0.034584198147058487f);
  p = fma2(p, t, both(-0.13515540957450867f));
  p = fma2(p, t, both(0.14259940385818481f));
  p = fma2(p, t, both(-0.005604110192507505f));
  p = fma2(p, t, both(0.10596947371959686f));
  p = fma2(p, t, both(0.10910952091217041f));
  p = fma2(p, t, both(0.12438424676656723f));
  p = fma2(p, t, both(0.12411251664161682f));
  const uint64_t c = mul2(mul2(p, t), *e);
  float cx, cy, vx, vy;
  unpair(c, cx, cy);
  unpair(fma2(c, both(-1.f), both(1.f)), x, y);
  unpair(v, vx, vy);
  return pair(vx < 0.f ? cx : x, vy < 0.f ? cy : y);
}

// 1 / (1 + e^-v) for float32 results: expf's 2 ulp and the approximate reciprocal's 1, where a rounded division takes
// eight instructions (21459 x 440 x 72 float32 with silu: 67 us with it).  0 below -87.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + expf(-v)); }

// The activation of a pair.  FAST: for results rounded to bfloat16.
template <bool FAST>
__device__ __forceinline__ uint64_t activate2(uint64_t v, int act) {
  if (act == kActNone) return v;
  if (FAST) {
    if (act == kActSilu) return silu2(v);
    uint64_t e;
    return mul2(v, gauss_cdf2(v, &e));
  }
  float x, y;
  unpair(v, x, y);
  if (act == kActSilu) return pair(x * sigmoid(x), y * sigmoid(y));
  return pair(x * (0.5f * erfcf(-x * kSqrtHalf)), y * (0.5f * erfcf(-y * kSqrtHalf)));
}

__device__ __forceinline__ float slope_of(float v, int act) {
  if (act == kActSilu) {
    const float s = sigmoid(v);
    return s * fmaf(v, 1.f - s, 1.f);
  }
  return fmaf(v, kInvSqrt2Pi * expf(-0.5f * v * v), 0.5f * erfcf(-v * kSqrtHalf));
}

// Its derivative (act is not kActNone).
template <bool FAST>
__device__ __forceinline__ uint64_t slope2(uint64_t v, int act) {
  float x, y;
  if (!FAST) {
    unpair(v, x, y);
    return pair(slope_of(x, act), slope_of(y, act));
  }
  if (act == kActSilu) {
    unpair(mul2(v, both(-1.44269504088896341f)), x, y);
    unpair(add2(pair(ex2(x), ex2(y)), both(1.f)), x, y);
    const uint64_t s = pair(rcp(x), rcp(y));
    return mul2(s, fma2(v, fma2(s, both(-1.f), both(1.f)), both(1.f)));
  }
  uint64_t e;
  const uint64_t cdf = gauss_cdf2(v, &e);
  return fma2(v, mul2(e, both(kInvSqrt2Pi)), cdf);
}

template <bool FAST>
__device__ __forceinline__ float activate(float v, int act) {
  float x, y;
  unpair(activate2<FAST>(pair(v, 0.f), act), x, y);
  return x;
}

// A launch whose CTAs may start before the one before it on the stream is done (see launch_second).  Every thread of them waits for
// it in wait_for_first before it touches memory, and only a launch of the same call may lie before, of which the same holds:
// so what is done when it is done includes everything earlier on the stream.  follows: false for the first launch of a call.
template <typename... P, typename... A>
cudaError_t launch_after(bool follows, void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned int)threads);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = follows ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, static_cast<A&&>(args)...);
}

// What happens to the accumulator of output (m, n):
//   v = acc * x_scale[m] * w_scale[n] + bias[n];  pre <- v;  y <- act(v) + residual
struct Epilogue {
  const float* x_scale;   // [M] or NULL
  const float* w_scale;   // [N] or NULL
  const float* bias;      // [N] or NULL
  const void* residual;   // y's type, or NULL; may be y itself
  void* pre;              // y's type, or NULL
  void* y;                // bfloat16 or float32
  long long res_row, pre_row, y_row;
  int act;
  bool y_bf16;
};

// C [M, N] = sum over Kd of A B.  A lies in memory as M rows of Kd adjacent values, or (a_mn) as Kd rows of M;
// B as N rows of Kd, or (b_mn) as Kd rows of N.  Built: neither; b_mn alone and both, as a gradient's dx and dw;  e4m3: neither MN.
struct ProductArgs {
  const void* a;
  const void* b;
  long long M, N, Kd;
  long long a_row, b_row;   // distance of rows in values
  bool a_mn, b_mn;
  bool follows;             // a launch of the same call, whose CTAs say all_started, lies before on the stream
  Epilogue out;
  void* ws;
  int sm_count;
  DevStatus* status;
  unsigned long long wait_limit;   // of a wait, in ns (0: its self-test)
};
// One or two products (count) that may run together, of one type and with one workspace (p[0].ws).
cudaError_t launch_products(const ProductArgs* p, int count, int mat, cudaStream_t s);
// Bytes that they need there; of the operands only sizes, strides, alignment and which are the same count.
size_t products_ws(const ProductArgs* p, int count, int mat);

// g = dy * act'(pre) [M, N] (when pre is not NULL), and db[n] = sum_m g (when db is not NULL; float32, from g
// before it is rounded).
struct SlopeArgs {
  const void* dy;
  const void* pre;
  void* g;            // dense [M, N] with rows of g_row, or NULL without pre
  float* db;
  float* partial;     // [blocks of rows][N]
  long long M, N, dy_row, pre_row, g_row;
  int act;
  int sm_count;
};
cudaError_t launch_slope(const SlopeArgs& a, bool bf16, cudaStream_t s);
size_t slope_ws(long long M, long long N, int sm_count);

struct LayerNormArgs {
  const void* x;
  const float* w;
  const float* b;       // or NULL
  void* residual;       // or NULL; updated in place
  void* y;
  float* stats;         // [rows][2] mean, reciprocal deviation; or NULL
  long long rows, D, x_row, res_row, y_row;
  float eps;
  bool res_bf16;
  int sm_count;
};
cudaError_t launch_layer_norm(const LayerNormArgs& a, bool bf16, cudaStream_t s);

struct LayerNormBackArgs {
  const void* dy;
  const void* x;        // what was normalised: the residual stream's type, like dres and dx
  const float* w;
  const float* stats;
  const void* dres;     // or NULL
  void* dx;
  float* dw;
  float* db;            // or NULL
  float* partial;
  long long rows, D, dy_row, x_row, dres_row, dx_row;
  int sm_count;
  DevStatus* status;
  unsigned long long wait_limit;   // of a wait, in ns (0: its self-test)
};
cudaError_t launch_layer_norm_back(const LayerNormBackArgs& a, bool dy_bf16, bool x_bf16, cudaStream_t s);
size_t layer_norm_back_ws(long long rows, long long D, int sm_count);

}  // namespace vla
