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

// erfc(z) for z = |v| / sqrt(2), and e = exp(-z^2) (approximate exponential and reciprocal):
// erfc(z) = e t P(t) with t = 1 / (1 + 0.44 z), P a polynomial of degree 7 fitted to the smallest largest
// relative error over z >= 0: 6e-7 in float32, some thousandth of half a step of bfloat16, the type that the
// results of this form are rounded to (and of the size of a bias gradient's own rounding).
__device__ __forceinline__ float erfc_fast(float z, float* e) {
  const float t = rcp(fmaf(0.44f, z, 1.f));
  *e = ex2(z * z * -1.44269504088896341f);
  float p = 0.06916839629411697f;
  p = fmaf(p, t, -0.27031081914901733f);
  p = fmaf(p, t, 0.28519880771636963f);
  p = fmaf(p, t, -0.01120822038501501f);
  p = fmaf(p, t, 0.21193894743919373f);
  p = fmaf(p, t, 0.21821904182434082f);
  p = fmaf(p, t, 0.24876849353313446f);
  p = fmaf(p, t, 0.24822503328323364f);
  return p * t * *e;
}

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;

// Phi(v) = erfc(-v / sqrt(2)) / 2, and (DERIV) the density phi(v).  FAST: for results rounded to bfloat16.
template <bool FAST>
__device__ __forceinline__ float gauss_cdf(float v, float* density) {
  if (FAST) {
    float e;
    const float c = 0.5f * erfc_fast(fabsf(v) * kSqrtHalf, &e);
    *density = kInvSqrt2Pi * e;
    return v < 0.f ? c : 1.f - c;
  }
  *density = kInvSqrt2Pi * expf(-0.5f * v * v);
  return 0.5f * erfcf(-v * kSqrtHalf);
}

template <bool FAST>
__device__ __forceinline__ float activate(float v, int act) {
  if (act == kActSilu) return silu<FAST>(v);
  if (act == kActGelu) {
    float d;
    return v * gauss_cdf<FAST>(v, &d);
  }
  return v;
}

// The activation's derivative at v.
template <bool FAST>
__device__ __forceinline__ float activate_slope(float v, int act) {
  if (act == kActSilu) {
    const float s = FAST ? __fdividef(1.f, 1.f + __expf(-v)) : 1.f / (1.f + expf(-v));
    return s * fmaf(v, 1.f - s, 1.f);
  }
  if (act == kActGelu) {
    float d;
    const float c = gauss_cdf<FAST>(v, &d);
    return fmaf(v, d, c);
  }
  return 1.f;
}

// A launch whose CTAs may start before the one before it on the stream is done (see launch_second): they wait for it in
// wait_for_first before they touch memory.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned int)threads);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
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
// B as N rows of Kd, or (b_mn) as Kd rows of N.  Built: neither, b_mn alone, both; e4m3: neither.
struct ProductArgs {
  const void* a;
  const void* b;
  long long M, N, Kd;
  long long a_row, b_row;   // distance of rows in values
  bool a_mn, b_mn;
  Epilogue out;
  void* ws;
  int sm_count;
  DevStatus* status;
};
cudaError_t launch_product(const ProductArgs& p, int mat, cudaStream_t s);
// Bytes that it needs at p.ws; of the operands only sizes, strides and alignment count.
size_t product_ws(const ProductArgs& p, int mat);

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
};
cudaError_t launch_layer_norm_back(const LayerNormBackArgs& a, bool dy_bf16, bool x_bf16, cudaStream_t s);
size_t layer_norm_back_ws(long long rows, long long D, int sm_count);

}  // namespace vla
