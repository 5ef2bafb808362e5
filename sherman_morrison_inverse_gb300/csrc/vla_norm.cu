// Root-mean-square norm with the residual's addition and an output in 8 bits:
//   r = x + residual (float32; residual <- r in its own type),  v = r / sqrt(mean(r^2) + eps) * w,
//   and either v in x's type, or codes q with scale = max|v| / 448 (e4m3) or / 127 (integers) over a
//   row or over every 128 values, q = v * (1 / scale) rounded to nearest even.
// A scale below the smallest normal float32 (a row of zeros) is 1; a NaN makes its scale NaN.
//
// One pass: a row stays in the registers of its threads between the sum of squares, the maximum and
// the rounding, so x and the residual are read once and every output written once (7 bytes a value
// for bfloat16 with a residual and e4m3); memory bound.  A row has TPR threads (a warp at least),
// each with NV vectors of VEC adjacent values (16 bytes where alignment allows); short rows share
// a block.  Sums run in float32 in a fixed order: the same bits every time.
#include "vla.h"
#include "vla_layer.cuh"

namespace vla {
namespace {

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) { return MAX ? max_nan(a, b) : a + b; }

// Sum or maximum over the threads of a row (warps [w0, w0 + wn) of the block; `part` has a place
// for each warp of the block).  Every thread of the block calls it.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* part, int w0, int wn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (wn == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();   // `part` may still be read from the previous call
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < wn ? part[w0 + lane] : 0.f;   // 0 is neutral: sums of squares and magnitudes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int OUT>
__device__ __forceinline__ unsigned char code(float v) {
  if (OUT == VLA_OUT_E4M3) return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  const int q = __float2int_rn(v);   // NaN gives 0 (its scale is NaN)
  return (unsigned char)(signed char)(q > 127 ? 127 : q < -127 ? -127 : q);
}

// RES: 0 none, 1 bfloat16, 2 float32
template <typename T, int RES, int OUT, int VEC, int NV>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a, int tpr, int rows_per_cta) {
  using R = typename std::conditional<RES == 1, __nv_bfloat16, float>::type;
  __shared__ float part[32];
  __shared__ float gmax[VEC == 1 && OUT != VLA_OUT_IO ? NV * 32 : 1];
  const int slot = threadIdx.x / tpr, tid = threadIdx.x - slot * tpr;
  const long long row = (long long)blockIdx.x * rows_per_cta + slot;
  const bool live = row < a.rows;
  const int w0 = slot * (tpr >> 5), wn = tpr >> 5;
  const T* x = static_cast<const T*>(a.x) + row * a.x_row;
  R* res = static_cast<R*>(a.residual) + row * a.res_row;

  float r[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long long e = ((long long)i * tpr + tid) * VEC;
    if (live && e < a.D) {
      const Vec<T, VEC> in = ld_vec<T, VEC>(x + e);
      if (RES != 0) {
        constexpr int RV = sizeof(R) * VEC > 16 ? 16 / (int)sizeof(R) : VEC;   // 16 bytes an access
#pragma unroll
        for (int j = 0; j < VEC; j += RV) {
          Vec<R, RV> p = ld_vec<R, RV>(res + e + j);
#pragma unroll
          for (int v = 0; v < RV; ++v) {
            r[i][j + v] = to_f32<T>(in.v[j + v]) + to_f32<R>(p.v[v]);
            p.v[v] = from_f32<R>(r[i][j + v]);
          }
          st_vec<R, RV>(res + e + j, p);
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[i][v] = to_f32<T>(in.v[v]);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) ss = fmaf(r[i][v], r[i][v], ss);
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) r[i][v] = 0.f;
    }
  }
  ss = row_reduce<false>(ss, part, w0, wn);
  const float rstd = rsqrtf(ss / (float)a.D + a.eps);
  float top[NV], all = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long long e = ((long long)i * tpr + tid) * VEC;
    top[i] = 0.f;
    if (live && e < a.D) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        r[i][v] = r[i][v] * rstd * a.w[e + v];
        if (OUT != VLA_OUT_IO) top[i] = max_nan(top[i], fabsf(r[i][v]));
      }
    }
    all = max_nan(all, top[i]);
  }
  if (OUT == VLA_OUT_IO) {
    T* y = static_cast<T*>(a.y) + row * a.y_row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const long long e = ((long long)i * tpr + tid) * VEC;
      if (!live || e >= a.D) continue;
      Vec<T, VEC> o;
#pragma unroll
      for (int v = 0; v < VEC; ++v) o.v[v] = from_f32<T>(r[i][v]);
      st_vec<T, VEC>(y + e, o);
    }
    return;
  }
  // the maximum over a row, or over the 128 / VEC adjacent threads of a group
  if (a.group == 0) {
    all = row_reduce<true>(all, part, w0, wn);
  } else if (VEC > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int o = 64 / VEC; o > 0; o >>= 1) top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
  } else {
    const int warp = threadIdx.x >> 5;   // a group is 4 warps (tpr is a multiple of 128 here)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      if ((threadIdx.x & 31) == 0) gmax[i * 32 + warp] = top[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float* g = gmax + i * 32 + (warp & ~3);
      top[i] = max_nan(max_nan(g[0], g[1]), max_nan(g[2], g[3]));
    }
  }
  unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.y_row;
  const float full = OUT == VLA_OUT_E4M3 ? 448.f : 127.f;
  const long long groups = (a.D + 127) / 128;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const long long e = ((long long)i * tpr + tid) * VEC;
    if (!live || e >= a.D) continue;
    float scale = (a.group ? top[i] : all) / full;
    if (scale < 1.17549435e-38f) scale = 1.f;   // false for a NaN
    const float inv = 1.f / scale;
    Vec<unsigned char, VEC == 1 ? 2 : VEC> o;   // VEC == 1 stores its byte alone
#pragma unroll
    for (int v = 0; v < VEC; ++v) o.v[v] = code<OUT>(r[i][v] * inv);
    if constexpr (VEC == 1) y[e] = o.v[0];
    else st_vec<unsigned char, VEC>(y + e, o);
    if (a.group) {
      if (e % 128 == 0) a.scale[row * groups + e / 128] = scale;
    } else if (e == 0) {
      a.scale[row] = scale;
    }
  }
}

template <typename T, int RES, int OUT, int VEC, int NV>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const int unit = VEC == 1 && a.group ? 128 : 32;
  const long long need = (a.D + (long long)VEC * NV - 1) / ((long long)VEC * NV);
  const int tpr = (int)((need + unit - 1) / unit * unit);
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const long long ctas = (a.rows + rows - 1) / rows;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  rms_norm_kernel<T, RES, OUT, VEC, NV><<<(unsigned int)ctas, tpr * rows, 0, s>>>(a, tpr, rows);
  return cudaGetLastError();
}

template <typename T, int RES, int OUT, int VEC>
cudaError_t by_width(const NormArgs& a, cudaStream_t s) {
  if (a.D <= 1024LL * VEC) return launch<T, RES, OUT, VEC, 1>(a, s);
  if (a.D <= 4096LL * VEC) return launch<T, RES, OUT, VEC, 4>(a, s);
  return launch<T, RES, OUT, VEC, 32 / VEC>(a, s);   // up to 32768 values (the entry point's limit)
}

template <typename T, int RES, int OUT>
cudaError_t by_alignment(const NormArgs& a, cudaStream_t s) {
  constexpr int VEC = 16 / (int)sizeof(T);
  const size_t out = OUT == VLA_OUT_IO ? sizeof(T) : 1, res = RES == 1 ? 2 : 4;
  bool ok = a.D % VEC == 0;
  ok = ok && (reinterpret_cast<uintptr_t>(a.x) | (unsigned long long)a.x_row * sizeof(T)) % 16 == 0;
  ok = ok && (reinterpret_cast<uintptr_t>(a.y) | (unsigned long long)a.y_row * out) % (VEC * out) == 0;
  if (RES != 0) {
    const size_t need = VEC * res > 16 ? 16 : VEC * res;
    ok = ok && (reinterpret_cast<uintptr_t>(a.residual) | (unsigned long long)a.res_row * res) % need == 0;
  }
  return ok ? by_width<T, RES, OUT, VEC>(a, s) : by_width<T, RES, OUT, 1>(a, s);
}

template <typename T, int RES>
cudaError_t by_output(const NormArgs& a, cudaStream_t s) {
  switch (a.out) {
    case VLA_OUT_E4M3: return by_alignment<T, RES, VLA_OUT_E4M3>(a, s);
    case VLA_OUT_INT8: return by_alignment<T, RES, VLA_OUT_INT8>(a, s);
    default: return by_alignment<T, RES, VLA_OUT_IO>(a, s);
  }
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) {
    if (!a.residual) return by_output<__nv_bfloat16, 0>(a, s);
    return a.res_bf16 ? by_output<__nv_bfloat16, 1>(a, s) : by_output<__nv_bfloat16, 2>(a, s);
  }
  if (!a.residual) return by_output<float, 0>(a, s);
  return a.res_bf16 ? by_output<float, 1>(a, s) : by_output<float, 2>(a, s);
}

}  // namespace vla
