// Matrix products with an epilogue, and the element-wise part of their gradient.
#include "vla_dense.cuh"

namespace vla {
namespace {

// A tile of 64 x 64 outputs a block of 256 threads, 4 x 4 a thread, 16 of Kd at a time through shared
// memory; float32 products and sums in the order of Kd.
constexpr int kT = 64, kK = 16;

template <typename I, typename T>
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs p) {
  __shared__ float as[kK][kT + 4], bs[kK][kT + 4];
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const long long m0 = (long long)blockIdx.x * kT, n0 = (long long)blockIdx.y * kT;
  const I* a = static_cast<const I*>(p.a);
  const I* b = static_cast<const I*>(p.b);
  float acc[4][4] = {};
  for (long long k0 = 0; k0 < p.Kd; k0 += kK) {
#pragma unroll
    for (int i = t; i < kK * kT; i += 256) {
      // the index that is adjacent in memory runs fastest
      const int ak = p.a_k == 1 ? i % kK : i / kT, am = p.a_k == 1 ? i / kK : i % kT;
      const int bk = p.b_k == 1 ? i % kK : i / kT, bn = p.b_k == 1 ? i / kK : i % kT;
      as[ak][am] = m0 + am < p.M && k0 + ak < p.Kd ? to_f32<I>(a[(m0 + am) * p.a_m + (k0 + ak) * p.a_k]) : 0.f;
      bs[bk][bn] = n0 + bn < p.N && k0 + bk < p.Kd ? to_f32<I>(b[(n0 + bn) * p.b_n + (k0 + bk) * p.b_k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m < p.M && n < p.N) epilogue_one<T>(p.out, acc[i][j], m, n);
    }
}

// A block takes a stretch of rows and 256 columns, a thread one of them.
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const SlopeArgs a, long long stretch) {
  const long long n = (long long)blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  const long long m0 = blockIdx.y * stretch, m1 = m0 + stretch < a.M ? m0 + stretch : a.M;
  float sum = 0.f;
  for (long long m = m0; m < m1; ++m) {
    float g = to_f32<T>(static_cast<const T*>(a.dy)[m * a.dy_row + n]);
    if (a.pre) {
      g *= activate_slope<sizeof(T) == 2>(to_f32<T>(static_cast<const T*>(a.pre)[m * a.pre_row + n]), a.act);
      static_cast<T*>(a.g)[m * a.g_row + n] = from_f32<T>(g);
    }
    sum += g;
  }
  if (a.db) a.partial[blockIdx.y * a.N + n] = sum;
}

__global__ void __launch_bounds__(256) slope_sum_kernel(const float* partial, float* db, long long N, long long parts) {
  const long long n = (long long)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float sum = 0.f;
  for (long long i = 0; i < parts; ++i) sum += partial[i * N + n];
  db[n] = sum;
}

long long slope_parts(long long M, long long N, int sm_count) {
  const long long across = (N + 255) / 256, want = (8LL * sm_count + across - 1) / across;
  const long long most = (M + 31) / 32;
  return want < most ? want : most;
}

}  // namespace

size_t product_ws(const ProductArgs&, int) { return 0; }

cudaError_t launch_product(const ProductArgs& p, int mat, cudaStream_t s) {
  const dim3 grid((unsigned int)((p.M + kT - 1) / kT), (unsigned int)((p.N + kT - 1) / kT));
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  };
  if (mat == kMatF32) return run(product_kernel<float, float>);
  if (mat == kMatBf16)
    return p.out.y_bf16 ? run(product_kernel<__nv_bfloat16, __nv_bfloat16>) : run(product_kernel<__nv_bfloat16, float>);
  return p.out.y_bf16 ? run(product_kernel<__nv_fp8_e4m3, __nv_bfloat16>) : run(product_kernel<__nv_fp8_e4m3, float>);
}

size_t slope_ws(long long M, long long N, int sm_count) { return (size_t)(slope_parts(M, N, sm_count) * N) * 4; }

cudaError_t launch_slope(const SlopeArgs& a, bool bf16, cudaStream_t s) {
  const long long want = slope_parts(a.M, a.N, a.sm_count), stretch = (a.M + want - 1) / want;
  const long long parts = (a.M + stretch - 1) / stretch;
  const dim3 grid((unsigned int)((a.N + 255) / 256), (unsigned int)parts);
  if (bf16) slope_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, stretch);
  else slope_kernel<float><<<grid, 256, 0, s>>>(a, stretch);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.db) return e;
  slope_sum_kernel<<<grid.x, 256, 0, s>>>(a.partial, a.db, a.N, parts);
  return cudaGetLastError();
}

}  // namespace vla
