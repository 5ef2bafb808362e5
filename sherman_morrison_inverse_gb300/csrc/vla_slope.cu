// The element-wise part of a product's gradient: g = dy * act'(pre), and db, the sum of g's rows.
#include "vla_dense.cuh"

namespace vla {
namespace {

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
