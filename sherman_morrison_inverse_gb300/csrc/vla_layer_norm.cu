// Layer norm with the residual's addition, and its gradients:
//   r = x + residual (float32; residual <- r in its own type),  mu = mean(r),
//   rstd = 1 / sqrt(mean((r - mu)^2) + eps),  y = (r - mu) rstd w + b
//   h = (r - mu) rstd, a = dy w:  dx = rstd (a - mean(a) - h mean(a h)) + dres,
//   dw = sum over rows of dy h,  db = sum over rows of dy
#include "vla_dense.cuh"

namespace vla {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Forward: a row stays in the registers of its tpr threads (whole warps), NV vectors of VEC adjacent
// values each, and is read once.  Each warp takes the mean and the squares around it of its own values, and one
// exchange joins them: sum of squares around mu = sum over warps of (theirs + n_w (mean_w - mu)^2), with no
// difference of large sums.
// RES: 0 none, 1 bfloat16, 2 float32
template <typename T, int RES, int VEC, int NV>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormArgs a, int tpr, int rows_per_cta, float inv_d) {
  using R = typename std::conditional<RES == 1, __nv_bfloat16, float>::type;
  constexpr int RV = sizeof(R) * VEC > 16 ? 16 / (int)sizeof(R) : VEC;
  __shared__ float part_sum[2][32], part_sq[2][32];
  const int slot = threadIdx.x / tpr, tid = threadIdx.x - slot * tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = slot * (tpr >> 5), wn = tpr >> 5;
  const int D = (int)a.D;
  // values of warp w of the row
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = D - (i * tpr + w * 32) * VEC;
      n += left < 0 ? 0 : left < 32 * VEC ? left : 32 * VEC;
    }
    return n;
  };
  const int mine = count(warp - w0);
  const float inv_mine = mine > 0 ? 1.f / (float)mine : 0.f;
  const int at = lane < wn ? lane : 0;
  const float theirs = lane < wn ? (float)count(at) : 0.f;

  Vec<T, VEC> in[NV];
  Vec<R, RV> res[NV][VEC / RV];
  auto load = [&](long long row) {
    if (row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    const R* r = static_cast<const R*>(a.residual) + row * a.res_row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
      if (e >= D) continue;
      in[i].raw = __ldcs(reinterpret_cast<const decltype(in[i].raw)*>(x + e));
      if (RES != 0) {
#pragma unroll
        for (int j = 0; j < VEC / RV; ++j) res[i][j].raw = __ldcs(reinterpret_cast<const decltype(res[i][j].raw)*>(r + e + j * RV));
      }
    }
  };
  const long long step = (long long)gridDim.x * rows_per_cta;
  long long row = (long long)blockIdx.x * rows_per_cta + slot;
  load(row);
  int par = 0;
  for (long long first = (long long)blockIdx.x * rows_per_cta; first < a.rows; first += step, row += step, par ^= 1) {
    const bool live = row < a.rows;
    float r[NV][VEC], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
      const bool on = live && e < D;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        r[i][v] = on ? to_f32<T>(in[i].v[v]) : 0.f;
        if (RES != 0 && on) r[i][v] += to_f32<R>(res[i][v / RV].v[v % RV]);
        sum += r[i][v];
      }
      if (RES != 0 && on) {
#pragma unroll
        for (int j = 0; j < VEC / RV; ++j) {
          Vec<R, RV> o;
#pragma unroll
          for (int v = 0; v < RV; ++v) o.v[v] = from_f32<R>(r[i][j * RV + v]);
          st_vec<R, RV>(static_cast<R*>(a.residual) + row * a.res_row + e + j * RV, o);
        }
      }
    }
    load(row + step);
    sum = warp_sum(sum);
    const float mean_w = sum * inv_mine;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float c = r[i][v] - mean_w;
        if (e < D) sq = fmaf(c, c, sq);
      }
    }
    sq = warp_sum(sq);
    float mean = mean_w;
    if (wn > 1) {
      // the other half of the parts is still read by warps that are a row behind
      if (lane == 0) {
        part_sum[par][warp] = sum;
        part_sq[par][warp] = sq;
      }
      __syncthreads();
      const float s = lane < wn ? part_sum[par][w0 + at] : 0.f;
      mean = warp_sum(s) * inv_d;
      const float off = theirs > 0.f ? s / theirs - mean : 0.f;
      sq = warp_sum(lane < wn ? fmaf(theirs * off, off, part_sq[par][w0 + at]) : 0.f);
    }
    const float rstd = __frsqrt_rn(fmaf(sq, inv_d, a.eps));
    if (!live) continue;
    if (a.stats && tid == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.y_row;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
      if (e >= D) continue;
      Vec<T, VEC> o;
#pragma unroll
      for (int v = 0; v < VEC; ++v) o.v[v] = from_f32<T>(fmaf((r[i][v] - mean) * rstd, a.w[e + v], a.b ? a.b[e + v] : 0.f));
      st_vec<T, VEC>(y + e, o);
    }
  }
}

template <typename T, int RES, int VEC, int NV>
cudaError_t forward(const LayerNormArgs& a, cudaStream_t s) {
  const long long need = (a.D + (long long)VEC * NV - 1) / ((long long)VEC * NV);
  const int tpr = (int)((need + 31) / 32 * 32);
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  const long long all = (a.rows + rows - 1) / rows, most = (long long)a.sm_count * (2048 / (tpr * rows));
  layer_norm_kernel<T, RES, VEC, NV><<<(unsigned int)(all < most ? all : most), tpr * rows, 0, s>>>(a, tpr, rows, 1.f / (float)a.D);
  return cudaGetLastError();
}

template <typename T, int RES>
cudaError_t forward_of(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int VEC = 16 / (int)sizeof(T);
  constexpr long long RS = RES == 2 ? 4 : 2;
  auto whole = [](const void* p, long long row, long long size) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(row * size)) & 15u) == 0;
  };
  const bool vec = a.D % VEC == 0 && whole(a.x, a.x_row, sizeof(T)) && whole(a.y, a.y_row, sizeof(T)) &&
                   (RES == 0 || whole(a.residual, a.res_row, RS));
  if (vec) {
    if (a.D <= 1024 * VEC) return forward<T, RES, VEC, 1>(a, s);
    if (a.D <= 2048 * VEC) return forward<T, RES, VEC, 2>(a, s);
    return forward<T, RES, VEC, 32 / VEC>(a, s);
  }
  if (a.D <= 1024) return forward<T, RES, 1, 1>(a, s);
  if (a.D <= 4096) return forward<T, RES, 1, 4>(a, s);
  if (a.D <= 16384) return forward<T, RES, 1, 16>(a, s);
  return forward<T, RES, 1, 32>(a, s);
}

// Backward, dx: a block a row, read twice.
template <typename TD, typename TX>
__global__ void __launch_bounds__(256) back_row_kernel(const LayerNormBackArgs a, float inv_d) {
  __shared__ float part[2][2][8];
  const int t = threadIdx.x, D = (int)a.D;
  int par = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const TD* dy = static_cast<const TD*>(a.dy) + row * a.dy_row;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_row;
    const float mean = a.stats[2 * row], rstd = a.stats[2 * row + 1];
    float s1 = 0.f, s2 = 0.f;
    for (int e = t; e < D; e += 256) {
      const float g = to_f32<TD>(dy[e]) * a.w[e];
      s1 += g;
      s2 = fmaf(g, (to_f32<TX>(x[e]) - mean) * rstd, s2);
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if ((t & 31) == 0) {
      part[par][0][t >> 5] = s1;
      part[par][1][t >> 5] = s2;
    }
    __syncthreads();
    s1 = s2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s1 += part[par][0][i];
      s2 += part[par][1][i];
    }
    s1 *= inv_d;
    s2 *= inv_d;
    for (int e = t; e < D; e += 256) {
      const float g = to_f32<TD>(dy[e]) * a.w[e], h = (to_f32<TX>(x[e]) - mean) * rstd;
      float v = rstd * (g - s1 - h * s2);
      if (a.dres) v += to_f32<TX>(static_cast<const TX*>(a.dres)[row * a.dres_row + e]);
      static_cast<TX*>(a.dx)[row * a.dx_row + e] = from_f32<TX>(v);
    }
  }
}

// Backward, dw and db: a block takes a stretch of rows and 256 columns, a thread one of them.
template <typename TD, typename TX>
__global__ void __launch_bounds__(256) back_column_kernel(const LayerNormBackArgs a, long long stretch) {
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.D) return;
  const long long m0 = blockIdx.y * stretch, m1 = m0 + stretch < a.rows ? m0 + stretch : a.rows;
  float dw = 0.f, db = 0.f;
  for (long long m = m0; m < m1; ++m) {
    const float dy = to_f32<TD>(static_cast<const TD*>(a.dy)[m * a.dy_row + e]);
    const float x = to_f32<TX>(static_cast<const TX*>(a.x)[m * a.x_row + e]);
    dw = fmaf(dy, (x - a.stats[2 * m]) * a.stats[2 * m + 1], dw);
    db += dy;
  }
  a.partial[(2 * blockIdx.y) * a.D + e] = dw;
  a.partial[(2 * blockIdx.y + 1) * a.D + e] = db;
}

__global__ void __launch_bounds__(256) back_sum_kernel(const float* partial, float* dw, float* db, long long D, long long parts) {
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= D) return;
  float s = 0.f, t = 0.f;
  for (long long i = 0; i < parts; ++i) {
    s += partial[2 * i * D + e];
    t += partial[(2 * i + 1) * D + e];
  }
  dw[e] = s;
  if (db) db[e] = t;
}

long long back_parts(long long rows, long long D, int sm_count) {
  const long long across = (D + 255) / 256, want = (8LL * sm_count + across - 1) / across;
  const long long most = (rows + 31) / 32;
  return want < most ? want : most;
}

template <typename TD, typename TX>
cudaError_t backward(const LayerNormBackArgs& a, cudaStream_t s) {
  const long long want = back_parts(a.rows, a.D, a.sm_count), stretch = (a.rows + want - 1) / want;
  const long long parts = (a.rows + stretch - 1) / stretch, most = 8LL * a.sm_count;
  back_row_kernel<TD, TX><<<(unsigned int)(a.rows < most ? a.rows : most), 256, 0, s>>>(a, 1.f / (float)a.D);
  const dim3 grid((unsigned int)((a.D + 255) / 256), (unsigned int)parts);
  back_column_kernel<TD, TX><<<grid, 256, 0, s>>>(a, stretch);
  back_sum_kernel<<<grid.x, 256, 0, s>>>(a.partial, a.dw, a.db, a.D, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) {
    if (!a.residual) return forward_of<__nv_bfloat16, 0>(a, s);
    return a.res_bf16 ? forward_of<__nv_bfloat16, 1>(a, s) : forward_of<__nv_bfloat16, 2>(a, s);
  }
  if (!a.residual) return forward_of<float, 0>(a, s);
  return a.res_bf16 ? forward_of<float, 1>(a, s) : forward_of<float, 2>(a, s);
}

size_t layer_norm_back_ws(long long rows, long long D, int sm_count) {
  return (size_t)(2 * back_parts(rows, D, sm_count) * D) * 4;
}

cudaError_t launch_layer_norm_back(const LayerNormBackArgs& a, bool dy_bf16, bool x_bf16, cudaStream_t s) {
  if (dy_bf16) return x_bf16 ? backward<__nv_bfloat16, __nv_bfloat16>(a, s) : backward<__nv_bfloat16, float>(a, s);
  return x_bf16 ? backward<float, __nv_bfloat16>(a, s) : backward<float, float>(a, s);
}

}  // namespace vla
