// Layer norm with the residual's addition, and its gradients:
//   r = x + residual (float32; residual <- r in its own type),  mu = mean(r),
//   rstd = 1 / sqrt(mean((r - mu)^2) + eps),  y = (r - mu) rstd w + b
//   h = (r - mu) rstd, a = dy w:  dx = rstd (a - mean(a) - h mean(a h)) + dres,
//   dw = sum over rows of dy h,  db = sum over rows of dy
#include "vla_dense.cuh"

#include <atomic>

namespace vla {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Forward: a row stays in the registers of its tpr threads (whole warps), NV vectors of VEC adjacent
// values each, and is read once; up to 16 values a thread, the next row is fetched before the present one is reduced
// and w and b stay in registers.  Each warp takes the mean and the squares around it of its own values, and one
// exchange joins them: sum of squares around mu = sum over warps of (theirs + n_w (mean_w - mu)^2), with no
// difference of large sums.  Memory bound.
// RES: 0 none, 1 bfloat16, 2 float32
template <typename T, int RES, int VEC, int NV>
__global__ void __launch_bounds__(VEC * NV <= 16 ? 512 : 1024, 1)
    layer_norm_kernel(const LayerNormArgs a, int tpr, int rows_per_cta, float inv_d) {
  using R = typename std::conditional<RES == 1, __nv_bfloat16, float>::type;
  constexpr int RV = sizeof(R) * VEC > 16 ? 16 / (int)sizeof(R) : VEC;
  constexpr bool AHEAD = VEC * NV <= 16;
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
  const float theirs = lane < wn ? (float)count(at) : 0.f, inv_theirs = theirs > 0.f ? 1.f / theirs : 0.f;

  float w[AHEAD ? NV : 1][VEC], b[AHEAD ? NV : 1][VEC];
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        w[i][v] = e < D ? a.w[e + v] : 0.f;
        b[i][v] = a.b && e < D ? a.b[e + v] : 0.f;
      }
    }
  }
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
  if (AHEAD) load(row);
  int par = 0;
  for (long long first = (long long)blockIdx.x * rows_per_cta; first < a.rows; first += step, row += step, par ^= 1) {
    const bool live = row < a.rows;
    if (!AHEAD) load(row);
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
    if (AHEAD) load(row + step);
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
      const float off = theirs > 0.f ? fmaf(s, inv_theirs, -mean) : 0.f;
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
      for (int v = 0; v < VEC; ++v) {
        const float wv = AHEAD ? w[AHEAD ? i : 0][v] : a.w[e + v], bv = AHEAD ? b[AHEAD ? i : 0][v] : a.b ? a.b[e + v] : 0.f;
        o.v[v] = from_f32<T>(fmaf((r[i][v] - mean) * rstd, wv, bv));
      }
      st_vec<T, VEC>(y + e, o);
    }
  }
}

// Blocks an SM of a kernel and block size, asked for once.
template <typename K>
cudaError_t blocks_of(K kern, int threads, size_t smem, std::atomic<unsigned int>& known, int* blocks) {
  unsigned int k = known.load(std::memory_order_relaxed);   // size | blocks
  if (k >> 16 != (unsigned int)threads) {
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
    if (e != cudaSuccess) return e;
    k = (unsigned int)threads << 16 | (unsigned int)n;
    known.store(k, std::memory_order_relaxed);
  }
  *blocks = (k & 0xffffu) > 0 ? (int)(k & 0xffffu) : 1;
  return cudaSuccess;
}

template <typename T, int RES, int VEC, int NV>
cudaError_t forward(const LayerNormArgs& a, cudaStream_t s) {
  auto kern = layer_norm_kernel<T, RES, VEC, NV>;
  const long long need = (a.D + (long long)VEC * NV - 1) / ((long long)VEC * NV);
  const int tpr = (int)((need + 31) / 32 * 32);
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  static std::atomic<unsigned int> known{0};
  int per_sm = 1;
  const cudaError_t e = blocks_of(kern, tpr * rows, 0, known, &per_sm);
  if (e != cudaSuccess) return e;
  const long long all = (a.rows + rows - 1) / rows, most = (long long)per_sm * a.sm_count;
  kern<<<(unsigned int)(all < most ? all : most), tpr * rows, 0, s>>>(a, tpr, rows, 1.f / (float)a.D);
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
    if (a.D <= 2048) return forward<T, RES, VEC, 8 / VEC>(a, s);
    if (a.D <= 8192) return forward<T, RES, VEC, 16 / VEC>(a, s);
    return forward<T, RES, VEC, 32 / VEC>(a, s);
  }
  if (a.D <= 2048) return forward<T, RES, 1, 4>(a, s);
  if (a.D <= 8192) return forward<T, RES, 1, 16>(a, s);
  return forward<T, RES, 1, 32>(a, s);
}

// Backward up to 8192 values a row, one pass.  A thread has the same VEC NV columns of every row of its block, and
// with them its sums of dw and db; a row's two sums (of a and of a h) are joined by one barrier.
// VEC 4: rows on 16-byte boundaries arrive by bulk copies in a ring of stages of rows_per_cta rows, as many as shared
// memory holds, so that some 200 KB an SM are on their way whatever the registers hold; a stage is filled again
// behind the barrier of the next one, when nobody reads it any more.  VEC 1: rows anywhere, read directly.
// Blocks leave their sums of dw and db as rows of `partial`, which back_sum_kernel adds in their order.
constexpr int kBackStages = 8;
constexpr int kBackThreads = 512;

template <typename TD, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(kBackThreads, 1)
    back_kernel(const LayerNormBackArgs a, int tpr, int rows_per_cta, int stages, int row_bytes, float inv_d, DevStatus* status) {
  extern __shared__ __align__(128) unsigned char smem[];   // the ring; at the end the rows' sums
  __shared__ uint64_t full[kBackStages];
  __shared__ float part[2][2][kBackThreads / 32];
  const int slot = threadIdx.x / tpr, tid = threadIdx.x - slot * tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = slot * (tpr >> 5), wn = tpr >> 5;
  const int D = (int)a.D;
  const long long step = (long long)gridDim.x * rows_per_cta, base = (long long)blockIdx.x * rows_per_cta;
  const uint32_t dy_bytes = (uint32_t)(D * sizeof(TD)), x_bytes = (uint32_t)(D * sizeof(TX));

  auto fill = [&](long long first, int stage) {   // one thread
    int n = 0;
    for (int r = 0; r < rows_per_cta; ++r) n += first + r < a.rows;
    if (n == 0) return;
    mbar_arrive_expect_tx(full + stage, n * (dy_bytes + x_bytes * (a.dres ? 2 : 1)));
    for (int r = 0; r < n; ++r) {
      unsigned char* to = smem + (size_t)(stage * rows_per_cta + r) * row_bytes;
      bulk_g2s(to, static_cast<const TD*>(a.dy) + (first + r) * a.dy_row, dy_bytes, full + stage);
      bulk_g2s(to + dy_bytes, static_cast<const TX*>(a.x) + (first + r) * a.x_row, x_bytes, full + stage);
      if (a.dres) bulk_g2s(to + dy_bytes + x_bytes, static_cast<const TX*>(a.dres) + (first + r) * a.dres_row, x_bytes, full + stage);
    }
  };
  if (VEC > 1) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(full + i, 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < stages; ++i) fill(base + i * step, i);
  }
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int e = (i * tpr + tid) * VEC;
      w[i][v] = e < D ? a.w[e + v] : 0.f;
      dw[i][v] = db[i][v] = 0.f;
    }
  long long row = base + slot;
  float mean = 0.f, rstd = 0.f;
  auto stats = [&](long long r) {
    if (r < a.rows) {
      mean = a.stats[2 * r];
      rstd = a.stats[2 * r + 1];
    }
  };
  stats(row);
  int par = 0, stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (long long first = base; first < a.rows; first += step, row += step, par ^= 1) {
    const bool live = row < a.rows;
    const TD* dy = static_cast<const TD*>(a.dy) + row * a.dy_row;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_row;
    const TX* dres = static_cast<const TX*>(a.dres) + row * a.dres_row;
    if (VEC > 1) {
      const unsigned char* at = smem + (size_t)(stage * rows_per_cta + slot) * row_bytes;
      dy = reinterpret_cast<const TD*>(at);
      x = reinterpret_cast<const TX*>(at + dy_bytes);
      dres = reinterpret_cast<const TX*>(at + dy_bytes + x_bytes);
      ok = mbar_wait_bounded(full + stage, phase);
    }
    const float mu = mean, rs = rstd;
    stats(row + step);
    float g[NV][VEC], h[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
      Vec<TD, VEC> d;
      Vec<TX, VEC> c;
      const bool on = live && ok && e < D;
      if (on) {
        d = ld_vec<TD, VEC>(dy + e);
        c = ld_vec<TX, VEC>(x + e);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float y = on ? to_f32<TD>(d.v[v]) : 0.f;
        h[i][v] = on ? (to_f32<TX>(c.v[v]) - mu) * rs : 0.f;
        g[i][v] = y * w[i][v];
        dw[i][v] = fmaf(y, h[i][v], dw[i][v]);
        db[i][v] += y;
        s1 += g[i][v];
        s2 = fmaf(g[i][v], h[i][v], s2);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    // the other half of the parts is still read by warps that are a row behind
    if (lane == 0) {
      part[par][0][warp] = s1;
      part[par][1][warp] = s2;
    }
    if (VEC > 1) {
      if (__syncthreads_or(!ok)) {   // a copy that did not arrive: give up, all threads alike
        if (threadIdx.x == 0) atomicOr(&status->flags, kStatusTimeout);
        return;
      }
      // behind the barrier nobody reads the stage before this one: the row that is `stages` on goes there
      if (threadIdx.x == 0 && first > base) fill(first + (stages - 1) * step, stage > 0 ? stage - 1 : stages - 1);
    } else {
      __syncthreads();
    }
    if (wn > 1) {
      s1 = lane < wn ? part[par][0][w0 + lane] : 0.f;
      s2 = lane < wn ? part[par][1][w0 + lane] : 0.f;
#pragma unroll
      for (int o = kBackThreads / 64; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      s1 = __shfl_sync(0xffffffffu, s1, 0);
      s2 = __shfl_sync(0xffffffffu, s2, 0);
    }
    s1 *= inv_d;
    s2 *= inv_d;
    if (live) {
      TX* dx = static_cast<TX*>(a.dx) + row * a.dx_row;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + tid) * VEC;
        if (e >= D) continue;
        Vec<TX, VEC> o, r;
        if (a.dres) r = ld_vec<TX, VEC>(dres + e);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float t = rs * (g[i][v] - fmaf(h[i][v], s2, s1));
          if (a.dres) t += to_f32<TX>(r.v[v]);
          o.v[v] = from_f32<TX>(t);
        }
        st_vec<TX, VEC>(dx + e, o);
      }
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // the slots' sums, in their order
  float* sums = reinterpret_cast<float*>(smem);
  for (int r = 0; r < rows_per_cta; ++r) {
    if (rows_per_cta > 1) __syncthreads();   // the ring is read no more; the last slot has added its sums
    if (slot != r) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = (i * tpr + tid) * VEC + v;
        if (e >= D) continue;
        if (r > 0) {
          dw[i][v] += sums[e];
          db[i][v] += sums[D + e];
        }
        if (r + 1 < rows_per_cta) {
          sums[e] = dw[i][v];
          sums[D + e] = db[i][v];
        } else {
          a.partial[2 * blockIdx.x * a.D + e] = dw[i][v];
          a.partial[(2 * blockIdx.x + 1) * a.D + e] = db[i][v];
        }
      }
  }
}

// Wider rows: dx by a block a row, read twice, and the columns' sums by a kernel of their own.
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
#pragma unroll 4
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
#pragma unroll 4
    for (int e = t; e < D; e += 256) {
      const float g = to_f32<TD>(dy[e]) * a.w[e], h = (to_f32<TX>(x[e]) - mean) * rstd;
      float v = rstd * (g - fmaf(h, s2, s1));
      if (a.dres) v += to_f32<TX>(static_cast<const TX*>(a.dres)[row * a.dres_row + e]);
      static_cast<TX*>(a.dx)[row * a.dx_row + e] = from_f32<TX>(v);
    }
  }
}

// A block takes a stretch of rows and 256 columns, a thread one of them.
template <typename TD, typename TX>
__global__ void __launch_bounds__(256) back_column_kernel(const LayerNormBackArgs a, long long stretch) {
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.D) return;
  const long long m0 = blockIdx.y * stretch, m1 = m0 + stretch < a.rows ? m0 + stretch : a.rows;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (long long m = m0; m < m1; ++m) {
    const float dy = to_f32<TD>(static_cast<const TD*>(a.dy)[m * a.dy_row + e]);
    const float x = to_f32<TX>(static_cast<const TX*>(a.x)[m * a.x_row + e]);
    dw = fmaf(dy, (x - a.stats[2 * m]) * a.stats[2 * m + 1], dw);
    db += dy;
  }
  a.partial[(2 * blockIdx.y) * a.D + e] = dw;
  a.partial[(2 * blockIdx.y + 1) * a.D + e] = db;
}

// The parts' sums, of dw (blockIdx.y 0) and db: a block has 32 columns, its 8 warps take every eighth part.
__global__ void __launch_bounds__(256) back_sum_kernel(const float* partial, float* dw, float* db, long long D, long long parts) {
  __shared__ float sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long e = (long long)blockIdx.x * 32 + lane;
  const float* p = partial + blockIdx.y * D + e;
  float sum = 0.f;
  if (e < D) {
#pragma unroll 8
    for (long long i = warp; i < parts; i += 8) sum += p[2 * i * D];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && e < D) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += sums[i][lane];
    (blockIdx.y ? db : dw)[e] = sum;
  }
}

constexpr long long kOnePass = 8192;   // values of a row that back_kernel takes
constexpr int kRing = 208 * 1024;      // bytes of its stages an SM

// Threads a row, rows and blocks of back_kernel.
struct BackShape {
  int n, tpr, rows, per_sm;
};
BackShape back_shape(long long D) {
  BackShape b{};
  b.n = D <= 2048 ? 8 : 16;
  b.tpr = (int)(((D + b.n - 1) / b.n + 31) / 32 * 32);
  b.rows = b.tpr >= 256 ? 1 : 256 / b.tpr;
  b.per_sm = b.tpr * b.rows > 256 ? 1 : 2;
  return b;
}

long long back_parts(long long rows, long long D, int sm_count) {
  if (D <= kOnePass) {
    const BackShape b = back_shape(D);
    const long long all = (rows + b.rows - 1) / b.rows, most = (long long)b.per_sm * sm_count;
    return all < most ? all : most;
  }
  const long long across = (D + 255) / 256, want = (8LL * sm_count + across - 1) / across;
  const long long most = (rows + 31) / 32;
  return want < most ? want : most;
}

template <typename TD, typename TX, int VEC, int NV>
cudaError_t one_pass(const LayerNormBackArgs& a, cudaStream_t s) {
  auto kern = back_kernel<TD, TX, VEC, NV>;
  const BackShape b = back_shape(a.D);
  const int row_bytes = (int)(a.D * (sizeof(TD) + sizeof(TX) * (a.dres ? 2 : 1)));
  int stages = 1;
  size_t bytes = b.rows > 1 ? 8 * (size_t)a.D : 0;
  if (VEC > 1) {
    stages = kRing / b.per_sm / (row_bytes * b.rows);
    stages = stages > kBackStages ? kBackStages : stages;
    const size_t ring = (size_t)stages * row_bytes * b.rows;
    bytes = ring > bytes ? ring : bytes;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    // more than 48 KB of shared memory: allowed once a kernel and device (the first 64)
    static std::atomic<unsigned long long> ready{0};
    if (device >= 64 || !(ready.load(std::memory_order_relaxed) >> device & 1)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
      if (e != cudaSuccess) return e;
      if (device < 64) ready.fetch_or(1ull << device, std::memory_order_relaxed);
    }
  }
  kern<<<(unsigned int)back_parts(a.rows, a.D, a.sm_count), b.tpr * b.rows, bytes, s>>>(
      a, b.tpr, b.rows, stages, row_bytes, 1.f / (float)a.D, a.status);
  return cudaGetLastError();
}

template <typename TD, typename TX>
cudaError_t backward(const LayerNormBackArgs& a, cudaStream_t s) {
  long long parts = back_parts(a.rows, a.D, a.sm_count);
  cudaError_t e = cudaSuccess;
  if (a.D <= kOnePass) {
    auto whole = [](const void* p, long long row, size_t size) {
      return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)((size_t)row * size)) & 15u) == 0;
    };
    constexpr size_t SD = sizeof(TD), SX = sizeof(TX);
    const bool ring = a.D * SD % 16 == 0 && a.D * SX % 16 == 0 && whole(a.dy, a.dy_row, SD) && whole(a.x, a.x_row, SX) &&
                      whole(a.dx, a.dx_row, SX) && (!a.dres || whole(a.dres, a.dres_row, SX));
    if (back_shape(a.D).n == 8) e = ring ? one_pass<TD, TX, 4, 2>(a, s) : one_pass<TD, TX, 1, 8>(a, s);
    else e = ring ? one_pass<TD, TX, 4, 4>(a, s) : one_pass<TD, TX, 1, 16>(a, s);
  } else {
    const long long stretch = (a.rows + parts - 1) / parts, most = 8LL * a.sm_count;
    parts = (a.rows + stretch - 1) / stretch;
    back_row_kernel<TD, TX><<<(unsigned int)(a.rows < most ? a.rows : most), 256, 0, s>>>(a, 1.f / (float)a.D);
    back_column_kernel<TD, TX><<<dim3((unsigned int)((a.D + 255) / 256), (unsigned int)parts), 256, 0, s>>>(a, stretch);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  back_sum_kernel<<<dim3((unsigned int)((a.D + 31) / 32), a.db ? 2 : 1), 256, 0, s>>>(a.partial, a.dw, a.db, a.D, parts);
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
