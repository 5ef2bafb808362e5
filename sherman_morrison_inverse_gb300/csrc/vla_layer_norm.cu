// Layer norm with the residual's addition, and its gradients:
//   r = x + residual (float32; residual <- r in its own type),  mu = mean(r),
//   rstd = 1 / sqrt(mean((r - mu)^2) + eps),  y = (r - mu) rstd w + b
//   h = (r - mu) rstd, a = dy w:  dx = rstd (a - mean(a) - h mean(a h)) + dres,
//   dw = sum over rows of dy h,  db = sum over rows of dy
#include "vla_dense.cuh"

#include <atomic>
#include <type_traits>

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
// difference of large sums.  Memory bound: 16384 x 4096 bfloat16 with residual and statistics 91 us, 5.9 TB/s, 88 % of a
// copy's rate (with 8 values a thread, 512 threads a row, 115 us); 24 x 5120 4.3 us.  Wider than 8192, without the next row ahead:
// 4096 x 16384 208 us.  VEC 1, for rows off 16-byte boundaries or odd widths, value by value: 16384 x 4095 182 us, 4096 x 16383
// 869, 4099 x 1001 float32 12.6 (1000 columns: 8.7).
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
// behind the barrier of the next one, when nobody reads it any more.  Waits are bounded: a block that gives up waits (bounded too)
// for its copies under way and leaves the sums that it has.  VEC 1: rows anywhere, read directly.
// Blocks leave their sums of dw and db as rows of `partial`, which back_sum_kernel adds in their order.
// 16384 x 4096 bfloat16 with the residual's gradient 103 us, 5.2 TB/s, 78 % of a copy's rate: a row's chain of barriers on the 16 warps
// that the registers of 16 values a thread allow.  Value by value: 4099 x 1001 float32 17.5 us (1000 columns, copied ahead: 17.9),
// 16384 x 4095 bfloat16 326.
constexpr int kBackStages = 8;
constexpr int kBackThreads = 512;

// The column of a thread's value v: VEC adjacent ones, then the next vector's.
template <int VEC>
__device__ __forceinline__ int column_of(int v, int tpr, int tid) { return (v / VEC * tpr + tid) * VEC + v % VEC; }

// A thread's values of a row as float32 pairs (2 i, 2 i + 1), zero where there is no column or, without `on`, no row.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void get_row(const T* p, bool on, int tpr, int tid, int D, uint64_t (&o)[VEC * NV / 2]) {
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = column_of<VEC>(4 * i, tpr, tid);
      o[2 * i] = o[2 * i + 1] = 0;
      if (!on || e >= D) continue;
      const Vec<T, 4> x = ld_vec<T, 4>(p + e);
      if constexpr (sizeof(T) == 2) {
        o[2 * i] = pair(lo_f(x.raw.x), hi_f(x.raw.x));
        o[2 * i + 1] = pair(lo_f(x.raw.y), hi_f(x.raw.y));
      } else {
        o[2 * i] = pair(__uint_as_float(x.raw.x), __uint_as_float(x.raw.y));
        o[2 * i + 1] = pair(__uint_as_float(x.raw.z), __uint_as_float(x.raw.w));
      }
    }
  } else {
    T x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = column_of<VEC>(i, tpr, tid);
      x[i] = on && e < D ? p[e] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) o[i] = pair(to_f32<T>(x[2 * i]), to_f32<T>(x[2 * i + 1]));
  }
}

template <typename TD, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(kBackThreads, 1)
    back_kernel(const LayerNormBackArgs a, int tpr, int rows_per_cta, int stages, int row_bytes, float inv_d, DevStatus* status) {
  extern __shared__ __align__(128) unsigned char smem[];   // the ring; at the end the rows' sums
  __shared__ uint64_t full[kBackStages];
  __shared__ float2 part[2][kBackThreads / 32];
  const int slot = threadIdx.x / tpr, tid = threadIdx.x - slot * tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = slot * (tpr >> 5), wn = tpr >> 5;
  const int D = (int)a.D;
  const long long step = (long long)gridDim.x * rows_per_cta, base = (long long)blockIdx.x * rows_per_cta;
  all_started();   // the sums' kernel
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
  constexpr int P = VEC * NV / 2;
  auto column = [&](int v) { return column_of<VEC>(v, tpr, tid); };
  // 16 values a thread leave no registers for w: it is read again every row, from the first-level cache
  constexpr bool KEEP = VEC * NV <= 8;
  uint64_t w[P], dw[P] = {}, db[P] = {};
  if (KEEP) get_row<float, VEC, NV>(a.w, true, tpr, tid, D, w);
  long long row = base + slot;
  float mean = 0.f, rstd = 0.f;
  auto stats = [&](long long r) {   // a row that there is not counts nothing
    mean = r < a.rows ? a.stats[2 * r] : 0.f;
    rstd = r < a.rows ? a.stats[2 * r + 1] : 0.f;
  };
  stats(row);
  // rows read directly: up to 8 values a thread, the next row's are on their way while the present one is reduced
  constexpr bool AHEAD = VEC == 1 && NV <= 8;
  uint64_t g_next[AHEAD ? P : 1], h_next[AHEAD ? P : 1];
  if constexpr (AHEAD) {
    get_row<TD, VEC, NV>(static_cast<const TD*>(a.dy) + row * a.dy_row, row < a.rows, tpr, tid, D, g_next);
    get_row<TX, VEC, NV>(static_cast<const TX*>(a.x) + row * a.x_row, row < a.rows, tpr, tid, D, h_next);
  }
  int par = 0, stage = 0, span = 2;   // span: the power of two from wn on
  while (span < wn) span *= 2;
  uint32_t phase = 0;
  bool ok = true, gave_up = false;
  long long first = base;
  for (; first < a.rows; first += step, row += step, par ^= 1) {
    const bool live = row < a.rows;
    const TD* dy = static_cast<const TD*>(a.dy) + row * a.dy_row;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_row;
    const TX* dres = static_cast<const TX*>(a.dres) + row * a.dres_row;
    if (VEC > 1) {
      const unsigned char* at = smem + (size_t)(stage * rows_per_cta + slot) * row_bytes;
      dy = reinterpret_cast<const TD*>(at);
      x = reinterpret_cast<const TX*>(at + dy_bytes);
      dres = reinterpret_cast<const TX*>(at + dy_bytes + x_bytes);
      ok = a.wait_limit > 0 && mbar_wait_bounded(full + stage, phase, a.wait_limit);
    }
    uint64_t g[P], h[P], r[P] = {}, t1 = 0, t2 = 0;
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        g[i] = g_next[i];
        h[i] = h_next[i];
      }
      get_row<TD, VEC, NV>(dy + step * a.dy_row, row + step < a.rows, tpr, tid, D, g_next);
      get_row<TX, VEC, NV>(x + step * a.x_row, row + step < a.rows, tpr, tid, D, h_next);
      if (a.dres) get_row<TX, VEC, NV>(dres, live, tpr, tid, D, r);
    } else {
      get_row<TD, VEC, NV>(dy, live, tpr, tid, D, g);
      get_row<TX, VEC, NV>(x, live, tpr, tid, D, h);
    }
    const float rs = rstd;
    const uint64_t scale = pair(rs, rs), shift = pair(-mean, -mean);
    stats(row + step);
    if (!KEEP) get_row<float, VEC, NV>(a.w, true, tpr, tid, D, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      h[i] = mul2(add2(h[i], shift), scale);   // x rstd - mean rstd would round off 2^-24 of |mean| rstd
      dw[i] = fma2(g[i], h[i], dw[i]);
      db[i] = add2(g[i], db[i]);
      g[i] = mul2(g[i], w[i]);
      t1 = add2(t1, g[i]);
      t2 = fma2(g[i], h[i], t2);
    }
    float s1, s2, other;
    unpair(t1, s1, other);
    s1 += other;
    unpair(t2, s2, other);
    s2 += other;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    // the other half of the parts is still read by warps that are a row behind
    if (lane == 0) part[par][warp] = make_float2(s1, s2);
    if (VEC > 1) {
      if (__syncthreads_or(!ok)) {   // a copy that did not arrive: give up, all threads alike
        gave_up = true;
        break;
      }
      // behind the barrier nobody reads the stage before this one: the row that is `stages` on goes there
      if (threadIdx.x == 0 && first > base) fill(first + (stages - 1) * step, stage > 0 ? stage - 1 : stages - 1);
    } else {
      __syncthreads();
    }
    if (wn > 1) {
      const int at = lane & (span - 1);   // every lane ends up with the row's sums
      const float2 q = at < wn ? part[par][w0 + at] : make_float2(0.f, 0.f);
      s1 = q.x;
      s2 = q.y;
      for (int o = span >> 1; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
    }
    const uint64_t m1 = pair(-s1 * inv_d, -s1 * inv_d), m2 = pair(-s2 * inv_d, -s2 * inv_d);
    if (live) {
      TX* dx = static_cast<TX*>(a.dx) + row * a.dx_row;
      if (!AHEAD && a.dres) get_row<TX, VEC, NV>(dres, true, tpr, tid, D, r);
#pragma unroll
      for (int i = 0; i < P; ++i) r[i] = fma2(fma2(h[i], m2, add2(g[i], m1)), scale, r[i]);
      if constexpr (VEC == 4) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (column(4 * i) >= D) continue;
          float v[4];
          unpair(r[2 * i], v[0], v[1]);
          unpair(r[2 * i + 1], v[2], v[3]);
          Vec<TX, 4> o;
          if constexpr (sizeof(TX) == 2) {
            o.raw = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o.v[k] = v[k];
          }
          st_vec<TX, 4>(dx + column(4 * i), o);
        }
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float u, v;
          unpair(r[i], u, v);
          if (column(2 * i) < D) dx[column(2 * i)] = from_f32<TX>(u);
          if (column(2 * i + 1) < D) dx[column(2 * i + 1)] = from_f32<TX>(v);
        }
      }
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (gave_up) {
    if (threadIdx.x == 0) {
      // filled so far: the first `stages`, then one an iteration but the first, as long as there are rows
      const long long passed = (first - base) / step, all = (a.rows - base + step - 1) / step;
      const long long most = passed > 0 ? passed + stages - 1 : stages;
      drain_ring(full, stages, (uint32_t)(most < all ? most : all));
      atomicOr(&status->flags, kStatusTimeout);
    }
    __syncthreads();
  }
  // the slots' sums, in their order
  float* sums = reinterpret_cast<float*>(smem);
  for (int r = 0; r < rows_per_cta; ++r) {
    if (rows_per_cta > 1) __syncthreads();   // the ring is read no more; the last slot has added its sums
    if (slot != r) continue;
    float* to_w = r + 1 < rows_per_cta ? sums : a.partial + 2 * blockIdx.x * a.D;
    float* to_b = to_w + D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float u[2], v[2];
      unpair(dw[i], u[0], u[1]);
      unpair(db[i], v[0], v[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = column(2 * i + k);
        if (e >= D) continue;
        to_w[e] = r > 0 ? u[k] + sums[e] : u[k];
        to_b[e] = r > 0 ? v[k] + sums[D + e] : v[k];
      }
    }
  }
}

// Wider rows: dx by a block a row, read twice, and the columns' sums by a kernel of their own: 4096 x 16384 bfloat16 with the residual's
// gradient 313 us, a quarter of a copy's rate.
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

// The parts' sums, of dw (blockIdx.y 0) and db: a block has 32 columns, its 32 warps take every 32nd part.
__global__ void __launch_bounds__(1024) back_sum_kernel(const float* partial, float* dw, float* db, long long D, long long parts) {
  __shared__ float sums[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long e = (long long)blockIdx.x * 32 + lane;
  const float* p = partial + blockIdx.y * D + e;
  float sum = 0.f;
  wait_for_first();
  if (e < D) {
#pragma unroll 4
    for (long long i = warp; i < parts; i += 32) sum += p[2 * i * D];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  sum = warp_sum(sums[lane][warp]);   // column `warp` of the block
  const long long c = (long long)blockIdx.x * 32 + warp;
  if (lane == 0 && c < D) (blockIdx.y ? db : dw)[c] = sum;
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
                      whole(a.dx, a.dx_row, SX) && (!a.dres || whole(a.dres, a.dres_row, SX)) && whole(a.w, 0, 4);
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
  return launch_after(true, back_sum_kernel, dim3((unsigned int)((a.D + 31) / 32), a.db ? 2 : 1), 1024, s, a.partial, a.dw, a.db, a.D, parts);
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
