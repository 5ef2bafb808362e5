// Root-mean-square norm with the residual's addition and an output in 8 bits:
//   r = x + residual (float32; residual <- r in its own type),  v = r / sqrt(mean(r^2) + eps) * w,
//   and either v in x's type, or codes q with scale = max|v| / 448 (e4m3) or / 127 (integers) over a
//   row or over every 128 values, q = v / scale rounded to nearest even.
// A scale below the smallest normal float32 (a row of zeros) is 1; a NaN makes its scale NaN.
//
// One pass: a row stays in the registers of its threads between the sum of squares, the maximum and
// the rounding, so x and the residual are read once and every output written once (7 bytes a value
// for bfloat16 with a residual and e4m3): memory bound, with an instruction count close behind (so
// values are taken in packed pairs and the warp's maximum is one integer reduction of their bits).
// 16384 x 4096 of that kind: 82.3 us, 5.71 TB/s, 84 % of a plain copy's rate, warp issue 71 % busy.
// Rows that start unaligned: 4099 x 1001 float32 12.3 us (9.3 on the GPU), 20000 x 3333 bfloat16 with
// residual to e4m3 130 us, 3.6 TB/s.
// v is taken as (r w) / sqrt(..): the largest |v| of a row is then the largest |r w| times the same
// factor, and the sum and the maximum are reduced together, one barrier a row.  Blocks are persistent: w stays in registers
// and the next row is loaded before the present one is reduced.  A row has `tpr` threads (whole
// warps), each with NV vectors of VEC adjacent values (16 bytes where alignment allows); short rows
// share a block.  Sums run in float32 in a fixed order: the same bits every time.
#include "vla.h"
#include "vla_layer.cuh"

#include <atomic>

namespace vla {
namespace {

// The larger of two, a NaN if either is one (then without a sign: 0x7fffffff).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// The largest of a warp's magnitudes, in every lane: they compare like their bits, and a NaN lies
// above them all.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// The 16 (sizeof 2) or fewer values of a vector as float32 pairs, and back with one rounding.
template <typename T, int N>
__device__ __forceinline__ void widen(const Vec<T, N>& x, uint64_t (&p)[(N + 1) / 2]) {
  if constexpr (N == 1) {
    p[0] = pair(to_f32<T>(x.v[0]), 0.f);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x.raw);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = pair(lo_f(w[i]), hi_f(w[i]));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = pair(to_f32<T>(x.v[2 * i]), to_f32<T>(x.v[2 * i + 1]));
  }
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> narrow(const uint64_t (&p)[(N + 1) / 2]) {
  Vec<T, N> x;
  float a, b;
  if constexpr (N == 1) {
    unpair(p[0], a, b);
    x.v[0] = from_f32<T>(a);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      unpair(p[i], a, b);
      if constexpr (sizeof(T) == 2) {
        reinterpret_cast<uint32_t*>(&x.raw)[i] = pack2(a, b);
      } else {
        x.v[2 * i] = from_f32<T>(a);
        x.v[2 * i + 1] = from_f32<T>(b);
      }
    }
  }
  return x;
}

// N values to N codes: e4m3 saturated to 448, or integers to nearest even.  A NaN keeps e4m3's
// code for it and gives the integer 0 (its scale is NaN).
template <int OUT, int N>
__device__ __forceinline__ void codes(const float (&v)[N], unsigned char* o) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    if (OUT == VLA_OUT_E4M3) {
      unsigned short r;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v[i + 1]), "f"(v[i]));
      o[i] = (unsigned char)(r & 0xff);
      o[i + 1] = (unsigned char)(r >> 8);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int r;
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(v[i + j]));
        o[i + j] = (unsigned char)r;
      }
    }
  }
  if (N == 1) {
    if (OUT == VLA_OUT_E4M3) {
      o[0] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
      int r;
      asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(v[0]));
      o[0] = (unsigned char)r;
    }
  }
}

// Scale and factors of values r w whose largest magnitude is m: v / scale = r w (full / m), rstd cancels
// and with it its error.  full / m passes float32's range for m below 2^-119, where the scale can still be
// a normal number (rstd is 1000 for a row of such values with eps 1e-6): where f is infinite, r w and m
// are first multiplied by kLift (the branch for it: 81.4 -> 82.3 us at 16384 x 4096).
constexpr float kLift = 0x1p100f;
__device__ __forceinline__ void norm_factors(float m, float rstd, float full, float& scale, float& f) {
  scale = m * rstd / full;
  f = full / m;
  if (scale < 1.17549435e-38f) {   // false for a NaN
    scale = 1.f;
    f = rstd;
  }
}

// RES: 0 none, 1 bfloat16, 2 float32
template <typename T, int RES, int OUT, int VEC, int NV>
__global__ void __launch_bounds__(NV <= 2 ? 512 : 1024) rms_norm_kernel(const NormArgs a, int tpr, int rows_per_cta, float inv_d) {
  using R = typename std::conditional<RES == 1, __nv_bfloat16, float>::type;
  constexpr int RV = sizeof(R) * VEC > 16 ? 16 / (int)sizeof(R) : VEC;   // 16 bytes an access
  constexpr bool QUANT = OUT != VLA_OUT_IO;
  __shared__ float part_ss[2][32], part_top[2][32];
  __shared__ float gmax[2][VEC == 1 && QUANT ? NV * 32 : 1];
  const int slot = threadIdx.x / tpr, tid = threadIdx.x - slot * tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = slot * (tpr >> 5), wn = tpr >> 5;
  const int D = (int)a.D;

  constexpr int PAIRS = (VEC + 1) / 2, RP = (RV + 1) / 2;
  uint64_t w[NV][PAIRS];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * tpr + tid) * VEC;
#pragma unroll
    for (int v = 0; v < PAIRS; ++v) {
      const float w0_ = e < D ? a.w[e + 2 * v] : 0.f, w1_ = VEC > 1 && e < D ? a.w[e + 2 * v + 1] : 0.f;
      w[i][v] = pair(w0_, w1_);
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
      in[i].raw = __ldcs(reinterpret_cast<const decltype(in[i].raw)*>(x + e));   // read once
      if (RES != 0) {
#pragma unroll
        for (int j = 0; j < VEC / RV; ++j) res[i][j].raw = __ldcs(reinterpret_cast<const decltype(res[i][j].raw)*>(r + e + j * RV));
      }
    }
  };
  const long long step = (long long)gridDim.x * rows_per_cta;
  long long row = (long long)blockIdx.x * rows_per_cta + slot;
  load(row);
  int span = 2;   // the power of two from wn on
  while (span < wn) span *= 2;
  int par = 0;
  for (long long first = (long long)blockIdx.x * rows_per_cta; first < a.rows; first += step, row += step, par ^= 1) {
    const bool live = row < a.rows;
    uint64_t r[NV][PAIRS], sum = 0;   // r w; the squares' sums (two zeros)
    float all = 0.f, top[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + tid) * VEC;
      top[i] = 0.f;
      if (live && e < D) {
        widen<T, VEC>(in[i], r[i]);
        if (RES != 0) {
#pragma unroll
          for (int j = 0; j < VEC / RV; ++j) {
            uint64_t p[RP];
            widen<R, RV>(res[i][j], p);
#pragma unroll
            for (int v = 0; v < RP; ++v) p[v] = r[i][j * RP + v] = add2(r[i][j * RP + v], p[v]);
            st_vec<R, RV>(static_cast<R*>(a.residual) + row * a.res_row + e + j * RV, narrow<R, RV>(p));
          }
        }
#pragma unroll
        for (int v = 0; v < PAIRS; ++v) {
          sum = fma2(r[i][v], r[i][v], sum);
          r[i][v] = mul2(r[i][v], w[i][v]);
          float p, q;
          unpair(r[i][v], p, q);
          if (QUANT) top[i] = max_nan(max_nan(top[i], fabsf(p)), fabsf(q));
        }
        if (QUANT) all = max_nan(all, top[i]);
      } else {
#pragma unroll
        for (int v = 0; v < PAIRS; ++v) r[i][v] = 0;
      }
    }
    load(row + step);
    // sum of squares and maximum over the row
    float s0, s1;
    unpair(sum, s0, s1);
    float ss = s0 + s1;
    const bool row_top = QUANT && a.group == 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (row_top) all = warp_max(all);
    if (QUANT && VEC == 1 && a.group) {   // a group is 4 warps (tpr is a multiple of 128 here)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        top[i] = warp_max(top[i]);
        if (lane == 0) gmax[par][i * 32 + warp] = top[i];
      }
    }
    if (wn > 1) {
      // the other half of `part` is still read by warps that are a row behind
      if (lane == 0) {
        part_ss[par][warp] = ss;
        if (row_top) part_top[par][warp] = all;
      }
      __syncthreads();
      const int at = lane & (span - 1);   // every lane ends up with the row's sum
      ss = at < wn ? part_ss[par][w0 + at] : 0.f;
      for (int o = span >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (row_top) all = warp_max(at < wn ? part_top[par][w0 + at] : 0.f);
    }
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
    if (!QUANT) {
      T* y = static_cast<T*>(a.y) + row * a.y_row;
      const uint64_t f2 = pair(rstd, rstd);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + tid) * VEC;
        if (!live || e >= D) continue;
#pragma unroll
        for (int v = 0; v < PAIRS; ++v) r[i][v] = mul2(r[i][v], f2);
        st_vec<T, VEC>(y + e, narrow<T, VEC>(r[i]));
      }
      continue;
    }
    unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.y_row;
    const float full = OUT == VLA_OUT_E4M3 ? 448.f : 127.f;
    const int groups = (D + 127) / 128;
    float scale, f;
    auto factors = [&](float m) { norm_factors(m, rstd, full, scale, f); };
    if (!a.group) factors(all);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (a.group) {
        if (VEC > 1) {
#pragma unroll
          for (int o = 64 / VEC; o > 0; o >>= 1) top[i] = max_nan(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        } else {
          const float* g = gmax[par] + i * 32 + (warp & ~3);
          top[i] = max_nan(max_nan(g[0], g[1]), max_nan(g[2], g[3]));
        }
        factors(top[i]);
      }
      const int e = (i * tpr + tid) * VEC;
      if (!live || e >= D) continue;
      float fi = f;
      if (fi == INFINITY) {
        fi = full / ((a.group ? top[i] : all) * kLift);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) r[i][j] = mul2(r[i][j], pair(kLift, kLift));
      }
      const uint64_t f2 = pair(fi, fi);
      float v[2 * PAIRS];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) unpair(mul2(r[i][j], f2), v[2 * j], v[2 * j + 1]);
      if constexpr (VEC == 1) {
        const float one[1] = {v[0]};
        codes<OUT, 1>(one, y + e);
      } else {
        Vec<unsigned char, VEC> o;
        codes<OUT, VEC>(v, o.v);
        st_vec<unsigned char, VEC>(y + e, o);
      }
      if (a.group) {
        if (e % 128 == 0) a.scale[row * groups + e / 128] = scale;
      } else if (e == 0) {
        a.scale[row] = scale;
      }
    }
  }
}

template <typename T, int RES, int OUT, int VEC, int NV>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  auto kern = rms_norm_kernel<T, RES, OUT, VEC, NV>;
  const int unit = VEC == 1 && a.group ? 128 : 32;
  const long long need = (a.D + (long long)VEC * NV - 1) / ((long long)VEC * NV);
  const int tpr = (int)((need + unit - 1) / unit * unit);
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  // blocks an SM for this kernel and block size: asked for once, packed as size | blocks
  static std::atomic<unsigned int> known{0};
  const unsigned int threads = (unsigned int)(tpr * rows);
  unsigned int k = known.load(std::memory_order_relaxed);
  if (k >> 16 != threads) {
    int blocks = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kern, (int)threads, 0);
    if (e != cudaSuccess) return e;
    k = threads << 16 | (unsigned int)blocks;
    known.store(k, std::memory_order_relaxed);
  }
  const int per_sm = (int)(k & 0xffffu);
  const long long all = (a.rows + rows - 1) / rows, most = (long long)(per_sm > 0 ? per_sm : 1) * a.sm_count;
  kern<<<(unsigned int)(all < most ? all : most), tpr * rows, 0, s>>>(a, tpr, rows, 1.f / (float)a.D);
  return cudaGetLastError();
}

// Rows off 16-byte boundaries, most of them (launch_odd): a row's group of warps copies it to shared memory, to
// a place with the same offset from a 16-byte boundary, so that all but its ends moves in 16-byte
// pieces; outputs leave the same way.  Blocks of 128 values belong to a warp each, 4 values a lane.  No row is
// fetched ahead (that took a third more: the memory of a second row costs as many warps).
constexpr int kOddThreads = 256;

constexpr int kOddMost = 200 * 1024;   // bytes of shared memory
__host__ __device__ constexpr long long odd_bytes(long long n, int size) { return (n * size + 16 + 15) / 16 * 16; }

// n values at p, moved by threads t of nt: `head` single ones, `pieces` of 16 bytes, then the rest.
template <typename V>
struct Span {
  static constexpr int E = 16 / (int)sizeof(V);
  int head, pieces, rest;
  __device__ __forceinline__ Span(const V* p, int n) {
    head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (int)sizeof(V);
    if (head > n) head = n;
    pieces = (n - head) / E;
    rest = head + pieces * E;   // where the rest begins
  }
};
template <typename V>
__device__ __forceinline__ V* odd_place(unsigned char* region, const V* p) {
  return reinterpret_cast<V*>(region + (reinterpret_cast<uintptr_t>(p) & 15u));
}
template <typename V>
__device__ __forceinline__ void odd_in(unsigned char* region, const V* p, int n, int t, int nt) {
  const Span<V> s(p, n);
  V* to = odd_place(region, p);
  const uint32_t at = smem_u32(to + s.head);
  for (int i = t; i < s.pieces; i += nt)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 16 * i), "l"(p + s.head + i * Span<V>::E) : "memory");
  if (t < s.head) to[t] = p[t];
  if (t < n - s.rest) to[s.rest + t] = p[s.rest + t];
}
template <typename V>
__device__ __forceinline__ void odd_out(unsigned char* region, V* p, int n, int t, int nt) {
  const Span<V> s(p, n);
  const V* from = odd_place(region, p);
  for (int i = t; i < s.pieces; i += nt)
    *reinterpret_cast<uint4*>(p + s.head + i * Span<V>::E) = *reinterpret_cast<const uint4*>(from + s.head + i * Span<V>::E);
  if (t < s.head) p[t] = from[t];
  if (t < n - s.rest) p[s.rest + t] = from[s.rest + t];
}

template <typename T, int RES, int OUT>
__global__ void __launch_bounds__(kOddThreads) rms_norm_odd_kernel(const NormArgs a, int warps, float inv_d) {
  using R = typename std::conditional<RES == 1, __nv_bfloat16, float>::type;
  using Y = typename std::conditional<OUT == VLA_OUT_IO, T, unsigned char>::type;
  constexpr bool QUANT = OUT != VLA_OUT_IO;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part_ss[kOddThreads / 32], part_top[kOddThreads / 32];
  const int nt = warps * 32, grp = threadIdx.x / nt, t = threadIdx.x - grp * nt, lane = t & 31, gw = t >> 5;
  const int D = (int)a.D, groups = (D + 127) / 128;
  const long long x_bytes = odd_bytes(D, sizeof(T)), r_bytes = RES ? odd_bytes(D, sizeof(R)) : 0;
  float* rw = reinterpret_cast<float*>(smem + grp * (x_bytes + r_bytes + odd_bytes(D, 4)));   // r w
  unsigned char* xs = reinterpret_cast<unsigned char*>(rw) + odd_bytes(D, 4);   // x, later y
  unsigned char* rs = xs + x_bytes;
  auto sync = [&]() {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(nt) : "memory");
  };
  const int per = kOddThreads / nt;
  const long long step = (long long)gridDim.x * per;
  for (long long row = (long long)blockIdx.x * per + grp; row < a.rows; row += step) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    R* res = static_cast<R*>(a.residual) + row * a.res_row;
    Y* y = static_cast<Y*>(a.y) + row * a.y_row;
    odd_in<T>(xs, x, D, t, nt);
    if (RES) odd_in<R>(rs, res, D, t, nt);
    asm volatile("cp.async.wait_all;" ::: "memory");
    sync();
    const T* xr = odd_place(xs, x);
    R* rr = RES ? odd_place(rs, res) : nullptr;
    float ss = 0.f, all = 0.f;
    auto first = [&](int e) {
      float r = to_f32<T>(xr[e]);
      if (RES) {
        r += to_f32<R>(rr[e]);
        rr[e] = from_f32<R>(r);
      }
      ss = fmaf(r, r, ss);
      r *= a.w[e];
      rw[e] = r;
      if (QUANT) all = max_nan(all, fabsf(r));
    };
    for (int b = gw; b < groups; b += warps) {
      const int e = b * 128 + lane;
      if ((b + 1) * 128 <= D) {
#pragma unroll
        for (int j = 0; j < 4; ++j) first(e + 32 * j);
      } else {
        for (int j = e; j < D; j += 32) first(j);
      }
    }
    const bool row_top = QUANT && a.group == 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (row_top) all = warp_max(all);
    if (warps > 1 && lane == 0) {
      part_ss[grp * warps + gw] = ss;
      part_top[grp * warps + gw] = all;
    }
    sync();   // the row's r and rw are there, x is done with
    if (warps > 1) {
      const float* ps = part_ss + grp * warps;
      const float* pt = part_top + grp * warps;
      ss = 0.f;
      for (int i = 0; i < warps; ++i) {
        ss += ps[i];
        if (row_top) all = max_nan(all, pt[i]);
      }
    }
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
    const float full = OUT == VLA_OUT_E4M3 ? 448.f : 127.f;
    float scale, f = rstd, lift = 1.f;
    auto factors = [&](float m) {
      norm_factors(m, rstd, full, scale, f);
      lift = f == INFINITY ? kLift : 1.f;
      if (f == INFINITY) f = full / (m * kLift);
    };
    if (row_top) {
      factors(all);
      if (t == 0) a.scale[row] = scale;
    }
    Y* yr = odd_place(xs, y);
    for (int b = gw; b < groups; b += warps) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = b * 128 + j * 32 + lane;
        v[j] = e < D ? rw[e] : 0.f;
      }
      if (QUANT && a.group) {
        factors(warp_max(max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])))));
        if (lane == 0) a.scale[row * groups + b] = scale;
      }
      const bool whole = (b + 1) * 128 <= D;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = b * 128 + j * 32 + lane;
        const float one[1] = {v[j] * lift * f};
        if (!whole && e >= D) continue;
        if constexpr (QUANT) codes<OUT, 1>(one, yr + e);
        else yr[e] = from_f32<T>(one[0]);
      }
    }
    sync();
    odd_out<Y>(xs, y, D, t, nt);
    if (RES) odd_out<R>(rs, res, D, t, nt);
    sync();   // before the next row comes in
  }
}

// Values a thread: few, so that many threads have a load in flight (16384 x 4096 bfloat16 with residual
// and e4m3, before values were taken in pairs: 8 values 87 us, 16 values 94 us, 32 values 195 us).
template <typename T, int RES, int OUT, int VEC>
cudaError_t by_width(const NormArgs& a, cudaStream_t s) {
  if constexpr (VEC > 1) {
    if (a.D <= 512LL * VEC) return launch<T, RES, OUT, VEC, 1>(a, s);
    if (a.D <= 1024LL * VEC) return launch<T, RES, OUT, VEC, 2>(a, s);
  }
  if (a.D <= 4096LL * VEC) return launch<T, RES, OUT, VEC, 4>(a, s);
  return launch<T, RES, OUT, VEC, 32 / VEC>(a, s);   // up to 32768 values (the entry point's limit)
}

// Rows off 16-byte boundaries.  Value by value from global memory where that is quicker: few rows (a
// shorter chain; 152 rows of 3333 bfloat16 to e4m3 3.9 us against 5.9, 608 rows 11.3 against 7.0; 608
// rows of 1001 4.3 against 6.5), or narrow ones and float32 without a residual (100000 x 65 float32 19 us
// against 33, 40990 x 1001 77 against 83, 50000 x 255 bfloat16 23.7 against 25).  Else through shared
// memory (20000 x 3333 bfloat16 with residual to e4m3 130 us against 424, 40000 x 1001 82 against 197,
// 20000 x 1001 float32 with residual 79 against 98), where a row fits there.
template <typename T, int RES, int OUT>
cudaError_t launch_odd(const NormArgs& a, cudaStream_t s) {
  const bool few = a.D <= 4096 && a.rows <= 4096LL * a.sm_count / a.D;
  if (few || (RES == 0 && a.D <= (sizeof(T) == 4 ? 2048 : 256))) return by_width<T, RES, OUT, 1>(a, s);
  const int warps = a.D <= 1024 ? 1 : a.D <= 2048 ? 2 : a.D <= 4096 ? 4 : 8, per = kOddThreads / 32 / warps;
  const long long bytes =
      per * (odd_bytes(a.D, sizeof(T)) + (RES ? odd_bytes(a.D, RES == 1 ? 2 : 4) : 0) + odd_bytes(a.D, 4));
  if (bytes > kOddMost) return by_width<T, RES, OUT, 1>(a, s);
  auto kern = rms_norm_odd_kernel<T, RES, OUT>;
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kOddMost);
    if (e != cudaSuccess) return e;
  }
  // blocks an SM for these bytes: asked for once, packed as bytes | blocks
  static std::atomic<unsigned int> known{0};
  unsigned int k = known.load(std::memory_order_relaxed);
  if (k >> 8 != (unsigned int)bytes) {
    int blocks = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kern, kOddThreads, (size_t)bytes);
    if (e != cudaSuccess) return e;
    k = (unsigned int)bytes << 8 | (unsigned int)blocks;
    known.store(k, std::memory_order_relaxed);
  }
  const long long all = (a.rows + per - 1) / per, most = (long long)((k & 0xffu) ? k & 0xffu : 1) * a.sm_count;
  kern<<<(unsigned int)(all < most ? all : most), kOddThreads, (size_t)bytes, s>>>(a, warps, 1.f / (float)a.D);
  return cudaGetLastError();
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
  return ok ? by_width<T, RES, OUT, VEC>(a, s) : launch_odd<T, RES, OUT>(a, s);
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
