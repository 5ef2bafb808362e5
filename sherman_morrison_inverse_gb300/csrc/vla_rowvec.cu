// Products of a few rows (single tokens): y = x w^T with its epilogue for M up to 8 at a time, on CUDA cores.
//
// Every weight is read once for 8 rows of x, and that bounds it.  A warp takes 4 rows of w and all of Kd (or a
// share of it, where there are too few rows to fill the SMs: the shares of a block's warps are then added in shared memory):
// its lanes read 16 bytes of each row at a time, several steps ahead, and x comes from the first-level cache.  Products
// and sums are float32 in packed pairs.  A warp's sums are folded over the lanes together, so that
// every lane ends with one of them.
// Rows off 16-byte boundaries, or Kd in no whole pieces, are read value by value.
// One row, us a launch in a row of them whose weights pass L2 (by itself 2 to 3 more): N 8192, K 8192 bfloat16 21.9 (6.1 TB/s,
// 92 % of a copy's rate), e4m3 14.9 (4.5 TB/s), float32 47.3 (5.7 TB/s); N 8512, K 2048 bfloat16 7.7; N 520, K 264 2.6.  Eight
// rows of float32 N 8192, K 8192: 81, by arithmetic and the first-level cache.
#include "vla_dense.cuh"

namespace vla {
namespace {

// 16 bytes as float32 pairs.
template <typename T>
struct Wide {
  static constexpr int E = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void widen(const uint4& x, uint64_t (&p)[E / 2]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4) {
      p[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
      p[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = pair(lo_f(w[i]), hi_f(w[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(w[i]));
        const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a)), v = __half22float2(*reinterpret_cast<const __half2*>(&b));
        p[2 * i] = pair(u.x, u.y);
        p[2 * i + 1] = pair(v.x, v.y);
      }
    }
  }
};

// y's element, the epilogue of a single sum.
template <typename TY>
__device__ __forceinline__ void out_one(const Epilogue& e, float v, long long m, long long n) {
  if (e.x_scale) v *= e.x_scale[m];
  if (e.w_scale) v *= e.w_scale[n];
  if (e.bias) v += e.bias[n];
  if (e.pre) static_cast<TY*>(e.pre)[m * e.pre_row + n] = from_f32<TY>(v);
  v = activate<sizeof(TY) == 2>(v, e.act);
  if (e.residual) v += to_f32<TY>(static_cast<const TY*>(e.residual)[m * e.res_row + n]);
  static_cast<TY*>(e.y)[m * e.y_row + n] = from_f32<TY>(v);
}

// MT: rows of x at a time; R: rows of w a warp; AHEAD: steps whose loads are in flight together.
template <typename T, bool VEC, int MT, int R, int AHEAD>
__global__ void __launch_bounds__(256, 2) few_rows_kernel(const ProductArgs p, int shares) {
  constexpr int E = VEC ? Wide<T>::E : 1;
  __shared__ float part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = 8 / shares, group = warp / shares, share = warp - group * shares;
  const long long n0 = ((long long)blockIdx.x * groups + group) * R;
  const long long m0 = (long long)blockIdx.y * MT;
  const T* x = static_cast<const T*>(p.a) + m0 * p.a_row;
  const T* w = static_cast<const T*>(p.b) + n0 * p.b_row;
  uint64_t acc[R][MT] = {};
  if (n0 < p.N) {
    const long long pieces = (p.Kd + 32 * E - 1) / (32 * E);   // steps of the whole warp
    const long long s0 = pieces * share / shares, s1 = pieces * (share + 1) / shares;
    for (long long s = s0; s < s1; s += AHEAD) {
      if constexpr (VEC) {
        uint4 wv[AHEAD][R];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const long long k = ((s + i) * 32 + lane) * E;
          const bool on = s + i < s1 && k < p.Kd;
#pragma unroll
          for (int r = 0; r < R; ++r)
            wv[i][r] = on && n0 + r < p.N ? __ldcs(reinterpret_cast<const uint4*>(w + r * p.b_row + k)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const long long k = ((s + i) * 32 + lane) * E;
          const bool on = s + i < s1 && k < p.Kd;
          uint64_t wp[R][E / 2];
#pragma unroll
          for (int r = 0; r < R; ++r) Wide<T>::widen(wv[i][r], wp[r]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint64_t xp[E / 2];
            Wide<T>::widen(on && m0 + m < p.M ? *reinterpret_cast<const uint4*>(x + m * p.a_row + k) : make_uint4(0, 0, 0, 0), xp);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int j = 0; j < E / 2; ++j) acc[r][m] = fma2(wp[r][j], xp[j], acc[r][m]);
          }
        }
      } else {
        T wv[AHEAD][R], xv[AHEAD][MT];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const long long k = (s + i) * 32 + lane;
          const bool on = s + i < s1 && k < p.Kd;
#pragma unroll
          for (int r = 0; r < R; ++r) wv[i][r] = on && n0 + r < p.N ? w[r * p.b_row + k] : T(0.f);
#pragma unroll
          for (int m = 0; m < MT; ++m) xv[i][m] = on && m0 + m < p.M ? x[m * p.a_row + k] : T(0.f);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              float lo, hi;
              unpair(acc[r][m], lo, hi);
              acc[r][m] = pair(fmaf(to_f32<T>(wv[i][r]), to_f32<T>(xv[i][m]), lo), hi);
            }
      }
    }
  }
  // fold: with V sums left, a lane keeps the half of them that the bit of its number says and adds its partner's
  constexpr int SUMS = R * MT;
  float v[SUMS];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float lo, hi;
      unpair(acc[r][m], lo, hi);
      v[m * R + r] = lo + hi;
    }
  int bit = 1;
#pragma unroll
  for (int left = SUMS; left > 1; left >>= 1, bit <<= 1) {
    const bool upper = lane & bit;
#pragma unroll
    for (int i = 0; i < left / 2; ++i) {
      const float mine = upper ? v[2 * i + 1] : v[2 * i], other = upper ? v[2 * i] : v[2 * i + 1];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
    }
  }
#pragma unroll
  for (; bit < 32; bit <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  // lane l has sum l % SUMS
  if (shares > 1) {
    part[warp][lane] = v[0];
    __syncthreads();
    if (share > 0) return;
    v[0] = 0.f;
    for (int i = 0; i < shares; ++i) v[0] += part[warp + i][lane];
  }
  const long long n = n0 + lane % R, m = m0 + lane / R;
  if (lane >= SUMS || n >= p.N || m >= p.M) return;
  if (p.out.y_bf16) out_one<__nv_bfloat16>(p.out, v[0], m, n);
  else out_one<float>(p.out, v[0], m, n);
}

template <typename T, bool VEC, int MT>
cudaError_t launch(const ProductArgs& p, cudaStream_t s) {
  // AHEAD: what 128 registers hold.  (Two rows of w a warp and 8 steps for a single row of x: 25.6 us against 24.6 with N 8192,
  // K 8192, 7.8 against 6.6 with N 2048, K 4096.)
  constexpr int E = Wide<T>::E, R = 4;
  constexpr int AHEAD = !VEC ? (MT <= 4 ? 8 : 4) : E * MT <= 16 ? 4 : E * MT <= 32 ? 2 : 1;
  // as many shares of Kd as keep the warps within 16 an SM, which is one wave, of 4 steps at least
  const long long rows = (p.N + R - 1) / R, tall = (p.M + MT - 1) / MT;
  const long long pieces = p.Kd / (32 * (VEC ? Wide<T>::E : 1));
  int shares = 1;
  while (shares < 8 && 2 * rows * tall * shares <= 16LL * p.sm_count && pieces >= 8LL * shares) shares *= 2;
  const dim3 grid((unsigned int)((rows * shares + 7) / 8), (unsigned int)tall);
  few_rows_kernel<T, VEC, MT, R, AHEAD><<<grid, 256, 0, s>>>(p, shares);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_of(const ProductArgs& p, cudaStream_t s) {
  auto whole = [](const void* x, long long row) {
    return ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)((size_t)row * sizeof(T))) & 15u) == 0;
  };
  const bool vec = p.Kd % Wide<T>::E == 0 && whole(p.a, p.M > 1 ? p.a_row : 0) && whole(p.b, p.N > 1 ? p.b_row : 0);
  auto run = [&](auto v) -> cudaError_t {
    constexpr bool VEC = decltype(v)::value;
    if (p.M == 1) return launch<T, VEC, 1>(p, s);
    if (p.M == 2) return launch<T, VEC, 2>(p, s);
    return p.M <= 4 ? launch<T, VEC, 4>(p, s) : launch<T, VEC, 8>(p, s);
  };
  return vec ? run(std::true_type()) : run(std::false_type());
}

}  // namespace

cudaError_t launch_few_rows(const ProductArgs& p, int mat, cudaStream_t s) {
  if (mat == kMatF32) return launch_of<float>(p, s);
  return mat == kMatBf16 ? launch_of<__nv_bfloat16>(p, s) : launch_of<__nv_fp8_e4m3>(p, s);
}

}  // namespace vla
