// Products of some ten to a hundred rows of x on the tensor cores: y = x w^T with its epilogue.
//
// The weights bound it: each is read once, and there are more of them than of anything else.  So the roles are swapped:
// 128 rows of w are the long side of the tensor core's product and 16 to 128 rows of x the short one, and Kd is shared by
// the 1 to 8 CTAs of a cluster, so that w arrives over all SMs: a ring of 3 to 5 stages of 16 KB of w a CTA, two
// CTAs an SM, keeps what memory's latency needs in flight.  Each CTA leaves its sums in its shared memory, one float32 row a token,
// and each then adds a share of the tokens from all of them, in order, over distributed shared memory, and takes it
// through the epilogue: no pass over memory and no second launch.
// Sums move from tensor memory to float32 registers every 4 stages (see vla_gemm.cu).  Waits are bounded; a CTA that gives up waits
// (bounded too) for its products and copies under way.
// us a launch in a row of them whose weights pass L2 (by itself 1 to 6 more): N 8192, K 8192 with 16 to 128 rows, bfloat16 26.2 to
// 31.8 (5.1 to 4.2 TB/s), e4m3 16.1 to 20.6 (4.2 to 3.3 TB/s), float32 with 32 to 128 rows 212 to 224, of which the copies of the
// weights' three terms are the most; bfloat16 N 2048, K 4096 with 128 rows 10.7; N 520, K 264 with 16 rows 4.3, which is what
// a call costs before its size does.
#include <atomic>

#include "vla_gemm.cuh"

namespace vla {
namespace gemm {
namespace {

constexpr int kThreads = 320;   // a producer, an issuer, eight warps of the epilogue

template <int BT>
struct Cfg {
  static constexpr int stages = 96 * 1024 / (128 * 128 + BT * 128);   // two CTAs an SM
  static constexpr uint32_t w_bytes = 128 * 128, x_bytes = BT * 128, stage = w_bytes + x_bytes;
  static constexpr uint32_t o_bar = stages * stage, bars = 2 * stages + 5;
  static constexpr uint32_t bytes = o_bar + 8 * bars + 16;
  static constexpr uint32_t cols = 2 * BT;
};

template <bool E4M3>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t one) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ void tma(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void ld8(uint32_t at, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[j]);
}

template <typename T, int BT, bool E4M3>
__global__ void __launch_bounds__(kThreads, 2)
    tokens_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const GemmArgs g) {
  using C = Cfg<BT>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::o_bar);
  uint64_t *empty = full + C::stages, *acc_full = empty + C::stages, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* failed = slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();   // the share of Kd
  const long long n0 = (long long)(blockIdx.x / g.splits) * 128, m0 = (long long)blockIdx.y * BT;
  const int k0 = k_begin(g, rank), k1 = k_begin(g, rank + 1);

  // the producer's place in the ring and in Kd
  uint32_t stage = 0, phase = 1, issued = 0;
  int k = k0, pass = k0 / g.k_iters, it = k0 - pass * g.k_iters;
  auto fill = [&]() {
    const uint32_t sw = base + stage * C::stage;
    constexpr int BK = E4M3 ? 128 : 64;
    mbar_arrive_expect_tx(full + stage, C::stage);
    tma(sw, &map_w, it * BK, (int)n0, g.passes > 1 ? term_b(pass) : 0, full + stage);
    tma(sw + C::w_bytes, &map_x, it * BK, (int)m0, g.passes > 1 ? term_a(pass) : 0, full + stage);
    ++k;
    ++issued;
    if (++stage == C::stages) {
      stage = 0;
      phase ^= 1;
    }
    if (++it == g.k_iters) {
      it = 0;
      ++pass;
    }
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 8);
    }
    mbar_init(drain, 1);
    *failed = (base & 1023u) != 0;   // the swizzled tiles need it; report rather than run misaligned
    fence_mbar_init();
    fence_proxy_async_smem();
    if (!*failed)
      while (issued < C::stages && k < k1) fill();   // nothing to wait for yet
  }
  if (warp == 1) tc::tmem_alloc(slot, C::cols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;

  if (warp == 0) {
    if (lane == 0 && !*failed) {
      while (k < k1 && wait_for(empty + stage, phase, g.limit, failed)) fill();
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t one = lane == 0;
    constexpr uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t)(BT >> 3) << 17 | (128u >> 4) << 24;
    uint32_t at = 0, at_phase = 0, buf = 0, buf_phase = 1;
    bool ok = !*failed;
    for (int k = k0; ok && k < k1;) {
      const int end = part_end(g, k, k1);
      if (!(ok = wait_for(acc_empty + buf, buf_phase, g.limit, failed))) break;
      tc::fence_after_sync();
      for (bool more = false; k < end; ++k, more = true) {
        if (!(ok = wait_for(full + at, at_phase, g.limit, failed))) break;
        tc::fence_after_sync();
        const uint32_t sw = base + at * C::stage;
        const uint64_t dw = desc128(sw, 8192), dx = desc128(sw + C::w_bytes, 8192);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_one<E4M3>(tmem + buf * BT, dw + 2 * i, dx + 2 * i, idesc, more || i > 0, one);
        commit_one(empty + at, one);
        if (++at == C::stages) {
          at = 0;
          at_phase ^= 1;
        }
      }
      if (!ok) break;
      commit_one(acc_full + buf, one);
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1;
      }
    }
    commit_one(drain, one);   // whoever gave up: no product reads the ring behind this
    mbar_wait_bounded(drain, 0);
  } else {
    // a lane has a row of w (its tensor memory lane) and the sums of half the tokens
    constexpr int HT = BT / 2, W = HT < 32 ? HT : 32;
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + half * HT;
    float sums[HT] = {};
    uint32_t buf = 0, buf_phase = 0;
    bool ok = g.limit > 0;   // 0: the wait's self-test, the others find out with copies and products under way
    if (!ok) *failed = 1;
    for (int k = k0; ok && k < k1; k = part_end(g, k, k1)) {
      if (!(ok = wait_warp(acc_full + buf, buf_phase, g.limit, failed))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int c = 0; c < HT / W; ++c) {
        float v[W];
        if constexpr (W == 8) ld8(from + buf * BT, v);
        else if constexpr (W == 16) tc::tmem_ld16(from + buf * BT, v);
        else tc::tmem_ld32(from + buf * BT + c * 32, v);
        if (c == HT / W - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(acc_empty + buf)) : "memory");
        }
#pragma unroll
        for (int j = 0; j < W; ++j) sums[c * W + j] += v[j];
      }
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1;
      }
    }
    // the last product is done and with it every read of the ring: it takes the sums
    float* row = reinterpret_cast<float*>(smem) + half * HT * 128 + quad * 32 + lane;
    if (ok) {
#pragma unroll
      for (int j = 0; j < HT; ++j) row[j * 128] = sums[j];
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *failed) drain_ring(full, C::stages, issued);
  __syncwarp();
  cluster_sync_all();   // every CTA's sums are there
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, C::cols);
  // a warp a token, a lane four columns; the shares of 8 / splits tokens are fetched together
  const long long n = n0 + lane * 4;
  const int left = g.N - n < 4 ? (int)(g.N - n) : 4;
  const int t0 = BT * rank / g.splits + warp, t1 = BT * (rank + 1) / g.splits;
  constexpr int STEP = kThreads / 32;
  auto join = [&](auto shares) {
    constexpr int S = decltype(shares)::value, AT = 8 / S;
    const Columns cols = columns_of(g.out, n, left);
    for (int t = t0; t < t1 && m0 + t < g.M; t += STEP * AT) {
      float u[AT][S][4];
      Vec<T, 4> res[AT];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int at = t + i * STEP;
        if (at >= t1 || m0 + at >= g.M) continue;
        if (g.out.residual) res[i] = load4<T>(static_cast<const T*>(g.out.residual) + (m0 + at) * g.out.res_row + n, g.res_vec, left);
#pragma unroll
        for (int r = 0; r < S; ++r)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(u[i][r][0]), "=f"(u[i][r][1]), "=f"(u[i][r][2]), "=f"(u[i][r][3])
                       : "r"(mapa_shared(base + at * 512 + lane * 16, r)));
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int at = t + i * STEP;
        if (at >= t1 || m0 + at >= g.M) continue;
        float v[4] = {};
#pragma unroll
        for (int r = 0; r < S; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += u[i][r][j];
        out4<T>(g, v, cols, res[i], m0 + at, n, left);
      }
    }
  };
  if (left > 0 && !*failed) {
    if (g.splits == 1) join(std::integral_constant<int, 1>());
    else if (g.splits == 2) join(std::integral_constant<int, 2>());
    else if (g.splits == 4) join(std::integral_constant<int, 4>());
    else join(std::integral_constant<int, 8>());
  }
  if (threadIdx.x == 0 && *failed) atomicOr(&g.status->flags, kStatusTimeout);
  __syncthreads();
  cluster_sync_all();   // no CTA leaves while others read its sums
}

template <typename T, int BT, bool E4M3>
cudaError_t launch(const TokensPlan& t, const GemmArgs& g, const Operand& x, const Operand& w, const void* x_at, const void* w_at,
                   cudaStream_t s) {
  CUtensorMap mx, mw;
  constexpr int BK = E4M3 ? 128 : 64;
  if (!encode(&mx, x, x_at, BK, BT) || !encode(&mw, w, w_at, BK, 128)) return cudaErrorInvalidValue;
  auto kern = tokens_kernel<T, BT, E4M3>;
  constexpr int bytes = (int)Cfg<BT>::bytes;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  // more than 48 KB of shared memory: allowed once a kernel and device (the first 64)
  static std::atomic<unsigned long long> ready{0};
  if (device >= 64 || !(ready.load(std::memory_order_relaxed) >> device & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (device < 64) ready.fetch_or(1ull << device, std::memory_order_relaxed);
  }
  const long long ctas = (g.N + 127) / 128 * t.splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned int)ctas, (unsigned int)((g.M + BT - 1) / BT));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = bytes;
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = t.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, mx, mw, g);
}

}  // namespace

// The narrowest tile that holds the rows, up to 64, or 128 where the weights are many: a tile of 64 has half the epilogue and twice
// the CTAs, and reads the weights twice, the second time from L2 (128 rows, bfloat16, us, tiles of 128 against 64: N 520,
// K 264: 8.4 against 6.7; N 2048, K 4096: 14.1 against 11.8; N 8192, K 8192: 38.1 against 40.6).  As many shares of Kd as keep
// the CTAs within two an SM, of two stages at least.
TokensPlan tokens_plan(long long M, long long N, long long w_values, int all_iters, int sm_count) {
  TokensPlan t{};
  t.rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 || w_values <= 1LL << 25 ? 64 : 128;
  t.splits = 1;
  const long long tiles = (N + 127) / 128 * ((M + t.rows - 1) / t.rows);
  while (t.splits < 8 && tiles * t.splits * 2 <= 2 * sm_count && all_iters >= 4 * t.splits) t.splits *= 2;
  return t;
}

cudaError_t launch_tokens(const TokensPlan& t, GemmArgs g, const Operand& x, const Operand& w, const void* x_at, const void* w_at,
                          cudaStream_t s) {
  g.splits = t.splits;
  g.part = kPart;
  auto run = [&](auto y, auto e4m3) -> cudaError_t {
    using T = decltype(y);
    constexpr bool E = decltype(e4m3)::value;
    if (t.rows == 16) return launch<T, 16, E>(t, g, x, w, x_at, w_at, s);
    if (t.rows == 32) return launch<T, 32, E>(t, g, x, w, x_at, w_at, s);
    if (t.rows == 64) return launch<T, 64, E>(t, g, x, w, x_at, w_at, s);
    return launch<T, 128, E>(t, g, x, w, x_at, w_at, s);
  };
  if (x.size == 1) return g.out.y_bf16 ? run(__nv_bfloat16(), std::true_type()) : run(float(), std::true_type());
  return g.out.y_bf16 ? run(__nv_bfloat16(), std::false_type()) : run(float(), std::false_type());
}

}  // namespace gemm
}  // namespace vla
