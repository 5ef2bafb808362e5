// Matrix products on the tensor cores: C [M, N] = sum over Kd of A B, with an epilogue.
//
// Two CTAs of a cluster share a tile of 256 x BN outputs (tcgen05.mma.cta_group::2): each holds 128 rows of A
// and BN / 2 columns of B in shared memory and 128 rows of the float32 sums in tensor memory.  Clusters are
// persistent and walk the tiles in blocks of 8 tiles of M, so that what runs at one time shares rows and columns in L2.
//   warp 0     one thread keeps a ring of stages filled by TMA: 128 bytes of Kd of both operands (64
//              bfloat16 or 128 e4m3), 128-byte swizzle.  Both CTAs' copies complete on the leader's barrier.
//   warp 1     of the leader issues the products of both CTAs, four a stage, into one of two accumulators.
//   warps 2, 3 only leave their registers to the others.
//   warps 4..11 take the other accumulator out, 32 columns of a lane's row at a time, through the epilogue to memory in
//              32-byte pieces; rows off 32-byte boundaries go through shared memory first.
// A launch holds one product, or the two of a gradient: their tiles follow one another, so that one's last wave is
// the other's first (8192 x 8192 x 2048, dx and dw: 345 us in two launches, 339 in one, of 4 + 4 and 7 waves).
// Operands lie in memory with Kd adjacent (as in x w^T) or with M or N adjacent (as in g w and g^T x): tiles
// of 64 along what is adjacent, and the matrix descriptors say which.
// float32 operands arrive as three bfloat16 terms each (x = x1 + x2 + x3 to 2^-24): six products, the small ones
// first.  Where the result is float32, sums stay in tensor memory for 4 stages and are then added to float32 registers:
// a tensor core cuts the bits off that an addition shifts out, always towards zero, and the error of a chain of them
// grows with its length (float32, K = 1161: 6.8e-7 of the result without, 1.4e-7 with; plain float32 products 3.6e-7).
// For results rounded to bfloat16 that matters where Kd is long, as a gradient's is by its tokens: terms of one sign come out
// smaller by 3.4e-5 after 128 stages (8192 of Kd, a hundredth of the rounding), by 3.3e-3 after 8192 (more than it).  A
// share of Kd of up to 128 stages stays in tensor memory whole; a longer one is added to registers every 64.
// Kd is split over clusters where there are fewer tiles than clusters; the parts are then added in order.
// Every wait is bounded: one that runs out sets the handle's timeout flag, and the cluster waits (bounded too) for the products and
// copies that both CTAs have under way and returns.
//
// What bounds it: the tensor pipe, and with it shared memory (a tile of 256 x 256 takes 64 bytes a cycle for the products'
// operands and 64 for the copies, all that there is; of 256 x 128 half as much again, so that its stages take as
// long).  bfloat16 8192 x 8192 x 2048: 148 us, 1.86 PFLOP/s, 99 % of cuBLAS's burst rate (with gelu 162); 32768 x 8512 x 2048
// in a row of calls, at the power limit: 701 us, 1.63 PFLOP/s, 96 % of cuBLAS's rate of that kind; e4m3 16384 x 2048 x 4096
// with a residual 99 us, 2.8 PFLOP/s.  With little Kd the epilogue bounds it: 8192 x 8192 x 512 51 us, with gelu 84 (four
// special functions a pair of values).
#include <atomic>

#include "vla_gemm.cuh"

namespace vla {

using namespace gemm;

namespace {

constexpr int kThreads = 384;
constexpr int kGroup = 8;          // tiles of M that are walked together
constexpr int kChunk = 32 * 32 * 4;   // a warp's staging: 32 rows of 32 float32

template <int BN>
struct Cfg {
  static constexpr int stages = BN == 256 ? 6 : 8;
  static constexpr uint32_t a_bytes = 128 * 128, b_bytes = BN / 2 * 128, stage = a_bytes + b_bytes;
  static constexpr uint32_t o_chunk = stages * stage, o_bar = o_chunk + 8 * kChunk;
  static constexpr uint32_t bars = 2 * stages + 5;
  static constexpr uint32_t bytes = o_bar + 8 * bars + 16;
  static constexpr uint32_t cols = 2 * BN;
};

// The products of a launch.  Forward: g[0] alone, Kd adjacent in both operands.  Backward: tiles [0, g[0].tiles) are dx's
// (B lies with N adjacent), the others dw's (both lie with M or N adjacent); either may have none.  Which layout a product has is
// known to the compiler: with descriptors' steps in registers the issue of the products takes a fifth longer.
struct GemmPair {
  GemmArgs g[2];
  DevStatus* status;
};
struct Maps {
  CUtensorMap a[2], b[2];
};

// One product of both CTAs for 32 bytes of Kd, issued by the lane whose `one` is set.  The whole warp runs the loop
// around it, predicated and not branched, so that descriptors stay in uniform registers.
template <bool E4M3>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t one) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
        : "memory");
}
// Arrive on `bar` of both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"((unsigned short)3), "r"(one)
      : "memory");
}
// A tile into this CTA's shared memory, its bytes counted on a barrier of either CTA (a cluster address).
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Arrive on a barrier of either CTA (see wait_for on the scope).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bytes that will not arrive, counted as if they had.
__device__ __forceinline__ void complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t t, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}

struct Tile {
  int m, n, split;
};
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, int t) {
  const uint32_t tiles_m = g.tiles_m, tiles_n = g.tiles_n;
  uint32_t split = 0, r = t;
  if (g.splits > 1) {
    split = r / (tiles_m * tiles_n);
    r -= split * tiles_m * tiles_n;
  }
  const uint32_t span = kGroup * tiles_n, group = r / span, at = r - group * span;
  const uint32_t first = group * kGroup, size = tiles_m - first < kGroup ? tiles_m - first : kGroup;
  const uint32_t n = size == kGroup ? at / kGroup : at / size;
  return {(int)(first + at - n * size), (int)n, (int)split};
}

// A warp's 32 x 32 sums, a row a lane, into its staging: rows of 32 float32, 16-byte piece j of row r at j ^ (r & 7).
__device__ __forceinline__ void stage_in(uint32_t chunk, int lane, const float* v) {
  __syncwarp();   // the last chunk has been read
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(chunk + lane * 128 + ((j ^ (lane & 7)) << 4)),
                 "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                 : "memory");
  __syncwarp();
}
// 32 bytes of a row, as one access.
struct Piece {
  uint32_t r[8];
};
__device__ __forceinline__ void ld_piece(Piece& x, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x.r[0]), "=r"(x.r[1]), "=r"(x.r[2]), "=r"(x.r[3]), "=r"(x.r[4]), "=r"(x.r[5]), "=r"(x.r[6]), "=r"(x.r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_piece(void* p, const Piece& x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x.r[0]), "r"(x.r[1]), "r"(x.r[2]),
               "r"(x.r[3]), "r"(x.r[4]), "r"(x.r[5]), "r"(x.r[6]), "r"(x.r[7])
               : "memory");
}
template <typename T, int COLS>
__device__ __forceinline__ Piece to_piece(const float* v) {
  Piece x;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.r[i] = pack2(v[2 * i], v[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.r[i] = __float_as_uint(v[i]);
  }
  return x;
}

__device__ __forceinline__ float4 ld_shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t at, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// 32 sums of a lane's row to memory, 32 bytes (whole sectors) an access.  n: their first column, the same in every lane;
// alive: the lane's row exists; bias, scale: their columns' values in shared memory.
template <typename T>
__device__ __forceinline__ void chunk_direct(const GemmArgs& g, float* v, float xs, long long m, long long n, bool alive, uint32_t bias,
                                             uint32_t scale) {
  constexpr int PIECES = (int)sizeof(T), COLS = 32 / PIECES;
  const Epilogue& e = g.out;
  Piece res[PIECES];
  if (e.residual) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
      if (alive && n + p * COLS < g.N) ld_piece(res[p], static_cast<const T*>(e.residual) + m * e.res_row + n + p * COLS);
  }
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const long long at = n + p * COLS;
    if (at >= g.N) break;
    float* u = v + p * COLS;
    if (e.x_scale) {
#pragma unroll
      for (int j = 0; j < COLS; ++j) u[j] *= xs;
    }
    if (e.w_scale) {
#pragma unroll
      for (int j = 0; j < COLS; j += 4) {
        const float4 s = ld_shared4(scale + (p * COLS + j) * 4);
        u[j] *= s.x; u[j + 1] *= s.y; u[j + 2] *= s.z; u[j + 3] *= s.w;
      }
    }
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < COLS; j += 4) {
        const float4 b = ld_shared4(bias + (p * COLS + j) * 4);
        u[j] += b.x; u[j + 1] += b.y; u[j + 2] += b.z; u[j + 3] += b.w;
      }
    }
    if (e.pre && alive) st_piece(static_cast<T*>(e.pre) + m * e.pre_row + at, to_piece<T, COLS>(u));
    if (e.act == kActSilu) {
#pragma unroll
      for (int j = 0; j < COLS; j += 2) unpair(activate2<sizeof(T) == 2>(pair(u[j], u[j + 1]), kActSilu), u[j], u[j + 1]);
    } else if (e.act == kActGelu) {
#pragma unroll
      for (int j = 0; j < COLS; j += 2) unpair(activate2<sizeof(T) == 2>(pair(u[j], u[j + 1]), kActGelu), u[j], u[j + 1]);
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 2) {
          u[2 * i] += lo_f(res[p].r[i]);
          u[2 * i + 1] += hi_f(res[p].r[i]);
        } else {
          u[i] += __uint_as_float(res[p].r[i]);
        }
      }
    }
    if (alive) st_piece(static_cast<T*>(e.y) + m * e.y_row + at, to_piece<T, COLS>(u));
  }
}

// The same through a warp's staging, for rows that do not start on 32-byte boundaries: a lane has one column and the
// warp a row at a time, so that what it reads and writes of the row is adjacent: 8000 x 4171 x 64 bfloat16 41 us (4176
// columns, directly: 22).
template <typename T>
__device__ __forceinline__ void chunk_staged(const GemmArgs& g, const float* v, uint32_t chunk, long long m0, long long n0, int lane) {
  constexpr int ROWS = 8;   // fetched together
  const Epilogue& e = g.out;
  stage_in(chunk, lane, v);
  const long long n = n0 + lane;
  if (n >= g.N) return;
  const int rows = g.M - m0 < 32 ? (int)(g.M - m0) : 32;
  const float scale = e.w_scale ? e.w_scale[n] : 1.f, bias = e.bias ? e.bias[n] : 0.f;
  const T* res = static_cast<const T*>(e.residual) + m0 * e.res_row + n;
  T* pre = static_cast<T*>(e.pre) + m0 * e.pre_row + n;
  T* y = static_cast<T*>(e.y) + m0 * e.y_row + n;
  // no branch within the eight rows but at the tile's last ones: their reads, sums and writes overlap
  auto eight = [&](int r0, auto all) {
    constexpr bool ALL = decltype(all)::value;
    float u[ROWS], add[ROWS] = {}, xs[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + i;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u[i]) : "r"(chunk + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4));
      xs[i] = 1.f;
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (ALL || r0 + i < rows) add[i] = to_f32<T>(res[(r0 + i) * e.res_row]);
    }
    if (e.x_scale) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (ALL || r0 + i < rows) xs[i] = e.x_scale[m0 + r0 + i];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) u[i] = fmaf(u[i] * xs[i], scale, bias);
    if (e.pre) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (ALL || r0 + i < rows) pre[(r0 + i) * e.pre_row] = from_f32<T>(u[i]);
    }
    if (e.act != kActNone) {
#pragma unroll
      for (int i = 0; i < ROWS; i += 2) unpair(activate2<sizeof(T) == 2>(pair(u[i], u[i + 1]), e.act), u[i], u[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (ALL || r0 + i < rows) y[(r0 + i) * e.y_row] = from_f32<T>(u[i] + add[i]);
  };
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    if (r0 + ROWS <= rows) eight(r0, std::true_type());
    else eight(r0, std::false_type());
  }
}

// Warps 4..11: a warp takes 32 rows (those of the tensor memory lanes that it can reach) and half the columns.
// PROMOTE: sums move to registers every g.part stages.
template <typename T, int BN, bool PROMOTE, bool BACK>
__device__ __forceinline__ void epilogue(const GemmPair& pair, uint32_t tmem, uint32_t chunk, uint64_t* acc_full,
                                         uint64_t* acc_empty, uint32_t rank, int warp, int lane, int first, int step,
                                         int n_tiles, volatile uint32_t* failed) {
  constexpr int CHUNKS = BN / 64;
  const int quad = warp & 3, half = (warp - 4) >> 2;
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  uint32_t buf = 0, phase = 0;
  auto next = [&]() {
    if (++buf == 2) {
      buf = 0;
      phase ^= 1;
    }
  };
  auto release = [&]() {
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive_at(mapa_shared(smem_u32(acc_empty + buf), 0));
  };
  for (int t = first; t < n_tiles; t += step) {
    const bool second = BACK && t >= pair.g[0].tiles;
    const GemmArgs& g = pair.g[second];
    const Tile at = tile_at(g, second ? t - pair.g[0].tiles : t);
    if (g.limit == 0) {   // the wait's self-test: the others find out with copies and products under way
      *failed = 1;
      return;
    }
    const long long m0 = (long long)at.m * 256 + rank * 128 + quad * 32, m = m0 + lane;
    const long long n0 = (long long)at.n * BN + half * (BN / 2);
    const bool alive = m < g.M;
    const float xs = g.out.x_scale && alive ? g.out.x_scale[m] : 1.f;
    // bias and weight scale of the warp's columns wait in its staging, which rows on 32-byte boundaries do not need
    if (g.direct && (g.out.bias || g.out.w_scale)) {
      const long long n = n0 + lane * 4;
      const bool mine = lane < BN / 8 && n < g.N;
      const float4 b = mine && g.out.bias ? *reinterpret_cast<const float4*>(g.out.bias + n) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 s = mine && g.out.w_scale ? *reinterpret_cast<const float4*>(g.out.w_scale + n) : make_float4(1.f, 1.f, 1.f, 1.f);
      __syncwarp();   // the last tile's have been read
      st_shared4(chunk + lane * 16, b);
      st_shared4(chunk + kChunk / 2 + lane * 16, s);
      __syncwarp();
    }
    auto out = [&](float* v, int c) {
      const long long n = n0 + c * 32;
      if (g.splits > 1) {   // rows of `partial` start on 32-byte boundaries
        float* p = g.partial + ((long long)at.split * g.M + m) * g.part_row + n;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (alive && n + 8 * i < g.N) st_piece(p + 8 * i, to_piece<float, 8>(v + 8 * i));
      } else if (g.direct) {
        chunk_direct<T>(g, v, xs, m, n, alive, chunk + c * 128, chunk + kChunk / 2 + c * 128);
      } else {
        chunk_staged<T>(g, v, chunk, m0, n, lane);
      }
    };
    if constexpr (PROMOTE) {
      float sums[CHUNKS][32] = {};
      const int k1 = k_begin(g, at.split + 1);
      for (int k = k_begin(g, at.split); k < k1; k = part_end(g, k, k1)) {
        if (!wait_warp(acc_full + buf, phase, g.limit, failed)) return;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          float v[32];
          tc::tmem_ld32(tmem + buf * BN + half * (BN / 2) + c * 32 + lanes, v);
          if (c == CHUNKS - 1) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) sums[c][j] += v[j];
        }
        next();
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) out(sums[c], c);
    } else {
      if (!wait_warp(acc_full + buf, phase, g.limit, failed)) return;
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < CHUNKS; ++c) {
        float v[32];
        tc::tmem_ld32(tmem + buf * BN + half * (BN / 2) + c * 32 + lanes, v);
        if (c == CHUNKS - 1) release();
        out(v, c);
      }
      next();
    }
  }
}

template <typename T, int BN, bool E4M3, bool PROMOTE, bool BACK>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmPair pair) {
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::o_bar);
  uint64_t *empty = full + C::stages, *acc_full = empty + C::stages, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile uint32_t* failed = slot + 1;
  volatile uint32_t* theirs = slot + 2;   // the other CTA's: failed, stages filled
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  uint32_t issued = 0;   // stages that the producer has filled
  const int n_tiles = pair.g[0].tiles + (BACK ? pair.g[1].tiles : 0), first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 16);
    }
    mbar_init(drain, 1);
    *failed = (base & 1023u) != 0;   // the swizzled tiles need it; report rather than run misaligned
    fence_mbar_init();
  }
  if (warp == 1) alloc_pair(smem_u32(slot), C::cols);
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  wait_for_first();   // copies, g
  all_started();      // the joining of parts

  // the block's registers, 168 a thread at launch: 128 x 40 + 256 x 232 = 384 x 168
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const uint32_t chunk = base + C::o_chunk + (warp - 4) * kChunk;
    epilogue<T, BN, PROMOTE, BACK>(pair, tmem, chunk, acc_full, acc_empty, rank, warp, lane, first, step, n_tiles, failed);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t rank_m = rank * 128, rank_n = rank * (BN / 2);
        uint32_t stage = 0, phase = 1;
        bool ok = !*failed;
        for (int t = first; ok && t < n_tiles; t += step) {
          const bool second = BACK && t >= pair.g[0].tiles;
          const GemmArgs& g = pair.g[second];
          const CUtensorMap *map_a = &maps.a[second], *map_b = &maps.b[second];
          const Tile at = tile_at(g, second ? t - pair.g[0].tiles : t);
          const int m0 = at.m * 256 + rank_m, n0 = at.n * BN + rank_n;
          const int k1 = k_begin(g, at.split + 1);
          int k = k_begin(g, at.split), pass = g.passes == 1 ? 0 : k / g.k_iters, it = k - pass * g.k_iters;
          for (; k < k1; ++k) {
            if (!(ok = wait_for(empty + stage, phase, g.limit, failed))) break;
            const uint32_t sa = base + stage * C::stage, sb = sa + C::a_bytes;
            const uint32_t bar = mapa_shared(smem_u32(full + stage), 0);
            if (rank == 0) mbar_arrive_expect_tx(full + stage, 2 * C::stage);
            const int ta = g.passes > 1 ? term_a(pass) : 0, tb = g.passes > 1 ? term_b(pass) : 0;
            const int at_k = it * (E4M3 ? 128 : 64);
            if (BACK && second) {
#pragma unroll
              for (int j = 0; j < 2; ++j) tma_pair(sa + j * 8192, map_a, m0 + 64 * j, at_k, ta, bar);
            } else {
              tma_pair(sa, map_a, at_k, m0, ta, bar);
            }
            if (BACK) {
#pragma unroll
              for (int j = 0; j < BN / 128; ++j) tma_pair(sb + j * 8192, map_b, n0 + 64 * j, at_k, tb, bar);
            } else {
              tma_pair(sb, map_b, at_k, n0, tb, bar);
            }
            ++issued;
            if (++stage == C::stages) {
              stage = 0;
              phase ^= 1;
            }
            if (++it == g.k_iters) {
              it = 0;
              ++pass;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        const uint32_t one = lane == 0;
        uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1;
        bool ok = !*failed;
        auto tile = [&](const GemmArgs& g, int t, auto a_mn, auto b_mn) {
          constexpr bool A = decltype(a_mn)::value, B = decltype(b_mn)::value;
          constexpr uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) | (A ? 1u << 15 : 0u) | (B ? 1u << 16 : 0u) |
                                     (uint32_t)(BN >> 3) << 17 | (256u >> 4) << 24;
          constexpr uint32_t step_a = A ? 2048 >> 4 : 32 >> 4, step_b = B ? 2048 >> 4 : 32 >> 4;
          const int split = g.splits == 1 ? 0 : t / (g.tiles_m * g.tiles_n), k1 = k_begin(g, split + 1);
          for (int k = k_begin(g, split); ok && k < k1;) {
            const int end = PROMOTE ? part_end(g, k, k1) : k1;
            if (!(ok = wait_for(acc_empty + buf, buf_phase, g.limit, failed))) return;
            tc::fence_after_sync();
            const uint32_t d = tmem + buf * BN;
            for (bool more = false; k < end; ++k, more = true) {
              if (!(ok = wait_for(full + stage, phase, g.limit, failed))) return;
              tc::fence_after_sync();
              const uint32_t sa = base + stage * C::stage;
              const uint64_t da = desc128(sa, 8192), db = desc128(sa + C::a_bytes, 8192);
#pragma unroll
              for (int i = 0; i < 4; ++i) mma_pair<E4M3>(d, da + i * step_a, db + i * step_b, idesc, more || i > 0, one);
              commit_pair(smem_u32(empty + stage), one);
              if (++stage == C::stages) {
                stage = 0;
                phase ^= 1;
              }
            }
            commit_pair(smem_u32(acc_full + buf), one);
            if (++buf == 2) {
              buf = 0;
              buf_phase ^= 1;
            }
          }
        };
        for (int t = first; ok && t < n_tiles; t += step) {
          if (!BACK) tile(pair.g[0], t, std::false_type(), std::false_type());
          else if (t < pair.g[0].tiles) tile(pair.g[0], t, std::false_type(), std::true_type());
          else tile(pair.g[1], t - pair.g[0].tiles, std::true_type(), std::true_type());
        }
        // whoever gave up: no product reads either CTA's memory behind this
        commit_pair(smem_u32(drain), one);
        mbar_wait_bounded(drain, 0);
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (rank == 1) mbar_wait_bounded(drain, 0);   // the leader signals nothing here behind this
    const uint32_t to = mapa_shared(smem_u32(slot + 2), rank ^ 1);
    st_cluster_s32(to, (int)*failed);
    st_cluster_s32(to + 4, (int)issued);
  }
  __syncwarp();
  cluster_sync_all();   // neither CTA leaves while the other can still signal it
  if (*failed | theirs[0]) {   // the same in both CTAs
    if (threadIdx.x == 0 && rank == 0) {
      // Both CTAs' copies complete on this one's barriers, where this one expects those of both: what only one of them
      // has asked for is counted here, then all of it has to land.  (They are `stages` apart at most.)
      const uint32_t other = theirs[1];
#pragma unroll 1
      for (uint32_t i = other; i < issued; ++i) complete_tx(full + i % C::stages, C::stage);
#pragma unroll 1
      for (uint32_t i = issued; i < other; ++i) mbar_arrive_expect_tx(full + i % C::stages, C::stage);
      drain_ring(full, C::stages, issued > other ? issued : other);
    }
    __syncwarp();
    cluster_sync_all();
  }
  tc::fence_after_sync();
  if (warp == 1) dealloc_pair(tmem, C::cols);
  if (threadIdx.x == 0 && *failed) atomicOr(&pair.status->flags, kStatusTimeout);
}

// ---------------------------------------------------------------------------------------------
// parts of a split Kd, added in their order, and the epilogue; without parts the sum is 0

template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ GemmPair pair) {
  const GemmArgs& g = pair.g[blockIdx.y];
  wait_for_first();
  if (g.splits == 1) return;
  const long long across = (g.N + 3) / 4, all = g.M * across;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const long long m = i / across, n = (i - m * across) * 4;
    const int left = g.N - n < 4 ? (int)(g.N - n) : 4;
    float v[4] = {};
    Vec<T, 4> res;
    if (g.out.residual) res = load4<T>(static_cast<const T*>(g.out.residual) + m * g.out.res_row + n, g.res_vec, left);
    const float* p = g.partial + m * g.part_row + n;
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const Vec<float, 4> x = ld_vec<float, 4>(p + s * g.M * g.part_row);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += x.v[j];
    }
    out4<T>(g, v, columns_of(g.out, n, left), res, m, n, left);
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether CUDA cores take the product (vla_rowvec.cu), eight rows of x at a time: with one or two rows (e4m3), four
// (bfloat16) or sixteen (float32) the weights' way from memory bounds them; with more, their arithmetic does, and they win only
// where the tensor cores' fixed cost is the larger part.  Measured (us, launches by themselves, CUDA cores against vla_gemm_tokens.cu): bfloat16
// N 8192, K 8192: 24.6 against 32 (1 row), 33.6 against 32 (4), 65 against 33 (8); N 520, K 264, 16 rows: 5.0 against 5.5,
// 4.8 against 9.7 with rows that a copy has to align; float32 N 8192, K 8192: 208 against 216 (16), 366 against 218 (32);
// e4m3: 17.4 against 18.8 (1), 22.0 against 18.9 (2), 31.7 against 18.9 (4).
bool few_rows(const ProductArgs& p, int mat, bool copies) {
  const long long most = mat == kMatF32 ? 16 : mat == kMatBf16 ? 4 : 2, eights = (p.M + 7) / 8;
  return p.M <= most || (p.M <= 128 && p.N * p.Kd <= (1LL << (mat == kMatF32 || copies ? 23 : 21)) / eights);
}

// Whether w's rows are the long side of the tensor cores' product (vla_gemm_tokens.cu): up to 128 rows of x, and up to 512
// where the weights are few (bfloat16, us against tiles of 256 rows: N 8192, K 8192: 37.6 against 43.2 with 128 rows,
// 46.0 against 45.5 with 256; N 2048, K 4096: 14.2 against 16.9, and 17.9 against 20.7 with 512).
bool tokens(const ProductArgs& p) { return p.M <= 128 || (p.M <= 512 && p.N * p.Kd <= 1LL << 23); }

struct Plan {
  Operand a[2], b[2];
  bool few;             // rows of x: CUDA cores
  TokensPlan tokens;    // rows 0: tiles of 256 rows
  int bn, passes, splits[2], tiles_m[2], tiles_n[2], k_iters[2];   // splits 0: no terms
  Copies copies;
  size_t at[4], parts_at[2], ws;   // where in the workspace copies and parts lie
};

// The copy of an operand, one for all that are the same.  (Without addresses, in a query, every operand has its own.)
int copy_of(const Plan& q, const Operand& o) {
  for (int i = 0; i < q.copies.count; ++i) {
    const Operand& c = q.copies.o[i];
    if (o.p && c.p == o.p && c.rows == o.rows && c.cols == o.cols && c.row == o.row) return i;
  }
  return -1;
}

Plan plan_of(const ProductArgs* p, int count, int mat) {
  Plan q{};
  const int size = mat == kMatF32 ? 4 : mat == kMatBf16 ? 2 : 1, per = mat == kMatE4m3 ? 128 : 64;
  q.passes = mat == kMatF32 ? kPasses : 1;
  for (int i = 0; i < count; ++i) {
    q.a[i] = operand(p[i].a, p[i].M, p[i].Kd, p[i].a_row, p[i].a_mn, size);
    q.b[i] = operand(p[i].b, p[i].N, p[i].Kd, p[i].b_row, p[i].b_mn, size);
    q.k_iters[i] = (int)((p[i].Kd + per - 1) / per);
    q.tiles_m[i] = (int)((p[i].M + 255) / 256);
  }
  auto copy = [&](const Operand& o) {
    if (!o.pack || copy_of(q, o) >= 0) return;
    q.at[q.copies.count] = q.ws;
    q.copies.o[q.copies.count++] = o;
    q.ws += up256(o.bytes);
  };
  const bool rows_of_k = count == 1 && !p[0].a_mn && !p[0].b_mn && p[0].Kd > 0;
  if (rows_of_k && few_rows(p[0], mat, q.a[0].pack || q.b[0].pack)) {
    q.few = true;
    return q;
  }
  for (int i = 0; i < count; ++i) {
    if (p[i].Kd == 0) continue;
    copy(q.a[i]);
    copy(q.b[i]);
  }
  if (rows_of_k && tokens(p[0])) {
    q.tokens = tokens_plan(p[0].M, p[0].N, p[0].N * p[0].Kd, q.k_iters[0] * q.passes, p[0].sm_count);
    if (q.ws) q.ws += 32;   // what the workspace's start is moved by at most
    return q;
  }
  // Cost of a choice in stages: what the cluster with the most has to do, units of a tile's stages or a share of them, each with
  // about 3 of latency at its ends; the parts' way through memory.  Each product's Kd is cut on its own, as long as its units are
  // two waves at most: of a gradient, one can have a few tiles with a long Kd and the other many short ones (float32, M 20781,
  // N 303, K 1232: 874 us with dw's 10 tiles whole).  A stage of a tile half as wide takes nearly as long (shared memory
  // bounds it).
  const int clusters = p[0].sm_count / 2 > 0 ? p[0].sm_count / 2 : 1;
  int longest = 1;
  for (int i = 0; i < count; ++i) longest = q.k_iters[i] * q.passes > longest ? q.k_iters[i] * q.passes : longest;
  double best = 1e300;
  for (int bn = 256; bn >= 128; bn /= 2) {
    const double stage = bn == 256 ? 1.0 : 0.9;
    int last[2] = {-1, -1};
    for (int shares = 1; shares == 1 || (shares <= 32 && longest >= 4 * shares); ++shares) {
      const int unit = (longest + shares - 1) / shares;   // stages at most
      long long units[2] = {}, all_units = 0;
      double parts = 0.0, length[2] = {};
      int splits[2] = {};
      for (int i = 0; i < count; ++i) {
        const int all = q.k_iters[i] * q.passes;
        const long long tiles = (long long)q.tiles_m[i] * ((p[i].N + bn - 1) / bn), most = 2 * clusters / tiles;
        splits[i] = p[i].Kd == 0 ? 0 : (all + unit - 1) / unit;
        if (splits[i] > most) splits[i] = most > 1 ? (int)most : splits[i] > 0;
        units[i] = tiles * splits[i];
        all_units += units[i];
        if (splits[i] > 0) length[i] = (double)all / splits[i] * stage + 3.0;
        if (splits[i] > 1) parts += (double)splits[i] * p[i].M * p[i].N;
      }
      if (splits[0] == last[0] && splits[1] == last[1]) continue;
      last[0] = splits[0];
      last[1] = splits[1];
      // units are dealt out in turn: a cluster's number of the first product's, and of both, changes where a wave of either ends
      double cost = 0.0;
      const long long ends[3] = {0, units[0] % clusters, all_units % clusters};
      for (int e = 0; e < (count == 1 ? 1 : 3); ++e) {
        const long long c = ends[e], first = c < units[0] ? (units[0] - c + clusters - 1) / clusters : 0;
        const long long both = c < all_units ? (all_units - c + clusters - 1) / clusters : 0;
        const double mine = (double)first * length[0] + (double)(both - first) * length[1];
        if (mine > cost) cost = mine;
      }
      // a launch, a part's read after the other, their bytes
      if (parts > 0.0) cost += 8.0 + 0.5 * (splits[0] > splits[1] ? splits[0] : splits[1]) + parts * 8.0 / 1.2e6;
      if (cost >= best) continue;
      best = cost;
      q.bn = bn;
      for (int i = 0; i < count; ++i) {
        q.splits[i] = splits[i];
        q.tiles_n[i] = (int)((p[i].N + bn - 1) / bn);
      }
    }
  }
  for (int i = 0; i < count; ++i) {
    if (q.splits[i] <= 1) continue;
    q.ws = up256(q.ws);
    q.parts_at[i] = q.ws;
    q.ws += (size_t)q.splits[i] * p[i].M * ((p[i].N + 7) / 8 * 8) * 4;
  }
  if (q.ws) q.ws += 32;   // parts lie on 32-byte boundaries, the workspace on a 16-byte one
  return q;
}

// follows: the launch before it on the stream is of the same call (see launch_after); others are waited for whole
template <typename T, int BN, bool E4M3, bool PROMOTE, bool BACK>
cudaError_t launch(const Maps& maps, const GemmPair& pair, bool follows, cudaStream_t s) {
  auto kern = gemm_kernel<T, BN, E4M3, PROMOTE, BACK>;
  constexpr int bytes = (int)Cfg<BN>::bytes;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(2);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = bytes;
  c.stream = s;
  // clusters that fit at once, asked for once a kernel and device (the first 64)
  static std::atomic<int> known[64];
  int clusters = device < 64 ? known[device].load(std::memory_order_relaxed) : 0;
  if (clusters == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    c.attrs = &attr;
    c.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &c);
    if (e != cudaSuccess) return e;
    if (clusters < 1) clusters = 1;
    if (device < 64) known[device].store(clusters, std::memory_order_relaxed);
  }
  const long long tiles = (long long)pair.g[0].tiles + pair.g[1].tiles;
  c.gridDim = dim3((unsigned int)(2 * (tiles < clusters ? tiles : clusters)));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = follows ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, maps, pair);
}

}  // namespace

size_t products_ws(const ProductArgs* p, int count, int mat) { return plan_of(p, count, mat).ws; }

cudaError_t launch_products(const ProductArgs* p, int count, int mat, cudaStream_t s) {
  Plan q = plan_of(p, count, mat);
  if (q.few) return launch_few_rows(p[0], mat, s);
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p[0].ws) + 31) & ~(uintptr_t)31);
  cudaError_t e = cudaSuccess;
  if (q.copies.count) {
    for (int i = 0; i < q.copies.count; ++i) q.copies.to[i] = ws + q.at[i];
    e = pack(q.copies, p[0].sm_count, s);
    if (e != cudaSuccess) return e;
  }
  auto place = [&](const Operand& o) -> const void* { return o.pack ? ws + q.at[copy_of(q, o)] : o.p; };
  GemmPair pair{};
  Maps maps;
  bool join = false, whole = true;   // whole: no share of Kd is longer than kWhole stages
  long long pieces = 0;
  const int per = mat == kMatE4m3 ? 128 : 64;
  const bool back = p[0].b_mn;
  pair.status = p[0].status;
  pair.g[0].splits = pair.g[1].splits = 1;   // nothing to join
  for (int i = 0; i < count; ++i) {
    const int at = back && p[i].a_mn;   // a gradient's dw is the second
    GemmArgs& g = pair.g[at];
    g = args_of(p[i]);
    g.k_iters = q.k_iters[i]; g.passes = q.passes;
    g.limit = p[i].wait_limit ? p[i].wait_limit + 4000ull * (unsigned long long)q.k_iters[i] * q.passes : 0;
    if (q.tokens.rows) return launch_tokens(q.tokens, g, q.a[0], q.b[0], place(q.a[0]), place(q.b[0]), s);
    g.tiles_m = q.tiles_m[i]; g.tiles_n = q.tiles_n[i]; g.splits = q.splits[i];
    g.part = p[i].out.y_bf16 ? kLongPart : kPart;
    if (g.splits > 0 && (q.k_iters[i] * q.passes + g.splits - 1) / g.splits > kWhole) whole = false;
    const long long tiles = (long long)g.tiles_m * g.tiles_n * g.splits;
    if (tiles > 0x1fffffff) return cudaErrorInvalidConfiguration;
    g.tiles = (int)tiles;
    g.partial = reinterpret_cast<float*>(ws + q.parts_at[i]);
    if (g.splits != 1) {
      join = true;
      if (g.M * ((g.N + 3) / 4) > pieces) pieces = g.M * ((g.N + 3) / 4);
    }
    if (g.splits > 0 &&
        (!encode(&maps.a[at], q.a[i], place(q.a[i]), p[i].a_mn ? 64 : per, p[i].a_mn ? per : 128) ||
         !encode(&maps.b[at], q.b[i], place(q.b[i]), back ? 64 : per, back ? per : q.bn / 2)))
      return cudaErrorInvalidValue;
  }
  const bool terms = pair.g[0].tiles + pair.g[1].tiles > 0;
  if (terms) {
    const bool wide = q.bn == 256, y16 = p[0].out.y_bf16, follows = p[0].follows || q.copies.count > 0;
    auto run = [&](auto y, auto bn, auto promote) -> cudaError_t {
      using T = decltype(y);
      constexpr int BN = decltype(bn)::value;
      constexpr bool P = decltype(promote)::value;
      if (back) return launch<T, BN, false, P, true>(maps, pair, follows, s);
      return mat == kMatE4m3 ? launch<T, BN, true, P, false>(maps, pair, follows, s) : launch<T, BN, false, P, false>(maps, pair, follows, s);
    };
    auto of = [&](auto y, auto promote) { return wide ? run(y, std::integral_constant<int, 256>(), promote) : run(y, std::integral_constant<int, 128>(), promote); };
    if (!y16) e = of(float(), std::true_type());
    else e = whole ? of(__nv_bfloat16(), std::false_type()) : of(__nv_bfloat16(), std::true_type());
    if (e != cudaSuccess) return e;
  }
  if (!join) return e;
  const long long want = (pieces + 255) / 256, most = 16LL * p[0].sm_count;
  const dim3 grid((unsigned int)(want < most ? want : most), back ? 2u : 1u);
  return p[0].out.y_bf16 ? launch_after(terms, join_kernel<__nv_bfloat16>, grid, 256, s, pair)
                         : launch_after(terms, join_kernel<float>, grid, 256, s, pair);
}

}  // namespace vla
