// Selective state space scan over prompts on the tensor cores: bfloat16 input and output, chunks of
// L = 128 tokens, one CTA for 64 columns p of a head (a "slice") and a run of chunks.
//
// With l_t = A s_t (the log decay), c_t = l_1 + .. + l_t within a chunk and h the state before it:
//   S = C B^T                                              (128 x 128, K = N)
//   M_ts = S_ts exp(c_t - c_s) s_s for s <= t, else 0
//   Y = exp(c_t) (C h^T)_t + M X + D X                     (128 x 64, K = N; K = 128)
//   h' = exp(c_L) h + [B^T X~]^T,  X~_s = s_s exp(c_L - c_s) x_s     (N x 64, K = 128)
// All four products are tcgen05.mma of bfloat16 with float32 accumulators in tensor memory.
//
// Precision.  The state is float32 and lives in the registers of its threads for the whole run.
// B and x are exact in bfloat16; X~ is carried as three bfloat16 terms (24 bits), so the state is
// as exact as a float32 scan's.  M and the copy of h that multiplies C are each rounded to bfloat16
// once (2^-9 relative, as the output itself is).  The suffix sums c_L - c_s are summed from
// the end, so that what is left of the last tokens does not suffer from a large c_L.
//
// exp(c_t - c_s) takes no exponential a pair: with e_j the sum at the end of block j of 32 tokens s,
// exp(c_t - e_j) exp(e_j - c_s) is one factor a row and one a column, both at most 1, for the rows
// behind the block.  In a diagonal block e_j is the sum before the block; the column's factor is
// then at least 1, so this holds while the block's sums stay below 2^100, and beyond that (nothing
// is left of a token a few tokens later) the exponentials are taken pair by pair.
//
// Roles.  Eight warps compute (thread = a row of the chunk, or a state n, and 32 of 64 columns);
// the ninth issues the loads and the products, and the tenth forms the decays, up to two chunks
// ahead.  They meet on mbarriers.  In the order of a chunk:
//   ninth: S, C h^T | computing: X~ | ninth: B^T X~ | computing: M, scaling of C h^T | ninth: M X,
//   loads of the next B and C | computing: state, Y | ninth: Y's store, load of the next X.
//
// Operands.  B, C [128 tokens][N] and X [128][64] arrive by TMA as 128-byte-swizzled tiles of 64
// columns; the same B tile is the K-major operand of S and the transposed (MN-major) one of the
// state's product.  M replaces S in tensor memory as the A operand of M X.  Shared memory is reused
// within a chunk (X~ overwrites C and the bfloat16 state once S and C h^T are done; Y overwrites X), which
// keeps a CTA below half an SM's: two CTAs an SM hide each other's latencies.
//
// Few slices: the sequence is cut into segments, one CTA each.  A first launch forms what every
// segment but a sequence's last adds to the state (B^T X~ alone), the second starts each segment from
// those, joined in a fixed order.
#include <cuda.h>   // CUtensorMap and the encode entry point's types (resolved at run time)

#include <algorithm>

#include "vla_layer.cuh"
#include "vla_ssm_prompt.cuh"
#include "vla_tc.cuh"

namespace vla {
namespace {

constexpr int kL = 128;            // tokens a chunk
constexpr int kCompute = 256;      // threads of the computing warps
constexpr int kThreads = 320;
constexpr uint32_t kTile = 16384;  // bytes of a [128][64] bfloat16 tile
constexpr uint32_t kCols = 256;    // tensor memory columns a CTA: S (M) | Y | the state's product U
constexpr uint32_t kColS = 0, kColY = 128, kColU = 192;
constexpr int kVec = 5 * kL + 16;  // floats of a chunk's decays (two buffers)
constexpr int kBars = 13;

// Shared memory: B | C | X | state (bfloat16, [n][64 p]) | more X~ | vectors | barriers
template <int NN>
struct Cfg {
  static constexpr uint32_t NT = NN / 64;
  static constexpr uint32_t oB = 0, oC = NT * kTile, oX = 2 * NT * kTile, oH = oX + kTile;
  static constexpr uint32_t HB = NN * 128;
  static constexpr uint32_t oMore = oH + HB;
  static constexpr uint32_t term0 = oC;
  static constexpr uint32_t term1 = NN == 128 ? oC + kTile : oMore;
  static constexpr uint32_t term2 = NN == 128 ? oH : oMore + kTile;
  static constexpr uint32_t oVec = NN == 128 ? oMore : oMore + 2 * kTile;
  static constexpr uint32_t bytes = oVec + 4 * 2 * kVec + 8 * kBars + 16;
};

// Matrix descriptor of a 128-byte-swizzled operand: `lbo` bytes between blocks of 64 in the
// contiguous dimension of a transposed operand, 1024 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;   // instruction descriptor: MN-major operands

// D (+)= X Y with X in tensor memory (bfloat16, two K elements a column)
__device__ __forceinline__ void mma_f16_tx(uint32_t d_tmem, uint32_t x_tmem, uint64_t ydesc, uint32_t idesc,
                                           bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(x_tmem), "l"(ydesc), "r"(idesc), "r"(acc)
      : "memory");
}

// 16 32-bit columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// the tile of a later load, from memory into L2
__device__ __forceinline__ void prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void store_4d(const CUtensorMap* map, int x, int y, int z, int w, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n\t"
               "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_read_done() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct PromptArgs {
  const __nv_bfloat16* dt;
  const float* A;
  const float* D;
  const __nv_bfloat16* z;
  const float* dt_bias;
  float* state;
  __nv_bfloat16* y;
  float* ws;
  Seqs seqs;
  int H, P, G, N, pslices;
  int nseg, seg_chunks;
  long long dt_seq, dt_tok, z_seq, z_tok, y_seq, y_tok;
  bool softplus, z_vec;
  DevStatus* status;
};

// Workspace of one (sequence, slice): nseg states of 64 x NN floats (the place of the last segment
// holds a copy of the state before the sequence), then their decays.
__host__ __device__ constexpr long long ws_floats(int nseg, int NN) { return (long long)nseg * 64 * NN + (nseg + 63) / 64 * 64; }

// FULL: the outputs and the final state; else what the segment adds to the state.
template <int NN, bool FULL>
__global__ void __launch_bounds__(kThreads, 2)
    ssm_prompt_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_B,
                      const __grid_constant__ CUtensorMap map_C, const __grid_constant__ CUtensorMap map_y,
                      const __grid_constant__ PromptArgs a) {
  using Cf = Cfg<NN>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = a.H * a.pslices;
  const int slice = (int)(blockIdx.x % slices);
  const long long rest = blockIdx.x / slices;
  const int seg = (int)(rest % a.nseg);
  const long long seq = rest / a.nseg;
  const int head = slice / a.pslices, p0 = (slice - head * a.pslices) * 64, group = head / (a.H / a.G);

  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, seq, &bad);
  if (bad && tid == 0 && FULL) atomicOr(&a.status->flags, bad);
  const long long chunks = (q.len + kL - 1) / kL;
  const long long c_begin = (long long)seg * a.seg_chunks;
  const long long c_end = c_begin + a.seg_chunks < chunks ? c_begin + a.seg_chunks : chunks;
  const bool last = c_end == chunks;
  if (!q.run || c_begin >= chunks || (!FULL && last)) return;
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {   // the swizzled tiles need it; report rather than run misaligned
    if (tid == 0) atomicOr(&a.status->flags, kStatusTimeout);
    return;
  }

  // decays of chunk c at vec + (c & 1) kVec: cum [128] log2 decay from the chunk's start up to a token;
  // wcol [128] s exp(e_j - c), j the token's block; wdg [128] the same with the sum before the
  // block; wx [128] s exp(c_L - c); step [128] s; then [4] sums before the blocks, [4] to their ends,
  // [8] the total, [12..16) whether wdg holds
  float* vec = reinterpret_cast<float*>(smem + Cf::oVec);
  uint64_t* bar = reinterpret_cast<uint64_t*>(vec + 2 * kVec);
  uint64_t *b_bc = bar, *b_x = bar + 1, *b_dec = bar + 2;           // B and C, X loaded; decays written [2]
  uint64_t *b_s = bar + 4, *b_u = bar + 5, *b_y = bar + 6;          // products done: S and C h^T, U, M X
  uint64_t *b_xt = bar + 7, *b_m = bar + 8, *b_free = bar + 9;      // X~, M written; decays read [2]
  uint64_t *b_next = bar + 11, *b_out = bar + 12;                   // tensor memory and h free; Y staged
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + kBars);
  volatile int* fail = reinterpret_cast<volatile int*>(tslot + 1);

  const bool packed = a.seqs.offsets != nullptr;
  const int row0 = packed ? (int)q.start : 0, batch = packed ? 0 : (int)seq;   // tensor map coordinates
  const __nv_bfloat16* dt = a.dt + (packed ? q.start * a.dt_tok : seq * a.dt_seq) + head;
  const float A2 = a.A[head] * 1.44269504088896341f, bias = a.dt_bias ? a.dt_bias[head] : 0.f;
  const float Dh = a.D ? a.D[head] : 0.f;

  if (tid == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(bar + i, 1);
    for (int i = 7; i < kBars; ++i) mbar_init(bar + i, kCompute / 32);
    *fail = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(tslot, kCols);

  // this thread's part of the state: n = row, 32 columns p from 32 half
  const int row = tid & (kL - 1), half = (tid >> 7) & 1;
  const int n = row;
  const bool n_ok = n < a.N;
  float h[32];
  if (tid < kCompute) {
    const int pc = a.P - p0 - 32 * half;   // columns of this thread that exist
    const bool from_ws = a.nseg > 1 && FULL && chunks > a.seg_chunks;
    float* wsq = from_ws || !FULL ? a.ws + (seq * slices + slice) * ws_floats(a.nseg, NN) : nullptr;
    const float* src = nullptr;
    long long pitch = 0;
    if (from_ws && seg == 0) { src = wsq + ((long long)(a.nseg - 1) * 64 + 32 * half) * NN; pitch = NN; }
    else if (!from_ws && a.state && seg == 0) { src = a.state + ((q.slot * a.H + head) * a.P + p0 + 32 * half) * a.N; pitch = a.N; }
    const bool mine = from_ws ? n < NN : n_ok;
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = src && mine && (from_ws || i < pc) ? src[i * pitch + n] : 0.f;
    if (!FULL && seg == 0 && n < NN) {   // the copy that the second launch starts from
      float* keep = wsq + ((long long)(a.nseg - 1) * 64 + 32 * half) * NN;
#pragma unroll
      for (int i = 0; i < 32; ++i) keep[i * NN + n] = h[i];
    }
    if (from_ws) {
      const float* dec = wsq + (long long)a.nseg * 64 * NN;
      for (int j = 0; j < seg; ++j) {
        const float d = j == 0 ? 0.f : dec[j];   // segment 0's result holds the state before the sequence
        const float* e = wsq + ((long long)j * 64 + 32 * half) * NN;
        if (n < NN) {
#pragma unroll
          for (int i = 0; i < 32; ++i) h[i] = fmaf(d, j == 0 ? 0.f : h[i], e[i * NN + n]);
        }
      }
    }
  }
  // the bfloat16 copy of the state, [n][64 p]: this thread's 64 bytes of row n
  auto put_state = [&]() {
    if (n < NN) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = make_uint4(pack2(h[8 * i], h[8 * i + 1]), pack2(h[8 * i + 2], h[8 * i + 3]),
                                   pack2(h[8 * i + 4], h[8 * i + 5]), pack2(h[8 * i + 6], h[8 * i + 7]));
        *reinterpret_cast<uint4*>(smem + Cf::oH + n * 128 + (((4 * half + i) ^ (n & 7)) << 4)) = v;
      }
    }
  };
  if (FULL && tid < kCompute) put_state();
  fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  constexpr uint32_t kIdS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t kId64 = (1u << 4) | (1u << 7) | (1u << 10) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
  // Bounded wait of a whole warp; gives up early when another one has.  The timer is read once in
  // many polls: it takes longer than a poll, and a wait ends when the poll after it is made.
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    bool ok = false;
    unsigned long long t_start = 0;
    while (true) {
#pragma unroll 1
      for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(b, parity);
      if (ok || *fail) break;
      const unsigned long long now = globaltimer_ns();
      if (t_start == 0) t_start = now;
      if (now - t_start > kWaitLimitNs) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *fail = 1;
    return ok;
  };
  // One arrival a warp, after everything its lanes have written to shared or tensor memory.
  auto arrive = [&](uint64_t* b) {
    fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
  };

  if (warp == kCompute / 32) {
    // ------------------------------------------------ loads, products, decays
    const bool one = lane == 0;
    auto load_bc = [&](long long c) {
      const int t = row0 + (int)(c * kL);
      mbar_arrive_expect_tx(b_bc, (FULL ? 2 : 1) * Cf::NT * kTile);
      for (uint32_t i = 0; i < Cf::NT; ++i) {
        load_4d(sbase + Cf::oB + i * kTile, &map_B, 64 * (int)i, group, t, batch, b_bc);
        if (FULL) load_4d(sbase + Cf::oC + i * kTile, &map_C, 64 * (int)i, group, t, batch, b_bc);
      }
    };
    auto load_x = [&](long long c) {
      mbar_arrive_expect_tx(b_x, kTile);
      load_4d(sbase + Cf::oX, &map_x, p0, head, row0 + (int)(c * kL), batch, b_x);
    };
    // a chunk's tiles are asked for when their places are free, which is late: their rows are fetched
    // into L2 two chunks ahead
    auto prefetch = [&](long long c) {
      const int t = row0 + (int)(c * kL);
      prefetch_4d(&map_x, p0, head, t, batch);
      for (uint32_t i = 0; i < Cf::NT; ++i) {
        prefetch_4d(&map_B, 64 * (int)i, group, t, batch);
        if (FULL) prefetch_4d(&map_C, 64 * (int)i, group, t, batch);
      }
    };
    if (one) {
      load_bc(c_begin);
      load_x(c_begin);
      if (c_begin + 1 < c_end) prefetch(c_begin + 1);
    }
    uint32_t ph = 0, bc_ph = 0, x_ph = 0;   // phases of the loads in flight
    bool bc_pending = true, x_pending = true;
    for (long long c = c_begin; c < c_end; ++c, ph ^= 1u) {
      const bool more = c + 1 < c_end;
      if (c > c_begin && !wait(b_next, ph ^ 1u)) break;
      if (!wait(b_bc, ph)) break;
      bc_pending = false;
      tc::fence_after_sync();
      if (FULL && one) {
#pragma unroll
        for (int k = 0; k < NN / 16; ++k) {
          const uint32_t at = (uint32_t)(k >> 2) * kTile + (uint32_t)(k & 3) * 32;
          tc::mma_f16(tmem + kColS, desc128(sbase + Cf::oC + at, 16), desc128(sbase + Cf::oB + at, 16), kIdS, k > 0);
        }
#pragma unroll
        for (int k = 0; k < NN / 16; ++k) {
          const uint32_t at = (uint32_t)(k >> 2) * kTile + (uint32_t)(k & 3) * 32;
          tc::mma_f16(tmem + kColY, desc128(sbase + Cf::oC + at, 16), desc128(sbase + Cf::oH + 2048u * k, 16),
                      kId64 | kTransB, k > 0);
        }
        tc::mma_commit(b_s);
      }
      __syncwarp();
      if (one && c + 2 < c_end) prefetch(c + 2);
      if (!wait(b_xt, ph)) break;
      x_pending = false;   // the computing warps have seen X
      tc::fence_after_sync();
      if (one) {
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const uint32_t term = t == 0 ? Cf::term2 : t == 1 ? Cf::term1 : Cf::term0;   // small terms first
#pragma unroll
          for (int k = 0; k < kL / 16; ++k)
            tc::mma_f16(tmem + kColU, desc128(sbase + Cf::oB + 2048u * k, kTile),
                        desc128(sbase + term + 2048u * k, 16), kId64 | kTransA | kTransB, t > 0 || k > 0);
        }
        tc::mma_commit(b_u);
      }
      __syncwarp();
      if (FULL) {
        if (!wait(b_m, ph)) break;
        tc::fence_after_sync();
        if (one) {
#pragma unroll
          for (int k = 0; k < kL / 16; ++k)
            mma_f16_tx(tmem + kColY, tmem + kColS + 64 * (k >> 2) + 8 * (k & 3), desc128(sbase + Cf::oX + 2048u * k, 16),
                       kId64 | kTransB, true);
          tc::mma_commit(b_y);
        }
        __syncwarp();
      }
      if (more) {
        if (!wait(b_u, ph)) break;
        if (one) {
          load_bc(c + 1);
          if (!FULL) load_x(c + 1);
        }
        bc_pending = true;
        bc_ph = ph ^ 1u;
        if (!FULL) x_pending = true, x_ph = ph ^ 1u;
        __syncwarp();
      }
      if (FULL) {
        if (!wait(b_out, ph)) break;
        const bool tail = packed && q.len - c * kL < kL;
        if (one) {
          if (!tail) store_4d(&map_y, p0, head, row0 + (int)(c * kL), batch, sbase + Cf::oX);
          if (more) {
            store_read_done();
            load_x(c + 1);
          }
        }
        if (more) x_pending = true, x_ph = ph ^ 1u;
        __syncwarp();
      }
    }
    // nothing lands after the CTA has gone
    if (*fail) {
      if (bc_pending) mbar_wait_bounded(b_bc, bc_ph);
      if (x_pending) mbar_wait_bounded(b_x, x_ph);
    }
    if (FULL && one) store_done();
  } else if (warp == kCompute / 32 + 1) {
    // ------------------------------------------------ decays, up to two chunks ahead
    float raw[4];   // dt of the chunk whose decays come next: tokens lane, 32 + lane, ..
    auto load_dt = [&](long long c) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long t = c * kL + 32 * j + lane;
        raw[j] = t < q.len ? __bfloat162float(dt[t * a.dt_tok]) : 0.f;
      }
    };
    auto decays = [&](long long c) {
      float* v = vec + (c & 1) * kVec;
      float s[4], inc[4], ex[4], end[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = c * kL + 32 * j + lane < q.len;
        s[j] = in ? time_step(raw[j], bias, a.softplus) : 0.f;
        inc[j] = in ? A2 * s[j] : 0.f;
        ex[j] = inc[j];
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = __shfl_up_sync(0xffffffffu, inc[j], o), d = __shfl_down_sync(0xffffffffu, ex[j], o);
          if (lane >= o) inc[j] += u;
          if (lane + o < 32) ex[j] += d;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        end[j] = __shfl_sync(0xffffffffu, inc[j], 31);
        ex[j] = __shfl_down_sync(0xffffffffu, ex[j], 1);
        if (lane == 31) ex[j] = 0.f;
      }
      float before = 0.f, after[4];
      after[3] = 0.f;
#pragma unroll
      for (int j = 2; j >= 0; --j) after[j] = after[j + 1] + end[j + 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 32 * j + lane;
        v[t] = before + inc[j];
        v[kL + t] = s[j] * ex2(ex[j]);
        v[2 * kL + t] = s[j] * ex2(-inc[j]);
        v[3 * kL + t] = s[j] * ex2(ex[j] + after[j]);
        v[4 * kL + t] = s[j];
        const bool small = __all_sync(0xffffffffu, fabsf(inc[j]) < 100.f);
        if (lane == 0) {
          v[5 * kL + j] = before;
          v[5 * kL + 4 + j] = before + end[j];
          v[5 * kL + 12 + j] = small ? 1.f : 0.f;
        }
        before += end[j];
      }
      if (lane == 0) v[5 * kL + 8] = before;
    };
    load_dt(c_begin);
    for (long long c = c_begin; c < c_end; ++c) {
      const uint32_t use = (uint32_t)((c - c_begin) >> 1), buf = (uint32_t)(c & 1);
      if (use > 0 && !wait(b_free + buf, (use - 1) & 1u)) break;
      decays(c);
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b_dec + buf)) : "memory");
      if (c + 1 < c_end) load_dt(c + 1);
    }
  } else {
    // ------------------------------------------------ arithmetic
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's lanes
    const int qd = warp & 3;                                            // its block of rows
    const uint32_t rsw = (uint32_t)(row & 7);
    const uint64_t D2 = pair(Dh, Dh);
    float log_total = 0.f;
    uint32_t ph = 0;
    for (long long c = c_begin; c < c_end; ++c, ph ^= 1u) {
      const long long t0 = c * kL;
      const bool tail = packed && q.len - t0 < kL;   // rows of the next sequence lie behind this one's
      const bool in = t0 + row < q.len;
      const float* v = vec + (c & 1) * kVec;
      if (!wait(b_dec + (c & 1), (uint32_t)((c - c_begin) >> 1) & 1u) || !wait(b_x, ph)) break;
      if (FULL ? !wait(b_s, ph) : !wait(b_bc, ph)) break;
      tc::fence_after_sync();
      // ---- X~ in three terms: token `row`, 32 columns
      {
        const float w = v[3 * kL + row];
        const uint64_t w2 = pair(w, w), minus = pair(-1.f, -1.f);
        const bool clear = tail && !in;
        uint4 xv[4];   // read ahead of the first store
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xv[i] = *reinterpret_cast<const uint4*>(smem + Cf::oX + (uint32_t)row * 128 + (((4 * half + i) ^ rsw) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = (uint32_t)row * 128 + (((4 * half + i) ^ rsw) << 4);
          if (clear) {
            xv[i] = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + Cf::oX + at) = xv[i];
            for (uint32_t k = 0; k < Cf::NT; ++k) *reinterpret_cast<uint4*>(smem + Cf::oB + k * kTile + at) = xv[i];
          }
          const uint32_t xi[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
          uint32_t t1[4], t2[4], t3[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float e, f;
            uint64_t u = mul2(pair(lo_f(xi[j]), hi_f(xi[j])), w2);
            unpair(u, e, f);
            t1[j] = pack2(e, f);
            u = fma2(pair(lo_f(t1[j]), hi_f(t1[j])), minus, u);   // exact
            unpair(u, e, f);
            t2[j] = pack2(e, f);
            u = fma2(pair(lo_f(t2[j]), hi_f(t2[j])), minus, u);
            unpair(u, e, f);
            t3[j] = pack2(e, f);
          }
          *reinterpret_cast<uint4*>(smem + Cf::term0 + at) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
          *reinterpret_cast<uint4*>(smem + Cf::term1 + at) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
          *reinterpret_cast<uint4*>(smem + Cf::term2 + at) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
        }
      }
      arrive(b_xt);
      if (FULL) {
        // ---- M from S in place; Y = D x + the state's part scaled by the row's decay
        const float my_cum = v[row];
#pragma unroll 1
        for (int jj = 0; jj < 2; ++jj) {
          const int j = 2 * half + jj;
          uint32_t m[16];
          if (j > qd) {
#pragma unroll
            for (int i = 0; i < 16; ++i) m[i] = 0;
          } else {
            float s[32];
            tc::tmem_ld32(tlane + kColS + 32 * j, s);
            const bool diag = j == qd;
            if (!diag || v[5 * kL + 12 + j] != 0.f) {
              const float r = ex2(my_cum - v[5 * kL + (diag ? 0 : 4) + j]);
              const float* wv = v + (diag ? 2 : 1) * kL + 32 * j;
              const uint64_t r2 = pair(r, r);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 w = *reinterpret_cast<const float4*>(wv + i);
                float e0, e1, e2, e3;
                unpair(mul2(mul2(pair(s[i], s[i + 1]), pair(w.x, w.y)), r2), e0, e1);
                unpair(mul2(mul2(pair(s[i + 2], s[i + 3]), pair(w.z, w.w)), r2), e2, e3);
                if (diag) {
                  e0 = i <= lane ? e0 : 0.f;
                  e1 = i + 1 <= lane ? e1 : 0.f;
                  e2 = i + 2 <= lane ? e2 : 0.f;
                  e3 = i + 3 <= lane ? e3 : 0.f;
                }
                m[i / 2] = pack2(e0, e1);
                m[i / 2 + 1] = pack2(e2, e3);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 cs = *reinterpret_cast<const float2*>(v + 32 * j + i);
                const float2 ss = *reinterpret_cast<const float2*>(v + 4 * kL + 32 * j + i);
                m[i / 2] = pack2(i <= lane ? s[i] * ex2(my_cum - cs.x) * ss.x : 0.f,
                                 i + 1 <= lane ? s[i + 1] * ex2(my_cum - cs.y) * ss.y : 0.f);
              }
            }
          }
          tmem_st16(tlane + kColS + 64 * half + 16 * jj, m);
        }
        {
          float y[32];
          tc::tmem_ld32(tlane + kColY + 32 * half, y);
          const float r = ex2(my_cum);
          const uint64_t r2 = pair(r, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 xv = *reinterpret_cast<const uint4*>(smem + Cf::oX + (uint32_t)row * 128 + (((4 * half + i) ^ rsw) << 4));
            const uint32_t xi[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int e = 8 * i + 2 * j;
              unpair(fma2(pair(y[e], y[e + 1]), r2, mul2(D2, pair(lo_f(xi[j]), hi_f(xi[j])))), y[e], y[e + 1]);
            }
          }
          tc::tmem_st32(tlane + kColY + 32 * half, y);
        }
        tmem_wait_st();
        arrive(b_m);
      }
      // ---- the state after the chunk
      const float total = v[5 * kL + 8];
      __syncwarp();   // the last that this chunk needs of its decays
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b_free + (c & 1))) : "memory");
      if (!wait(b_u, ph)) break;
      tc::fence_after_sync();
      {
        float u[32];
        tc::tmem_ld32(tlane + kColU + 32 * half, u);
        const float d = ex2(total);
        const uint64_t d2 = pair(d, d);
#pragma unroll
        for (int i = 0; i < 32; i += 2) unpair(fma2(d2, pair(h[i], h[i + 1]), pair(u[i], u[i + 1])), h[i], h[i + 1]);
        log_total += total;
      }
      if (!FULL) {
        arrive(b_next);
        continue;
      }
      if (c + 1 < c_end) put_state();
      uint4 zr[4];
      if (a.z) {
        const __nv_bfloat16* z = a.z + (packed ? (q.start + t0 + row) * a.z_tok : seq * a.z_seq + (t0 + row) * a.z_tok) +
                                 (long long)head * a.P + p0 + 32 * half;
        const int pc = a.P - p0 - 32 * half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          zr[i] = make_uint4(0, 0, 0, 0);
          if (!in || 8 * i >= pc) continue;
          if (a.z_vec) {
            zr[i] = *reinterpret_cast<const uint4*>(z + 8 * i);
          } else {
            const unsigned short* zs = reinterpret_cast<const unsigned short*>(z + 8 * i);
            zr[i] = make_uint4(zs[0] | (uint32_t)zs[1] << 16, zs[2] | (uint32_t)zs[3] << 16,
                               zs[4] | (uint32_t)zs[5] << 16, zs[6] | (uint32_t)zs[7] << 16);
          }
        }
      }
      if (!wait(b_y, ph)) break;
      tc::fence_after_sync();
      float y[32];
      tc::tmem_ld32(tlane + kColY + 32 * half, y);
      arrive(b_next);   // the next chunk's S and C h^T may start
      // ---- output rows: Y, gated, over X (every product that reads X is done)
      __nv_bfloat16* yp = a.y + (packed ? (q.start + t0 + row) * a.y_tok : 0) + (long long)head * a.P + p0 + 32 * half;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = (uint32_t)row * 128 + (((4 * half + i) ^ rsw) << 4);
        const uint32_t zi[4] = {zr[i].x, zr[i].y, zr[i].z, zr[i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float e = y[8 * i + 2 * j], f = y[8 * i + 2 * j + 1];
          if (a.z) unpair(mul2(pair(e, f), silu2(pair(lo_f(zi[j]), hi_f(zi[j])))), e, f);
          o[j] = pack2(e, f);
        }
        const uint4 ov = make_uint4(o[0], o[1], o[2], o[3]);
        if (!tail) *reinterpret_cast<uint4*>(smem + Cf::oX + at) = ov;
        else if (in && p0 + 32 * half + 8 * i < a.P) *reinterpret_cast<uint4*>(yp + 8 * i) = ov;
      }
      arrive(b_out);
    }
    if (*fail) {
      if (tid == 0) atomicOr(&a.status->flags, kStatusTimeout);
    } else if (!FULL) {
      if (n < NN) {
        float* wsq = a.ws + (seq * slices + slice) * ws_floats(a.nseg, NN);
        float* e = wsq + ((long long)seg * 64 + 32 * half) * NN;
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i * NN + n] = h[i];
        if (tid == 0) wsq[(long long)a.nseg * 64 * NN + seg] = ex2(log_total);
      }
    } else if (last && a.state && n_ok) {
      float* dst = a.state + ((q.slot * a.H + head) * a.P + p0 + 32 * half) * a.N + n;
      const int pc = a.P - p0 - 32 * half;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < pc) dst[(long long)i * a.N] = h[i];
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, kCols);
}

// ---------------------------------------------------------------------------
// host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = []() -> EncodeTiled {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// [batch][tokens][heads][width] bfloat16 in tiles of [128 tokens][64]
bool encode(CUtensorMap* m, const void* base, long long width, long long heads, long long tokens, long long batch,
            long long tok, long long seq) {
  EncodeTiled fn = encode_fn();
  if (!fn || (reinterpret_cast<uintptr_t>(base) & 15u) || tok % 8 || width % 8) return false;
  if (tokens <= 1) tok = width * heads;   // an unused stride need not be valid
  if (batch <= 1) seq = tok * tokens;
  if (tok < 8 || seq < 8 || seq % 8) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)tok * 2, (cuuint64_t)seq * 2};
  const cuuint32_t box[4] = {64, 1, kL, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NN>
cudaError_t launch(const SsmArgs& s, const PromptArgs& a, const PromptPlan& plan, const CUtensorMap* maps,
                   cudaStream_t st) {
  const long long ctas = s.seqs.n_seq * a.H * a.pslices * plan.nseg;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  constexpr int bytes = (int)Cfg<NN>::bytes;
  cudaError_t e = cudaFuncSetAttribute(ssm_prompt_kernel<NN, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if (plan.nseg > 1) {
    e = cudaFuncSetAttribute(ssm_prompt_kernel<NN, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    ssm_prompt_kernel<NN, false><<<(unsigned int)ctas, kThreads, bytes, st>>>(maps[0], maps[1], maps[2], maps[3], a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  ssm_prompt_kernel<NN, true><<<(unsigned int)ctas, kThreads, bytes, st>>>(maps[0], maps[1], maps[2], maps[3], a);
  return cudaGetLastError();
}

}  // namespace

PromptPlan ssm_prompt_plan(long long n_seq, long long max_len, long long H, long long P, long long N, bool bf16,
                           int sm_count) {
  PromptPlan p{};
  p.fits = bf16 && P % 8 == 0 && N % 8 == 0 && N <= 128 && max_len >= kPromptMin && H < (1 << 20) && P < (1 << 20);
  if (!p.fits) return p;
  const long long slices = H * ((P + 63) / 64), chunks = (max_len + kL - 1) / kL, slots = 2LL * sm_count;
  p.nn = N <= 64 ? 64 : 128;
  p.nseg = 1;
  p.seg_chunks = chunks;
  // Two CTAs an SM.  While the slices leave most of them idle, segments shorten the longest run of
  // chunks; a chunk of the first launch costs about half of one of the second.
  double best = (double)((n_seq * slices + slots - 1) / slots) * chunks;
  for (long long k = 2; k <= chunks && k <= 64 && n_seq * slices * k <= 2 * slots; ++k) {
    const long long per = (chunks + k - 1) / k, nseg = (chunks + per - 1) / per;
    if (nseg != k) continue;
    const double cost = 1.5 * (double)((n_seq * slices * k + slots - 1) / slots) * per + 2.0 + 0.1 * k;
    if (cost < best) {
      best = cost;
      p.nseg = (int)k;
      p.seg_chunks = per;
    }
  }
  if (p.nseg > 1) p.ws_bytes = (size_t)(n_seq * slices) * ws_floats(p.nseg, p.nn) * sizeof(float);
  return p;
}

cudaError_t launch_ssm_prompt(const SsmArgs& s, const PromptPlan& plan, cudaStream_t st, bool* used) {
  *used = false;
  const bool packed = s.seqs.offsets != nullptr;
  const long long tokens = s.seqs.T, batch = packed ? 1 : s.seqs.n_seq;
  CUtensorMap maps[4];
  if (!encode(&maps[0], s.x, s.P, s.H, tokens, batch, s.x_tok, s.x_seq) ||
      !encode(&maps[1], s.B, s.N, s.G, tokens, batch, s.B_tok, s.B_seq) ||
      !encode(&maps[2], s.C, s.N, s.G, tokens, batch, s.C_tok, s.C_seq) ||
      !encode(&maps[3], s.y, s.P, s.H, tokens, batch, s.y_tok, s.y_seq))
    return cudaSuccess;
  PromptArgs a{};
  a.dt = static_cast<const __nv_bfloat16*>(s.dt);
  a.A = s.A; a.D = s.D; a.dt_bias = s.dt_bias; a.state = s.state; a.ws = s.ws;
  a.z = static_cast<const __nv_bfloat16*>(s.z);
  a.y = static_cast<__nv_bfloat16*>(s.y);
  a.seqs = s.seqs;
  a.H = (int)s.H; a.P = (int)s.P; a.G = (int)s.G; a.N = (int)s.N;
  a.pslices = (int)((s.P + 63) / 64);
  a.nseg = plan.nseg;
  a.seg_chunks = (int)plan.seg_chunks;
  a.dt_seq = s.dt_seq; a.dt_tok = s.dt_tok; a.z_seq = s.z_seq; a.z_tok = s.z_tok; a.y_seq = s.y_seq; a.y_tok = s.y_tok;
  a.softplus = s.softplus;
  a.z_vec = ((reinterpret_cast<uintptr_t>(s.z) & 15u) | (unsigned long long)(s.z_tok % 8) |
             (unsigned long long)(packed ? 0 : s.z_seq % 8)) == 0;
  a.status = s.status;
  *used = true;
  return plan.nn == 64 ? launch<64>(s, a, plan, maps, st) : launch<128>(s, a, plan, maps, st);
}

}  // namespace vla
