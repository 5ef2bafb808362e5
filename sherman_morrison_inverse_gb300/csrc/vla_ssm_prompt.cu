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
// once: 2^-9 of each term, so of the sum of the terms' magnitudes.  An output that cancels is further off than
// its own rounding (over 8 x 4096 tokens the error against 64 bits is 0.0019 of the norm, 0.0017 of it the
// output's rounding); two terms of each would take 16 products more than these 40.  No decay is a difference of sums from the chunk's
// start: after a token that decays by e^-10^5 both would be large and keep few bits of what came since.
// c_L - c_s is summed from the end, c_t - c_s from the tokens and blocks strictly between.
//
// exp(c_t - c_s) takes no exponential a pair: with e_j the sum at the end of block j of 32 tokens s,
// exp(c_t - e_j) exp(e_j - c_s) is one factor a row (its sum within its own block, and the blocks
// between) and one a column, both at most 1, for the rows behind the block.  In a diagonal block both
// factors are of the sums from the block's start; the column's is then at least 1, so this holds while
// the block's sums stay below 2^100 and its steps below 2^26, and beyond that (nothing is left of a token
// a few tokens later) the exponentials are taken pair by pair, of a running sum from the row's token back.
//
// Roles (24 warps, one CTA an SM; they meet on mbarriers and every operand has two places, so the two
// sides of a chunk run side by side and ahead of each other):
//   0-7   output: M from S, then Y = D x + exp(c) C h^T, later y from Y
//   8-15  state: X~, then h' from its product U
//   16    issues C h^T and M X               17  issues B^T X~ and then S of the next chunk
//   18    issues the loads                    19  stores y
//   20-23 decays, 32 tokens of a chunk each
// (the first launch of a cut sequence has no output: warps 0-7 form half of X~ there)
// In order: S of the next chunk is formed while M of this one is, M of the next one while M X of
// this one runs.  The state's side takes X~, U, h, X~ .. in turn (X~ and U have one place each): so U
// comes before S, and h's copy is written after the next X~.
// A NaN or infinity of x must not meet the zeros above M's diagonal: it would reach earlier tokens.  The
// warp that issues M X looks the tile over while M is formed; what is not finite it takes out, once the state's
// warps have read it, and notes its column and token: from there on the column's outputs are NaN (so is its
// row of the state, where the recurrence may have infinities).  8 x 4096 tokens of 64 heads: 289.3 -> 291.2 us;
// by the output's warps, on their way to D x, 297.7; by the warp that stores y 300.
// All of this code runs once a chunk: what does not fit the instruction caches is fetched again
// every time (written out, 122 KB of it took three times as long), so loops stay rolled, a body
// takes 16 columns, and a wait that does not succeed at once goes through one shared function.
//
// Operands.  B, C [128 tokens][N] and X [128][64] arrive by TMA as 128-byte-swizzled tiles of 64
// columns; the same B tile is the K-major operand of S and the transposed (MN-major) one of the
// state's product.  M replaces S in tensor memory as the A operand of M X.  The terms t1, t2, t3 of X~ make
// two operands of 128 columns, [t1 | t2 / 2] and [t2 / 2 | t3], that share the tile of t2 / 2 and an
// accumulator (a product of 64 columns takes as long as one of 128: 16 of these, not 24).
//
// Few slices: the sequence is cut into segments, one CTA each.  A first launch forms what every
// segment but a sequence's last adds to the state (B^T X~ alone), the second starts each segment from
// those, joined in a fixed order.  The second launch's CTAs start beside the first's and wait where
// they read what it leaves.  Many slices, but the last wave of CTAs far from full: only what is left
// for that wave is cut, its first launch and the whole slices share the SMs.
//
// What bounds it.  8 sequences of 4096 tokens, 64 heads of 64, 128 states: 291 us (315 uncut), about
// 4450 cycles a chunk and SM.  The 40 products of a chunk take 65 to 75 cycles each, whatever their
// width up to 128 columns: at least 2800 cycles (the tensor pipe is 43 % busy by the counters, memory
// 24 %).  Both sides of a chunk take the whole period.  The state's: X~ 1370, its product 1900 (it shares the
// pipe with the output's), h 540, hand-overs 700, one after another because X~ and U have one place each and
// the same warps form X~ and read U (only h depends on the chunk before); the output's about 4400.  Side by side in one
// CTA with everything double-buffered, not as two CTAs an SM that hide each other (328 us, uncut) nor
// with 16 warps a side; dropping a term of X~ would save 4 % and lose the float32 state.
// One sequence of 16384 tokens, 16 heads, gated: 80 us in 9 segments (3.5 more without the overlap of the
// launches).  Nine packed prompts of 1 to 2047 tokens, 16 heads of 128, 64 states, gated: 56 us.
#include <cuda.h>   // CUtensorMap and the encode entry point's types (resolved at run time)

#include <algorithm>
#include <atomic>

#include "vla_layer.cuh"
#include "vla_ssm_prompt.cuh"
#include "vla_tc.cuh"

namespace vla {
namespace {

constexpr int kL = 128;            // tokens a chunk
constexpr int kSide = 256;         // threads of the output's and of the state's warps
constexpr int kThreads = 768;
constexpr uint32_t kTile = 16384;  // bytes of a [128][64] bfloat16 tile
constexpr uint32_t kCols = 512;    // tensor memory columns: S (M) [2] | Y [2] | U
constexpr uint32_t kColS = 0, kColY = 256, kColU = 384;
constexpr int kVec = 5 * kL + 24;  // floats of a chunk's decays
constexpr int kDec = 4;            // chunks of decays
constexpr int kUnits = 16;         // pieces of 32 tokens and 16 columns of X~
constexpr int kOdd = 65;           // words about X's values that are not finite

// mbarriers (where there are two or more, chunk i uses i mod their number)
enum : int {
  kFullB = 0,      // [2] B has landed
  kFullC = 2,      //     C
  kFullX = 3,      // [2] X
  kEmptyB = 5,     // [2] S and U have read B
  kEmptyC = 7,     //     S and C h^T have read C
  kEmptyX = 8,     // [2] X~, D x and M X have read X
  kFullS = 10,     // [2] S is formed
  kEmptyS = 12,    // [2] M X is formed: S's place is free
  kFullYi = 14,    // [2] C h^T is formed (and h's copy read)
  kM = 16,         //     M, and D x + exp(c) C h^T, are written
  kFullY = 17,     // [2] M X is added
  kH = 19,         //     the copy of h before chunk i is written
  kEmptyY = 20,    // [2] Y is read
  kXt = 22,        //     X~ is written, the U before it read
  kFullU = 23,     //     U is formed
  kFullDec = 24,   // [4] decays are written
  kEmptyDec = 28,  // [4] and read
  kStage = 32,     //     y is staged
  kStaged = 33,    //     and its store has read it
  kFullZ = 34,     //     z has landed where y will be staged
  kReadX = 35,     // [2] X~ has read X
  kBars = 37
};

// Shared memory: B [2] | C | X [2] | X~ (three terms) | state (bfloat16, [n][64 p]) | y | decays | barriers,
// two words | for each place of X: its columns' first tokens with a value that is not finite [64], and the
// chunk that has any
template <int NN>
struct Cfg {
  static constexpr uint32_t NT = NN / 64;
  static constexpr uint32_t oB = 0, oC = 2 * NT * kTile, oX = oC + NT * kTile, oT = oX + 2 * kTile;
  static constexpr uint32_t oH = oT + 3 * kTile, oY = oH + NN * 128, oVec = oY + kTile;
  static constexpr uint32_t oOdd = oVec + 4 * kDec * kVec + 8 * kBars + 8;
  static constexpr uint32_t bytes = oOdd + 2 * 4 * kOdd;
};

// Matrix descriptor of a 128-byte-swizzled operand: `lbo` bytes between blocks of 64 in the
// contiguous dimension of a transposed operand, 1024 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;   // instruction descriptor: MN-major operands

// One MMA, D (+)= X Y for a K step of 16, issued by the lane whose `one` is set.  The whole warp runs the
// loop around it, predicated and not branched, so that descriptors and addresses stay in uniform
// registers: from a divergent branch each MMA takes over a hundred cycles to issue.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t xdesc, uint64_t ydesc, uint32_t idesc, bool accumulate,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(xdesc), "l"(ydesc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
      : "memory");
}
// The same with X in tensor memory (bfloat16, two K elements a column).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t x_tmem, uint64_t ydesc, uint32_t idesc, bool accumulate,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(x_tmem), "l"(ydesc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(one)
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

// Bounded wait of a whole warp whose first poll has failed; gives up early when another warp has.
// One lane polls: two dozen warps that poll with all their lanes slow every access to shared memory.
__device__ __noinline__ bool wait_on(uint64_t* b, uint32_t parity, volatile int* fail) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) {
    unsigned long long t_start = 0;
    while (true) {
#pragma unroll 1
      for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(b, parity);
      if (ok || *fail) break;
      const unsigned long long now = globaltimer_ns();
      if (t_start == 0) t_start = now;
      if (now - t_start > kWaitLimitNs) {
        *fail = 1;
        break;
      }
    }
  }
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// a 0 + b for pairs of bfloat16
__device__ __forceinline__ uint32_t times_zero(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0u), "r"(b));
  return r;
}
// Takes what is not finite out of 8 bfloat16 values of X and notes it in their columns' words.  A word is
// (chunk + 1) 128 + 127 - row, so that the largest is the first row of the latest chunk.
__device__ __noinline__ void take_out(unsigned char* at, uint32_t* word, uint32_t value) {
  unsigned short* v = reinterpret_cast<unsigned short*>(at);
#pragma unroll 1
  for (int c = 0; c < 8; ++c)
    if ((v[c] & 0x7f80) == 0x7f80) {
      v[c] = 0;
      atomicMax(word + c, value);
    }
}

// NaN for those of 8 bfloat16 outputs whose columns had such a value at this row (`value`) or before.
__device__ __noinline__ void put_nan(void* at, const volatile uint32_t* word, uint32_t value) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c)
    if (word[c] >= value) static_cast<unsigned short*>(at)[c] = 0x7fff;
}

// Named barrier over n threads that also ORs a flag across them.
__device__ __forceinline__ bool named_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
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

// The n lowest bits set, n < 0: none, n > 32: all.
__device__ __forceinline__ uint32_t low_bits(int n) {
  uint32_t r;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(n < 0 ? 0 : n));
  return r;
}

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
  int whole;         // (sequence, slice) pairs that are not cut, the first ones
  long long dt_seq, dt_tok, z_seq, z_tok, y_seq, y_tok;
  bool softplus;
  DevStatus* status;
};

// Workspace of one (sequence, slice): nseg states of 64 x NN floats (the place of the last segment
// holds a copy of the state before the sequence), then their decays.
__host__ __device__ constexpr long long ws_floats(int nseg, int NN) { return (long long)nseg * 64 * NN + (nseg + 63) / 64 * 64; }

// FULL: the outputs and the final state; else what the segment adds to the state.
// GATE: 0 no z, 1 z by TMA through y's staging tile, 2 z read directly (rows not on 16-byte boundaries).
template <int NN, bool FULL, int GATE>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_prompt_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_B,
                      const __grid_constant__ CUtensorMap map_C, const __grid_constant__ CUtensorMap map_y,
                      const __grid_constant__ CUtensorMap map_z,
                      const __grid_constant__ PromptArgs a) {
  using Cf = Cfg<NN>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = a.H * a.pslices;
  if (!FULL) all_started();
  // the whole pairs' CTAs come first, then the segments; beside whole pairs the last ones, which are longer, first
  const int pairs = (int)a.seqs.n_seq * slices, block = (int)blockIdx.x + (FULL ? 0 : a.whole);
  const bool is_whole = FULL && block < a.whole;
  const int turn = is_whole ? 0 : (block - a.whole) / (pairs - a.whole);
  const int at = block - turn * (pairs - a.whole), seg = FULL && !is_whole && a.whole > 0 ? a.nseg - 1 - turn : turn;
  const int seq = at / slices, slice = at - seq * slices;
  const int head = slice / a.pslices, p0 = (slice - head * a.pslices) * 64, group = head / (a.H / a.G);

  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, seq, &bad);
  if (bad && tid == 0 && FULL) atomicOr(&a.status->flags, bad);
  const int chunks = (int)((q.len + kL - 1) / kL), seg_chunks = is_whole ? chunks : a.seg_chunks;
  // segments of this sequence, none without tokens; beside whole pairs the last one takes what is left
  int segs = seg_chunks > 0 ? (chunks + seg_chunks - 1) / seg_chunks : 0;
  if (segs > a.nseg) segs = a.nseg;
  const bool last = seg == segs - 1;
  if (!q.run || seg >= segs || (!FULL && last)) {
    if (FULL && a.nseg > 1) wait_for_first();
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {   // the swizzled tiles need it; report rather than run misaligned
    if (tid == 0) atomicOr(&a.status->flags, kStatusTimeout);
    return;
  }

  // decays of chunk i at vec + (i mod 4) kVec: inc [128] log2 decay from the block's start up to a token;
  // wcol [128] s exp(e_j - c), j the token's block; wdg [128] s exp(-inc), or where that does not hold the
  // token's own log2 decay; wx [128] s exp(c_L - c); step [128] s; then [4] sums before the blocks,
  // [8] the total, [12..16) the blocks' own sums, [16..20) whether wdg holds
  float* vec = reinterpret_cast<float*>(smem + Cf::oVec);
  uint64_t* bar = reinterpret_cast<uint64_t*>(vec + kDec * kVec);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + kBars);
  volatile int* fail = reinterpret_cast<volatile int*>(tslot + 1);

  const bool packed = a.seqs.offsets != nullptr;
  const int row0 = packed ? (int)q.start : 0, batch = packed ? 0 : (int)seq;   // tensor map coordinates
  const int n_chunks = last ? chunks - seg * seg_chunks : seg_chunks;
  const int t_first = seg * seg_chunks * kL;
  const unsigned int left = (unsigned int)((int)q.len - t_first);   // tokens from t_first on

  if (tid == 0) {
    constexpr int W = kSide / 32;
    for (int i = 0; i < kBars; ++i) {
      int count = 1;
      if (i == kEmptyB || i == kEmptyB + 1 || i == kEmptyC) count = FULL ? 2 : 1;
      if (i == kEmptyX || i == kEmptyX + 1) count = FULL ? 2 * W + 1 : 2 * W;
      if (i >= kEmptyDec && i < kEmptyDec + kDec) count = 2 * W;
      if (i >= kFullDec && i < kFullDec + kDec) count = 4;
      if (i == kM || i == kH || i == kEmptyY || i == kEmptyY + 1 || i == kStage) count = W;
      if (i == kXt) count = FULL ? W : 2 * W;
      if (i == kReadX || i == kReadX + 1) count = W;
      mbar_init(bar + i, count);
    }
    *fail = 0;
    fence_mbar_init();
  }
  uint32_t* odd = reinterpret_cast<uint32_t*>(smem + Cf::oOdd);
  if (tid < 2 * kOdd) odd[tid] = 0;
  if (warp == 1) tc::tmem_alloc(tslot, kCols);
  if (warp == 18 && lane < 4) prefetch_map(lane == 0 ? &map_B : lane == 1 ? &map_x : lane == 2 ? &map_C : &map_y);

  const int row = tid & (kL - 1), half = (tid >> 7) & 1;   // token or state n; columns 32 half ..
  const uint32_t rsw = (uint32_t)(row & 7);
  const uint32_t row_at = (uint32_t)row * 128;
  const int pc = a.P - p0 - 32 * half;   // columns of this thread that exist
  float* wsq = a.nseg > 1 && !is_whole ? a.ws + (at - a.whole) * ws_floats(a.nseg, NN) : nullptr;
  const int n = row;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);   // the same in every lane
  constexpr uint32_t kId = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);   // bf16, 128 rows
  constexpr uint32_t kN64 = (64u >> 3) << 17, kN128 = (128u >> 3) << 17;

  // Wait of a whole warp for completion `use` (0, 1, ..) of a barrier.
  auto wait = [&](int b, int use) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar + b, (uint32_t)use & 1u))) return true;
    return wait_on(bar + b, (uint32_t)use & 1u, fail);
  };
  // One arrival a warp.
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar + b)) : "memory");
  };
  const bool one = lane == 0;
  auto arrive_one = [&](int b) {   // by one lane, after a __syncwarp
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar + b)) : "memory");
  };
  const int last_i = n_chunks - 1;
  // whether rows of the next sequence lie behind this one's in the last chunk
  const bool ragged = packed && last && (left & (kL - 1)) != 0;

  const uint64_t minus = pair(-1.f, -1.f), minus_two = pair(-2.f, -2.f), one_half = pair(0.5f, 0.5f);
  // One piece of X~ of chunk i in three terms: 32 tokens and 16 columns
  auto make_piece = [&](int i, int piece) {
    const int token = 32 * (piece & 3) + lane, r = i & 1;
    const uint32_t c = 2 * ((uint32_t)piece >> 2), sw = (uint32_t)(token & 7);
    const uint32_t at0 = (uint32_t)token * 128 + ((c ^ sw) << 4), at1 = (uint32_t)token * 128 + (((c + 1) ^ sw) << 4);
    const float w = vec[(i % kDec) * kVec + 3 * kL + token];
    const uint64_t w2 = pair(w, w);
    uint4 xa = *reinterpret_cast<const uint4*>(smem + Cf::oX + r * kTile + at0);
    uint4 xb = *reinterpret_cast<const uint4*>(smem + Cf::oX + r * kTile + at1);
    // rows of the next sequence: none of them may reach the product
    if (ragged && i == last_i && (unsigned int)(i * kL + token) >= left) xa = xb = make_uint4(0, 0, 0, 0);
    const uint32_t xi[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
    uint32_t t1[8], t2[8], t3[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float e, f;
      uint64_t z = mul2(pair(lo_f(xi[j]), hi_f(xi[j])), w2);
      unpair(z, e, f);
      t1[j] = pack2(e, f);
      z = fma2(pair(lo_f(t1[j]), hi_f(t1[j])), minus, z);   // exact
      unpair(mul2(z, one_half), e, f);
      t2[j] = pack2(e, f);   // half of the second term
      z = fma2(pair(lo_f(t2[j]), hi_f(t2[j])), minus_two, z);
      unpair(z, e, f);
      t3[j] = pack2(e, f);
    }
    unsigned char* to = smem + Cf::oT;
    *reinterpret_cast<uint4*>(to + at0) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
    *reinterpret_cast<uint4*>(to + at1) = make_uint4(t1[4], t1[5], t1[6], t1[7]);
    *reinterpret_cast<uint4*>(to + kTile + at0) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
    *reinterpret_cast<uint4*>(to + kTile + at1) = make_uint4(t2[4], t2[5], t2[6], t2[7]);
    *reinterpret_cast<uint4*>(to + 2 * kTile + at0) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
    *reinterpret_cast<uint4*>(to + 2 * kTile + at1) = make_uint4(t3[4], t3[5], t3[6], t3[7]);
    fence_proxy_async_smem();
  };

  if (warp < kSide / 32) {
    if constexpr (!FULL) {
      // ------------------------------------------------ the other half of X~
      for (int i = 0; i < n_chunks; ++i) {
        if (!wait(kFullDec + i % kDec, i / kDec) || !wait(kFullX + (i & 1), i >> 1) || (i > 0 && !wait(kFullU, i - 1))) break;
        make_piece(i, kSide / 32 + warp);
        arrive(kXt);
        if (one) {
          arrive_one(kEmptyX + (i & 1));
          arrive_one(kEmptyDec + i % kDec);
        }
      }
    } else {
      // ------------------------------------------------ output
      const int qd = warp & 3;   // block of rows
      const uint32_t tlane = tmem + ((uint32_t)(32 * qd) << 16);
      const float Dh = a.D ? a.D[head] : 0.f;
      const uint64_t D2 = pair(Dh, Dh);
      // y of chunk i: Y, gated
      auto finish = [&](int i) -> bool {
        const long long t = t_first + (long long)i * kL + row;
        const bool in = (unsigned int)(i * kL + row) < left, tail = ragged && i == last_i;
        const __nv_bfloat16* z = GATE == 2 ? a.z + (packed ? (q.start + t) * a.z_tok : seq * a.z_seq + t * a.z_tok) +
                                                 (long long)head * a.P + p0 + 32 * half
                                           : nullptr;
        if (!wait(kFullY + (i & 1), i >> 1)) return false;
        if (GATE == 1 ? !wait(kFullZ, i) : (i > 0 && !wait(kStaged, i - 1))) return false;
        tc::fence_after_sync();
#pragma unroll 1
        for (int k = 0; k < 32; k += 16) {
          uint4 zr[2];
          if (GATE == 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              zr[j] = make_uint4(0, 0, 0, 0);
              const int c = k + 8 * j;
              if (!in || c >= pc) continue;
              const unsigned short* zs = reinterpret_cast<const unsigned short*>(z + c);
              zr[j] = make_uint4(zs[0] | (uint32_t)zs[1] << 16, zs[2] | (uint32_t)zs[3] << 16,
                                 zs[4] | (uint32_t)zs[5] << 16, zs[6] | (uint32_t)zs[7] << 16);
            }
          }
          float y[16];
          tc::tmem_ld16(tlane + kColY + 64 * (i & 1) + 32 * half + k, y);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = k + 8 * j;
            uint4* at = reinterpret_cast<uint4*>(smem + Cf::oY + row_at + (((uint32_t)(4 * half + (c >> 3)) ^ rsw) << 4));
            if (GATE == 1) zr[j] = *at;
            const uint32_t zi[4] = {zr[j].x, zr[j].y, zr[j].z, zr[j].w};
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float f = y[8 * j + 2 * e], g = y[8 * j + 2 * e + 1];
              if (GATE) unpair(mul2(pair(f, g), silu2(pair(lo_f(zi[e]), hi_f(zi[e])))), f, g);
              w[e] = pack2(f, g);
            }
            const uint4 o = make_uint4(w[0], w[1], w[2], w[3]);
            if (!tail) {
              *at = o;
            } else if (in && c < pc) {
              *reinterpret_cast<uint4*>(a.y + (q.start + t) * a.y_tok + (long long)head * a.P + p0 + 32 * half + c) = o;
            }
          }
        }
        const uint32_t* word = odd + (i & 1) * kOdd;
        if (*reinterpret_cast<const volatile uint32_t*>(word + 64) == (uint32_t)i + 1) {
#pragma unroll 1
          for (int c = 0; c < 32; c += 8) {
            void* at = smem + Cf::oY + row_at + (((uint32_t)(4 * half + (c >> 3)) ^ rsw) << 4);
            if (tail) {
              if (!in || c >= pc) continue;
              at = a.y + (q.start + t) * a.y_tok + (long long)head * a.P + p0 + 32 * half + c;
            }
            put_nan(at, word + 32 * half + c, ((uint32_t)i + 1) * kL + (kL - 1 - row));
          }
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        arrive(kEmptyY + (i & 1));
        if (one) arrive_one(kStage);
        return true;
      };
      for (int i = 0; i <= n_chunks; ++i) {   // the last turn finishes the last chunk only
        const int r = i & 1, u = i >> 1;
        const float* v = vec + (i % kDec) * kVec;
        float row_decay = 0.f;
        if (i < n_chunks) {
          if (!wait(kFullDec + i % kDec, i / kDec) || !wait(kFullS + r, u)) break;
          tc::fence_after_sync();
          const float my_inc = v[row], *sums = v + 5 * kL;
          row_decay = ex2(sums[qd] + my_inc);
          // M from S in place: blocks 2 half and 2 half + 1 of s end up at S's columns 64 half + 0 and + 16
          const uint32_t ts = tlane + kColS + 128 * r + 64 * half;
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            const int j = 2 * half + g;
            uint32_t m[16];
            if (j > qd) {
#pragma unroll
              for (int k = 0; k < 16; ++k) m[k] = 0;
            } else {
              float s[32];
              tc::tmem_ld32(ts + 32 * g, s);
              const bool diag = j == qd;
              if (!diag || sums[16 + j] != 0.f) {
                // the blocks strictly between: at most two
                const float f = ex2(my_inc + ((j + 1 < qd ? sums[13 + j] : 0.f) + (j + 2 < qd ? sums[14 + j] : 0.f)));
                const float* wv = v + (diag ? 2 : 1) * kL + 32 * j;
                const uint64_t f2 = pair(f, f);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                  const float4 w = *reinterpret_cast<const float4*>(wv + k);
                  float e0, e1, e2, e3;
                  // the factors first: one may be near 2^127, their product is at most the step
                  unpair(mul2(pair(s[k], s[k + 1]), mul2(pair(w.x, w.y), f2)), e0, e1);
                  unpair(mul2(pair(s[k + 2], s[k + 3]), mul2(pair(w.z, w.w), f2)), e2, e3);
                  m[k / 2] = pack2(e0, e1);
                  m[k / 2 + 1] = pack2(e2, e3);
                }
                if (diag) {   // columns behind the row's own are zero
#pragma unroll
                  for (int k = 0; k < 16; ++k) m[k] &= low_bits(16 * (lane + 1 - 2 * k));
                }
              } else {
                const float* cv = v + 32 * j;
                float back = 0.f;   // the tokens behind column k, up to the row's own
#pragma unroll
                for (int k = 31; k >= 0; --k) {
                  const bool in = k <= lane;
                  s[k] = in ? s[k] * (ex2(back) * cv[4 * kL + k]) : 0.f;
                  if (in) back += cv[2 * kL + k];
                  if ((k & 1) == 0) m[k / 2] = pack2(s[k], s[k + 1]);
                }
              }
            }
            tmem_st16(ts + 16 * g, m);
          }
          arrive(kEmptyDec + i % kDec);
        }
        if (i > 0 && !finish(i - 1)) break;
        if (i == n_chunks) break;
        // Y = D x + the state's part scaled by the row's decay
        if (!wait(kFullX + r, u) || !wait(kFullYi + r, u)) break;
        tc::fence_after_sync();
        const bool clear = ragged && i == last_i && (unsigned int)(i * kL + row) >= left;
        const uint32_t ty = tlane + kColY + 64 * r + 32 * half;
        const uint64_t f2 = pair(row_decay, row_decay);
#pragma unroll 1
        for (int k = 0; k < 32; k += 16) {
          float y[16];
          uint32_t bits[16];
          uint4* at = reinterpret_cast<uint4*>(smem + Cf::oX + r * kTile + row_at + (((uint32_t)(4 * half + (k >> 3)) ^ rsw) << 4));
          uint4* at2 = reinterpret_cast<uint4*>(smem + Cf::oX + r * kTile + row_at + (((uint32_t)(4 * half + (k >> 3) + 1) ^ rsw) << 4));
          const uint4 xa = *at, xb = *at2;
          tc::tmem_ld16(ty + k, y);
          if (clear) *at = *at2 = make_uint4(0, 0, 0, 0);   // M X multiplies these rows by zeros: no NaN may be there
          const uint32_t xi[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            unpair(fma2(pair(y[2 * j], y[2 * j + 1]), f2, mul2(D2, pair(lo_f(xi[j]), hi_f(xi[j])))), y[2 * j], y[2 * j + 1]);
            bits[2 * j] = __float_as_uint(y[2 * j]);
            bits[2 * j + 1] = __float_as_uint(y[2 * j + 1]);
          }
          tmem_st16(ty + k, bits);
        }
        if (clear) fence_proxy_async_smem();
        tmem_wait_st();
        tc::fence_before_sync();
        arrive(kM);
        if (one) arrive_one(kEmptyX + r);
      }
    }
  } else if (warp < 2 * kSide / 32) {
    // ------------------------------------------------ state
    // the state before the segment: state n, columns p (the first tiles and decays are on their way)
    float h[32];
    {
      const bool from_ws = FULL && segs > 1;
      if (from_ws) wait_for_first();
      const float* src = nullptr;
      long long pitch = 0;
      bool mine = n < a.N;
      if (from_ws && seg == 0) {
        src = wsq + ((long long)(a.nseg - 1) * 64 + 32 * half) * NN;
        pitch = NN;
        mine = n < NN;
      } else if (!from_ws && a.state && seg == 0) {
        src = a.state + ((q.slot * a.H + head) * a.P + p0 + 32 * half) * a.N;
        pitch = a.N;
      }
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
          *reinterpret_cast<uint4*>(smem + Cf::oH + row_at + (((uint32_t)(4 * half + i) ^ rsw) << 4)) = v;
        }
      }
    };
    if (FULL) {
      put_state();
      fence_proxy_async_smem();
      arrive(kH);
    }
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColU + 32 * half;
    float log_total = 0.f;
    // h <- exp(c_L) h + U
    auto update = [&](float total) {
      const float d = ex2(total);
      const uint64_t d2 = pair(d, d);
      log_total += total;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < 32; k += 16) {
        float e[16], f[16];
        tc::tmem_ld16(tlane + k, e);        // B^T (t1 + t2 / 2)
        tc::tmem_ld16(tlane + 64 + k, f);   // B^T (t2 / 2 + t3)
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          unpair(fma2(d2, pair(h[k + j], h[k + j + 1]), add2(pair(e[j], e[j + 1]), pair(f[j], f[j + 1]))), h[k + j],
                 h[k + j + 1]);
      }
    };
    float total = 0.f;   // of the chunk whose U comes next
    for (int i = 0; i <= n_chunks; ++i) {
      const int r = i & 1, u = i >> 1;
      if (i > 0) {
        if (!wait(kFullU, i - 1)) break;
        update(total);
        if (i == n_chunks) break;
      }
      if (ragged && i == last_i) {   // rows of the next sequence: none of B's may reach the product
        if (!wait(kFullB + r, u)) break;
        if (half == 0 && (unsigned int)(i * kL + row) >= left)
          for (uint32_t k = 0; k < 8 * Cf::NT; ++k)
            *reinterpret_cast<uint4*>(smem + Cf::oB + (r * Cf::NT + (k >> 3)) * kTile + row_at + ((k & 7) << 4)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      if (!wait(kFullDec + i % kDec, i / kDec) || !wait(kFullX + r, u)) break;
#pragma unroll 1
      for (int piece = warp - kSide / 32; piece < (FULL ? kUnits : kUnits / 2); piece += kSide / 32) make_piece(i, piece);
      tc::fence_before_sync();
      arrive(kXt);
      total = vec[(i % kDec) * kVec + 5 * kL + 8];
      __syncwarp();
      if (one) {
        arrive_one(kEmptyX + r);
        if (FULL) arrive_one(kReadX + r);
        arrive_one(kEmptyDec + i % kDec);
      }
      // the copy of the state before this chunk, once the one before it has been read
      if (FULL && i > 0) {
        if (!wait(kFullYi + (r ^ 1), (i - 1) >> 1)) break;
        put_state();
        fence_proxy_async_smem();
        arrive(kH);
      }
    }
    if (*fail) {
      if (tid == kSide) atomicOr(&a.status->flags, kStatusTimeout);
    } else if (!FULL) {
      if (n < NN) {
        float* e = wsq + ((long long)seg * 64 + 32 * half) * NN;
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i * NN + n] = h[i];
        if (tid == kSide) wsq[(long long)a.nseg * 64 * NN + seg] = ex2(log_total);
      }
    } else if (last && a.state && n < a.N) {
      float* dst = a.state + ((q.slot * a.H + head) * a.P + p0 + 32 * half) * a.N + n;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < pc) dst[(long long)i * a.N] = h[i];
    }
  } else if (warp == 16) {
    if constexpr (FULL) {
      // ------------------------------------------------ C h^T, M X
      const uint64_t c0 = desc128(sbase + Cf::oC, 16), h0 = desc128(sbase + Cf::oH, 16);
      for (int i = 0; i < n_chunks; ++i) {
        const int r = i & 1, u = i >> 1;
        const uint32_t ty = tmem + kColY + 64 * r, ts = tmem + kColS + 128 * r;
        const uint64_t x0 = desc128(sbase + Cf::oX + r * kTile, 16);
        if (!wait(kFullC, i) || !wait(kH, i) || (u > 0 && !wait(kEmptyY + r, u - 1))) break;
        tc::fence_after_sync();
#pragma unroll 4
        for (int k = 0; k < NN / 16; ++k)
          mma_ss(ty, c0 + (k >> 2) * (kTile >> 4) + (k & 3) * 2, h0 + k * 128, kId | kN64 | kTransB, k > 0, one);
        if (one) {
          tc::mma_commit(bar + kFullYi + r);
          tc::mma_commit(bar + kEmptyC);
        }
        __syncwarp();
        if (!wait(kFullX + r, u)) break;
        const unsigned char* xt = smem + Cf::oX + r * kTile + 16 * lane;
        uint32_t zero = 0, zero2 = 0;   // NaN once a value is not finite
#pragma unroll 8
        for (uint32_t k = 0; k < 32; ++k) {
          const uint4 x = *reinterpret_cast<const uint4*>(xt + 512 * k);
          zero = times_zero(x.x, times_zero(x.y, zero));
          zero2 = times_zero(x.z, times_zero(x.w, zero2));
        }
        if (__any_sync(0xffffffffu, ((zero | zero2) & 0x7fff7fffu) != 0)) {
          if (!wait(kReadX + r, u)) break;
          uint32_t* word = odd + r * kOdd;
#pragma unroll 1
          for (uint32_t k = 0; k < 32; ++k) {
            const uint32_t token = 4 * k + (uint32_t)lane / 8;
            if (ragged && i == last_i && i * kL + token >= left) continue;   // the next sequence's
            take_out(smem + Cf::oX + r * kTile + 512 * k + 16 * lane, word + 8 * ((lane ^ token) & 7),
                     ((uint32_t)i + 1) * kL + (kL - 1 - token));
          }
          word[64] = (uint32_t)i + 1;
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!wait(kM, i)) break;
        tc::fence_after_sync();
#pragma unroll 4
        for (int k = 0; k < kL / 16; ++k)
          mma_ts(ty, ts + 64 * (k >> 2) + 8 * (k & 3), x0 + k * 128, kId | kN64 | kTransB, true, one);
        if (one) {
          tc::mma_commit(bar + kFullY + r);
          tc::mma_commit(bar + kEmptyS + r);
          tc::mma_commit(bar + kEmptyX + r);
        }
        __syncwarp();
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------ B^T X~, then S of the next chunk
    const uint64_t c0 = desc128(sbase + Cf::oC, 16), t0 = desc128(sbase + Cf::oT, kTile);
    for (int i = FULL ? -1 : 0; i < n_chunks; ++i) {   // turn -1 forms the first S
      if (i >= 0) {
        const int r = i & 1;
        const uint64_t b0 = desc128(sbase + Cf::oB + r * Cf::NT * kTile, kTile);
        if (!wait(kXt, i) || !wait(kFullB + r, i >> 1)) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass)
#pragma unroll 4
          for (int k = 0; k < kL / 16; ++k)
            mma_ss(tmem + kColU, b0 + k * 128, t0 + pass * (kTile >> 4) + k * 128, kId | kN128 | kTransA | kTransB,
                   pass > 0 || k > 0, one);
        if (one) {
          tc::mma_commit(bar + kFullU);
          tc::mma_commit(bar + kEmptyB + r);
        }
        __syncwarp();
      }
      if (!FULL || i == last_i) continue;
      const int r = (i + 1) & 1, u = (i + 1) >> 1;
      if (!wait(kFullB + r, u) || !wait(kFullC, i + 1) || (u > 0 && !wait(kEmptyS + r, u - 1))) break;
      tc::fence_after_sync();
      const uint64_t b0 = desc128(sbase + Cf::oB + r * Cf::NT * kTile, 16);
#pragma unroll 4
      for (int k = 0; k < NN / 16; ++k) {
        const uint32_t at = (k >> 2) * (kTile >> 4) + (k & 3) * 2;
        mma_ss(tmem + kColS + 128 * r, c0 + at, b0 + at, kId | kN128, k > 0, one);
      }
      if (one) {
        tc::mma_commit(bar + kFullS + r);
        tc::mma_commit(bar + kEmptyB + r);
        tc::mma_commit(bar + kEmptyC);
      }
      __syncwarp();
    }
  } else if (FULL && warp == 19) {
    // ------------------------------------------------ stores of y, and z of the next chunk into the same tile
    for (int i = 0; i <= n_chunks; ++i) {
      if (i > 0 && !wait(kStage, i - 1)) break;
      if (one) {
        const int t = row0 + t_first + i * kL;
        if (i > 0) {
          if (!(ragged && i - 1 == last_i)) store_4d(&map_y, p0, head, t - kL, batch, sbase + Cf::oY);
          store_read_done();
          arrive_one(kStaged);
        }
        if (GATE == 1 && i < n_chunks) {
          mbar_arrive_expect_tx(bar + kFullZ, kTile);
          load_4d(sbase + Cf::oY, &map_z, p0, head, t, batch, bar + kFullZ);
        }
      }
      __syncwarp();
    }
    if (one) store_done();
    if (GATE == 1 && *fail)   // nothing lands after the CTA has gone
      for (int j = 0; j < 2; ++j) mbar_wait_bounded(bar + kFullZ, (uint32_t)j, kWaitLimitNs / 8);
  } else if (warp == 18) {
    // ------------------------------------------------ loads: B, X, C of a chunk in turn
    const int kinds = FULL ? 3 : 2;
    int i = 0, kind = 0;
    while (i < n_chunks) {
      const int r = i & 1;
      // the place is free: its use before has been read (C has one place, the others two)
      const int empty = kind == 0 ? kEmptyB + r : kind == 1 ? kEmptyX + r : kEmptyC;
      const int use = kind == 2 ? i : i >> 1;
      if (use > 0 && !wait(empty, use - 1)) break;
      if (one) {
        const int t = row0 + t_first + i * kL;
        const CUtensorMap* map = kind == 0 ? &map_B : kind == 1 ? &map_x : &map_C;
        uint64_t* full = bar + (kind == 0 ? kFullB + r : kind == 1 ? kFullX + r : kFullC);
        const uint32_t to = sbase + (kind == 0 ? Cf::oB + r * Cf::NT * kTile : kind == 1 ? Cf::oX + r * kTile : Cf::oC);
        const uint32_t tiles = kind == 1 ? 1u : Cf::NT;
        mbar_arrive_expect_tx(full, tiles * kTile);
#pragma unroll 1
        for (uint32_t k = 0; k < tiles; ++k) {
          load_4d(to + k * kTile, map, kind == 1 ? p0 : 64 * (int)k, kind == 1 ? head : group, t, batch, full);
          // C is asked for late: its rows are fetched into L2 beside B's
          if (FULL && kind == 0) prefetch_4d(&map_C, 64 * (int)k, group, t, batch);
        }
      }
      __syncwarp();
      if (++kind == kinds) {
        kind = 0;
        ++i;
      }
    }
    if (*fail)   // nothing lands after the CTA has gone
#pragma unroll 1
      for (int k = 0; k < 10; ++k) mbar_wait_bounded(bar + kFullB + (k >> 1), (uint32_t)k & 1u, kWaitLimitNs / 8);
  } else if (warp >= 20) {
    // ------------------------------------------------ decays: tokens 32 j + lane of every chunk
    const int j = warp - 20;
    const __nv_bfloat16* dt = a.dt + (packed ? q.start * a.dt_tok : seq * a.dt_seq) + head;
    const float A2 = a.A[head] * 1.44269504088896341f, bias = a.dt_bias ? a.dt_bias[head] : 0.f;
    long long t = t_first + 32 * j + lane;
    float raw = t < q.len ? __bfloat162float(dt[t * a.dt_tok]) : 0.f;
#pragma unroll 1
    for (int i = 0; i < n_chunks; ++i) {
      const bool in = t < q.len;
      const float s = in ? time_step(raw, bias, a.softplus) : 0.f;
      t += kL;
      if (t < q.len && i < last_i) raw = __bfloat162float(dt[t * a.dt_tok]);
      const float own = in ? A2 * s : 0.f;
      float inc = own, ex = own;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const float up = __shfl_up_sync(0xffffffffu, inc, o), down = __shfl_down_sync(0xffffffffu, ex, o);
        if (lane >= o) inc += up;
        if (lane + o < 32) ex += down;
      }
      ex = __shfl_down_sync(0xffffffffu, ex, 1);
      if (lane == 31) ex = 0.f;
      const bool small = __all_sync(0xffffffffu, fabsf(inc) < 100.f && s < 1e8f);   // s exp(-inc) is finite
      float* v = vec + (i % kDec) * kVec;
      float* sums = v + 5 * kL;
      // the four warps leave together: each reads the others' sums
      const bool ok = i < kDec || wait(kEmptyDec + i % kDec, i / kDec - 1);
      if (lane == 31) sums[12 + j] = inc;
      if (named_or(1, 128, !ok)) break;
      float before = 0.f, behind = 0.f;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const float e = sums[12 + k];
        if (k < j) before += e;
        if (k > j) behind += e;
      }
      v += 32 * j + lane;
      v[0] = inc;
      v[kL] = s * ex2(ex);
      v[2 * kL] = small ? s * ex2(-inc) : own;
      v[3 * kL] = s * ex2(ex + behind);
      v[4 * kL] = s;
      if (lane == 31) {
        sums[j] = before;
        sums[16 + j] = small ? 1.f : 0.f;
        if (j == 3) sums[8] = before + inc;
      }
      arrive(kFullDec + i % kDec);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, kCols);
  if (FULL && a.nseg > 1) wait_for_first();   // the call ends after both
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
                   int gate, cudaStream_t st) {
  const long long cut = (s.seqs.n_seq * a.H * a.pslices - plan.whole) * plan.nseg;
  if (cut + plan.whole > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  constexpr int bytes = (int)Cfg<NN>::bytes;
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  auto run = [&](auto kern, std::atomic<unsigned long long>& ready, bool first) -> cudaError_t {
    // more than 48 KB of shared memory: allowed once a kernel and device (the first 64)
    if (device >= 64 || !(ready.load(std::memory_order_relaxed) >> device & 1)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      if (device < 64) ready.fetch_or(1ull << device, std::memory_order_relaxed);
    }
    if (!first && plan.nseg > 1)
      return launch_second(kern, (unsigned int)(plan.whole + cut), kThreads, bytes, st, maps[0], maps[1], maps[2], maps[3],
                           maps[4], a);
    // a sequence's last segment has no first launch
    kern<<<(unsigned int)(first ? cut / plan.nseg * (plan.nseg - 1) : plan.whole + cut), kThreads, bytes, st>>>(maps[0], maps[1], maps[2], maps[3],
                                                                                maps[4], a);
    return cudaGetLastError();
  };
  static std::atomic<unsigned long long> ready[4];
  if (plan.nseg > 1) {
    const cudaError_t e = run(ssm_prompt_kernel<NN, false, 0>, ready[0], true);
    if (e != cudaSuccess) return e;
  }
  switch (gate) {
    case 0: return run(ssm_prompt_kernel<NN, true, 0>, ready[1], false);
    case 1: return run(ssm_prompt_kernel<NN, true, 1>, ready[2], false);
    default: return run(ssm_prompt_kernel<NN, true, 2>, ready[3], false);
  }
}

}  // namespace

PromptPlan ssm_prompt_plan(long long n_seq, long long tokens, long long max_len, long long H, long long P, long long N,
                           bool bf16, int sm_count) {
  PromptPlan p{};
  p.fits = bf16 && P % 8 == 0 && N % 8 == 0 && N <= 128 && max_len > 8 && H < (1 << 20) && P < (1 << 20);
  if (!p.fits) return p;
  const long long slices = H * ((P + 63) / 64), chunks = (max_len + kL - 1) / kL, slots = sm_count;
  p.nn = N <= 64 ? 64 : 128;
  p.nseg = 1;
  p.seg_chunks = chunks;
  // One CTA an SM.  While the slices leave SMs idle, segments shorten the longest run of chunks.  In
  // microseconds, measured: a chunk 2.3, a chunk of the first launch 1.2, a CTA's start 4.5, and 0.7 for
  // each segment that a start joins.  (One sequence of 16384 tokens, 16 heads: 9 segments; 19, which
  // fill the SMs twice, take a third longer.)
  constexpr double kStart = 4.5;
  const auto waves = [&](long long k) { return (double)((n_seq * slices * k + slots - 1) / slots); };
  // Sequences of several lengths, of which the longest and the tokens of all are known: the work that there
  // is, a CTA without any costing kEmpty, and half of what the longest CTA takes (it may start last).
  // (3000 and 500 tokens, 32 heads: uncut 61 us, in 2 55, 3 44, 4 42, 6 52; 30 prompts of 100 and one of 4096, 16
  // heads: 107, 104, 94, 99, 112; nine of 1 to 2047, 16 heads of 128: 51, 60, 64, 73, 88.)
  constexpr double kEmpty = 2.0;
  const bool even = tokens >= n_seq * max_len;
  const auto uneven = [&](long long k, long long per) {
    const double n = (double)n_seq, segs = (double)tokens / (kL * per) - 0.5 * n;
    const double first = k == 1 ? 0.0 : std::max((double)(k - 1), std::min(n * (k - 1), segs)), second = n + first;
    const double work2 =
        slices * (2.3 * ((double)tokens / kL + 0.5 * n) + kStart * second + kEmpty * (n * k - second)) / slots;
    const double work1 = slices * (first * (1.2 * per + kStart) + kEmpty * (n * k - first)) / slots;
    const double longest = 2.3 * per + kStart + (k > 1 ? 0.7 * k : 0.0);
    return (second * slices <= slots ? longest : std::max(longest, work2 + 0.5 * longest)) +
           (k == 1 ? 0.0 : std::max(work1, 1.2 * per + kStart));
  };
  double best = even ? waves(1) * (2.3 * chunks + kStart) : uneven(1, chunks);
  for (long long k = 2; k <= chunks && k <= 64; ++k) {
    const long long per = (chunks + k - 1) / k;
    if ((chunks + per - 1) / per != k) continue;
    const double cost = even ? waves(k) * (3.5 * per + 2 * kStart + 0.7 * k) : uneven(k, per);
    if (cost < best) {
      best = cost;
      p.nseg = (int)k;
      p.seg_chunks = per;
      p.whole = 0;
    }
  }
  // Or, of sequences of one length, only what the last wave of CTAs would have.  The CTAs of its first
  // launch delay as many SMs; the last segments, which have no first launch, are the longer ones and go
  // to the other SMs.  (8 sequences of 4096 tokens, 64 heads: 56 of 512 are left for a fourth wave;
  // uncut 315 us, in 3 equal segments 297, in 2 of 12 and 20 chunks 290.  3 of 2048 tokens: 85, 78, 68.)
  const long long tail = n_seq * slices % slots, full = n_seq * slices / slots;
  for (long long k = 2; even && tail > 0 && full > 0 && k * tail <= slots && k <= chunks && k <= 16; ++k) {
    const long long rest = slots - (k - 1) * tail;
    const auto delay = [&](long long per) { return 1.2 * per + kStart; };
    const auto lasts = [&](long long per) {
      return 2.3 * (chunks - (k - 1) * per) + kStart + 0.7 * k + (tail > rest ? delay(per) : 0.0);
    };
    const auto others = [&](long long per) {
      return 2.3 * per + kStart + 0.7 * (k - 1) + (k * tail > rest ? delay(per) : 0.0);
    };
    long long lo = 1, hi = (chunks - 1) / (k - 1);   // the shortest segments that take as long as the last ones
    while (lo < hi) {
      const long long mid = (lo + hi) / 2;
      if (others(mid) >= lasts(mid)) hi = mid;
      else lo = mid + 1;
    }
    for (long long per = lo > 1 ? lo - 1 : lo; per <= lo; ++per) {
      const double cost = full * (2.3 * chunks + kStart) + std::max(lasts(per), others(per));
      if (cost < best) {
        best = cost;
        p.nseg = (int)k;
        p.seg_chunks = per;
        p.whole = n_seq * slices - tail;
      }
    }
  }
  // The token-by-token form takes, measured: a launch and the states' traffic, then 0.2 us a token or
  // what its arithmetic needs.  (8 sequences of 64 heads of 64, 128 states: 16 tokens 29 us against
  // 21.5 us here; one sequence: 24 tokens 8.8 against 9.8, 32 tokens about 10.3 against 8.3.)
  const double units = (double)(n_seq * slices) * (double)N / 128.0;
  const double steps = 2.9 + 0.025 * units +
                       std::max(0.2 * (double)max_len, 0.0017 * (double)tokens * (double)slices * (double)N / 128.0);
  p.fits = best + 2.5 < steps;
  if (!p.fits) return p;
  if (p.nseg > 1) p.ws_bytes = (size_t)(n_seq * slices - p.whole) * ws_floats(p.nseg, p.nn) * sizeof(float);
  return p;
}

cudaError_t launch_ssm_prompt(const SsmArgs& s, const PromptPlan& plan, cudaStream_t st, bool* used) {
  *used = false;
  const bool packed = s.seqs.offsets != nullptr;
  const long long tokens = s.seqs.T, batch = packed ? 1 : s.seqs.n_seq;
  CUtensorMap maps[5];
  if (!encode(&maps[0], s.x, s.P, s.H, tokens, batch, s.x_tok, s.x_seq) ||
      !encode(&maps[1], s.B, s.N, s.G, tokens, batch, s.B_tok, s.B_seq) ||
      !encode(&maps[2], s.C, s.N, s.G, tokens, batch, s.C_tok, s.C_seq) ||
      !encode(&maps[3], s.y, s.P, s.H, tokens, batch, s.y_tok, s.y_seq))
    return cudaSuccess;
  maps[4] = maps[3];
  const int gate = !s.z ? 0 : encode(&maps[4], s.z, s.P, s.H, tokens, batch, s.z_tok, s.z_seq) ? 1 : 2;
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
  a.whole = (int)plan.whole;
  a.dt_seq = s.dt_seq; a.dt_tok = s.dt_tok; a.z_seq = s.z_seq; a.z_tok = s.z_tok; a.y_seq = s.y_seq; a.y_tok = s.y_tok;
  a.softplus = s.softplus;
  a.status = s.status;
  *used = true;
  return plan.nn == 64 ? launch<64>(s, a, plan, maps, gate, st) : launch<128>(s, a, plan, maps, gate, st);
}

}  // namespace vla
