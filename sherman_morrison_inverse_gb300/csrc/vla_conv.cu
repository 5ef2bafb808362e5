// Short causal convolution, one filter of K taps a channel:
//   y[t, c] = act(b[c] + sum_j w[c, j] x[t - K + 1 + j, c]),   act = identity or x * sigmoid(x),
// where inputs before the sequence's first token come from its state [K - 1, C] (zeros without one),
// and the state becomes the last K - 1 inputs.
//
// Every value is read and written once (2 sizeof(io) bytes a value against 2 K + 4 operations), so
// the kernel streams: a thread owns VEC adjacent channels and `tile` consecutive tokens, keeps the
// K - 1 previous inputs in registers and has kBatch rows in flight; only the K - 1 rows before a
// tile are read twice (from L2).  What it costs beyond memory is instructions: channels are taken
// in pairs with packed float32 arithmetic, and an access is 8 bytes rather than 16, because a thread
// then needs 64 registers and twice the threads fit (102 -> 98 us).
// 8 x 4096 tokens of 4352 channels, K = 4, bfloat16, SiLU: 98.4 us, 5.80 TB/s, 86 % of a plain copy's
// rate; what is left are waits for memory.  192 single tokens: 6.7 us on the GPU (2 us of memory).
// The thread of a sequence's first tile is the only one that touches the state: it has read the
// old one before it writes the new one.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;    // rows loaded before the first is used

// The rows of VEC channels as float32, in pairs where VEC is even.
template <typename T, int VEC>
struct Row {
  static constexpr int PAIRS = (VEC + 1) / 2;
  uint64_t p[PAIRS];
  __device__ void set(const Vec<T, VEC>& r) {
    if constexpr (VEC == 1) {
      p[0] = pair(to_f32<T>(r.v[0]), 0.f);
    } else if constexpr (sizeof(T) == 2) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.raw);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) p[i] = pair(lo_f(w[i]), hi_f(w[i]));
    } else {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) p[i] = pair(to_f32<T>(r.v[2 * i]), to_f32<T>(r.v[2 * i + 1]));
    }
  }
};

template <typename T, int K, int VEC>
__global__ void __launch_bounds__(kThreads, VEC <= 4 ? 8 : 4)
    short_conv_kernel(const ConvArgs a, int tiles, int cblocks, int tile_len, bool w_vec) {
  using R = Row<T, VEC>;
  constexpr int PAIRS = R::PAIRS;
  const int cb = (int)(blockIdx.x % cblocks);
  const long long rest = blockIdx.x / cblocks;
  const int tile = (int)(rest % tiles);
  const long long s = rest / tiles;
  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, s, &bad);
  if (bad && threadIdx.x == 0) atomicOr(&a.status->flags, bad);
  const long long c = ((long long)cb * kThreads + threadIdx.x) * VEC;
  const long long t0 = (long long)tile * tile_len;
  if (!q.run || c >= a.C || t0 >= q.len) return;

  const T* x = static_cast<const T*>(a.x) + (a.seqs.offsets ? q.start * a.x_tok : s * a.x_seq) + c;
  T* y = static_cast<T*>(a.y) + (a.seqs.offsets ? q.start * a.y_tok : s * a.y_seq) + c;
  T* state = a.state ? static_cast<T*>(a.state) + q.slot * (K - 1) * a.C + c : nullptr;

  // the VEC filters, one after another in memory: as VEC values an access where aligned (a call for
  // single tokens reads little else)
  float f[VEC * K], fb[VEC];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    if (w_vec) {
      const Vec<float, VEC> v = ld_vec<float, VEC>(a.w + c * K + i * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i * VEC + j] = v.v[j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i * VEC + j] = a.w[c * K + i * VEC + j];
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) fb[j] = 0.f;
  if (a.bias && w_vec) {
    const Vec<float, VEC> v = ld_vec<float, VEC>(a.bias + c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) fb[j] = v.v[j];
  } else if (a.bias) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) fb[j] = a.bias[c + j];
  }
  uint64_t w[K][PAIRS], b[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const int second = VEC == 1 ? 0 : 1;
    b[i] = pair(fb[2 * i], fb[2 * i + second]);
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = pair(f[2 * i * K + j], f[(2 * i + second) * K + j]);
  }
  // the K - 1 inputs before the tile; row i is input t0 - (K - 1) + i
  R h[K - 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const long long t = t0 - (K - 1) + i;
    Vec<T, VEC> old;
    if (t >= 0) old = ld_vec<T, VEC>(x + t * a.x_tok);
    else if (state) old = ld_vec<T, VEC>(state + (t + K - 1) * a.C);
    else
      for (int v = 0; v < VEC; ++v) old.v[v] = from_f32<T>(0.f);
    h[i].set(old);
  }
  if (tile == 0 && state) {
    // Row i keeps input len - (K - 1) + i; a sequence shorter than K - 1 keeps old rows too, moved
    // up (row i + len is read before row i is written, and later rows are not written yet).
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const long long t = q.len - (K - 1) + i;
      st_vec<T, VEC>(state + i * a.C, ld_vec<T, VEC>(t >= 0 ? x + t * a.x_tok : state + (t + K - 1) * a.C));
    }
  }
  const int n = (int)(q.len - t0 < tile_len ? q.len - t0 : tile_len);
  x += t0 * a.x_tok;
  y += t0 * a.y_tok;
  auto step = [&](const Vec<T, VEC>& in, T* dst) {
    R now;
    now.set(in);
    Vec<T, VEC> out;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      uint64_t r = fma2(w[K - 1][i], now.p[i], b[i]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) r = fma2(w[j][i], h[j].p[i], r);
#pragma unroll
      for (int j = 0; j + 1 < K - 1; ++j) h[j].p[i] = h[j + 1].p[i];
      h[K - 2].p[i] = now.p[i];
      float u, v;
      if (a.silu) {
        if constexpr (sizeof(T) == 2) {
          unpair(silu2(r), u, v);
        } else {
          unpair(r, u, v);
          u = silu<false>(u);
          if (VEC > 1) v = silu<false>(v);
        }
      } else {
        unpair(r, u, v);
      }
      if constexpr (VEC == 1) {
        out.v[0] = from_f32<T>(u);
      } else if constexpr (sizeof(T) == 2) {
        reinterpret_cast<uint32_t*>(&out.raw)[i] = pack2(u, v);
      } else {
        out.v[2 * i] = from_f32<T>(u);
        out.v[2 * i + 1] = from_f32<T>(v);
      }
    }
    st_vec<T, VEC>(dst, out);
  };
  int i0 = 0;
  for (; i0 + kBatch <= n; i0 += kBatch) {
    Vec<T, VEC> in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) in[i] = ld_vec<T, VEC>(x + i * a.x_tok);
    x += kBatch * a.x_tok;
#pragma unroll
    for (int i = 0; i < kBatch; ++i, y += a.y_tok) step(in[i], y);
  }
#pragma unroll 1
  for (; i0 < n; ++i0, x += a.x_tok, y += a.y_tok) step(ld_vec<T, VEC>(x), y);
}

// Tokens a thread: 64 where that still gives every SM 8 blocks, fewer for short or few sequences, down to
// kBatch.
template <typename T, int K, int VEC>
cudaError_t launch(const ConvArgs& a, cudaStream_t s) {
  const long long cblocks = (a.C + (long long)kThreads * VEC - 1) / ((long long)kThreads * VEC);
  long long tile = 64;
  while (tile > kBatch && (a.seqs.T + tile - 1) / tile * (a.seqs.offsets ? 1 : a.seqs.n_seq) * cblocks < 8LL * a.sm_count) tile /= 2;
  const long long tiles = (a.seqs.max_len + tile - 1) / tile;
  if (tiles > 0x7fffffffLL || cblocks > 0x7fffffffLL || tiles * cblocks > 0x7fffffffLL / a.seqs.n_seq)
    return cudaErrorInvalidConfiguration;
  const long long ctas = tiles * cblocks * a.seqs.n_seq;
  const bool w_vec = (reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.bias)) % (4 * VEC) == 0;
  short_conv_kernel<T, K, VEC><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (int)tiles, (int)cblocks, (int)tile, w_vec);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t by_taps(const ConvArgs& a, cudaStream_t s) {
  switch (a.K) {
    case 2: return launch<T, 2, VEC>(a, s);
    case 3: return launch<T, 3, VEC>(a, s);
    default: return launch<T, 4, VEC>(a, s);
  }
}

// Whether every row of x, y and the state starts on a `bytes` boundary and holds whole vectors.
bool vectors(const ConvArgs& a, size_t item, size_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                      reinterpret_cast<uintptr_t>(a.state);
  const unsigned long long strides =
      (unsigned long long)(a.x_seq | a.x_tok | a.y_seq | a.y_tok | a.C) * item;
  return (p | strides) % bytes == 0;
}

}  // namespace

cudaError_t launch_short_conv(const ConvArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) {
    if (vectors(a, 2, 8)) return by_taps<__nv_bfloat16, 4>(a, s);
    if (vectors(a, 2, 4)) return by_taps<__nv_bfloat16, 2>(a, s);
    return by_taps<__nv_bfloat16, 1>(a, s);
  }
  if (vectors(a, 4, 8)) return by_taps<float, 2>(a, s);
  return by_taps<float, 1>(a, s);
}

}  // namespace vla
