// Short causal convolution, one filter of K taps a channel:
//   y[t, c] = act(b[c] + sum_j w[c, j] x[t - K + 1 + j, c]),   act = identity or x * sigmoid(x),
// where inputs before the sequence's first token come from its state [K - 1, C] (zeros without one),
// and the state becomes the last K - 1 inputs.
//
// Every value is read and written once (2 sizeof(io) bytes a value against 2 K + 4 operations), so
// the kernel streams: a thread owns VEC adjacent channels (16 bytes where alignment allows) and
// kTile consecutive tokens, keeps the K - 1 previous inputs in registers and has kBatch rows in
// flight; only the K - 1 rows before a tile are read twice (K - 1 of kTile, from L2).  The thread
// of a sequence's first tile is the only one that touches the state: it has read the old one
// before it writes the new one.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;    // tokens a thread
constexpr int kBatch = 8;    // rows loaded before the first is used

template <typename T, int K, int VEC>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const ConvArgs a, int tiles, int cblocks) {
  const int cb = (int)(blockIdx.x % cblocks);
  const long long rest = blockIdx.x / cblocks;
  const int tile = (int)(rest % tiles);
  const long long s = rest / tiles;
  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, s, &bad);
  if (bad && threadIdx.x == 0) atomicOr(&a.status->flags, bad);
  const long long c = ((long long)cb * kThreads + threadIdx.x) * VEC;
  const long long t0 = (long long)tile * kTile;
  if (!q.run || c >= a.C || t0 >= q.len) return;

  const T* x = static_cast<const T*>(a.x) + (a.seqs.offsets ? q.start * a.x_tok : s * a.x_seq) + c;
  T* y = static_cast<T*>(a.y) + (a.seqs.offsets ? q.start * a.y_tok : s * a.y_seq) + c;
  T* state = a.state ? static_cast<T*>(a.state) + q.slot * (K - 1) * a.C + c : nullptr;

  float w[VEC][K], b[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    b[v] = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[v][j] = a.w[(c + v) * K + j];
  }
  // the K - 1 inputs before the tile; row i is input t0 - (K - 1) + i
  float h[K - 1][VEC];
  Vec<T, VEC> old[K - 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const long long t = t0 - (K - 1) + i;
    if (t >= 0) old[i] = ld_vec<T, VEC>(x + t * a.x_tok);
    else if (state) old[i] = ld_vec<T, VEC>(state + (t + K - 1) * a.C);
    else
      for (int v = 0; v < VEC; ++v) old[i].v[v] = from_f32<T>(0.f);
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[i][v] = to_f32<T>(old[i].v[v]);
  }
  const int n = (int)(q.len - t0 < kTile ? q.len - t0 : kTile);
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    Vec<T, VEC> in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) in[i] = ld_vec<T, VEC>(x + (t0 + i0 + i) * a.x_tok);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= n) break;
      Vec<T, VEC> out;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float now = to_f32<T>(in[i].v[v]);
        float r = b[v];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) r = fmaf(w[v][j], h[j][v], r);
        r = fmaf(w[v][K - 1], now, r);
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) h[j][v] = h[j + 1][v];
        h[K - 2][v] = now;
        out.v[v] = from_f32<T>(a.silu ? silu<sizeof(T) == 2>(r) : r);
      }
      st_vec<T, VEC>(y + (t0 + i0 + i) * a.y_tok, out);
    }
  }
  if (tile == 0 && state) {
    // row i keeps input len - (K - 1) + i; a sequence shorter than K - 1 keeps old ones too
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const long long t = q.len - (K - 1) + i;
      Vec<T, VEC> keep;
      if (t >= 0) {
        keep = ld_vec<T, VEC>(x + t * a.x_tok);
      } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          if (j == (int)t + K - 1) keep = old[j];
      }
      st_vec<T, VEC>(state + i * a.C, keep);
    }
  }
}

template <typename T, int K, int VEC>
cudaError_t launch(const ConvArgs& a, cudaStream_t s) {
  const long long tiles = (a.seqs.max_len + kTile - 1) / kTile;
  const long long cblocks = (a.C + (long long)kThreads * VEC - 1) / ((long long)kThreads * VEC);
  const long long ctas = tiles * cblocks * a.seqs.n_seq;
  if (tiles > 0x7fffffffLL || cblocks > 0x7fffffffLL || ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  short_conv_kernel<T, K, VEC><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (int)tiles, (int)cblocks);
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
    if (vectors(a, 2, 16)) return by_taps<__nv_bfloat16, 8>(a, s);
    if (vectors(a, 2, 4)) return by_taps<__nv_bfloat16, 2>(a, s);
    return by_taps<__nv_bfloat16, 1>(a, s);
  }
  if (vectors(a, 4, 16)) return by_taps<float, 4>(a, s);
  return by_taps<float, 1>(a, s);
}

}  // namespace vla
