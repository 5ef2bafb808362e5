// Selective state space scan, token by token (the decay is one number a head):
//   s_t = softplus(dt_t + bias),  h_t = exp(A s_t) h_{t-1} + s_t x_t B_t^T,
//   y_t = (h_t C_t + D x_t) * silu(z_t),   h in R^{P x N}, B_t, C_t in R^N shared by H / G heads.
//
// Rows of h never meet, so a CTA takes ROWS = 32 R of the P rows of one (sequence, head) and keeps
// them in registers for the whole call: 8 lanes a row, lane j holding the states 32 i + 4 j .. + 3
// (i < NI), so that a row of the state moves as 128-byte pieces.  This is the form for what the
// single-token form (vla_ssm_token.cu) and the tensor-core form (vla_ssm_prompt.cu) do not take:
// float32 input and output, short prompts, odd sizes and alignments.  On long prompts it is bound
// by the 3 float32 operations a state element and token.
// Everything is float32 and every sum has a fixed order: the same bits every time.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 16;   // tokens staged in shared memory at a time

template <typename T, int NI, int R>
__global__ void __launch_bounds__(kThreads) ssm_steps_kernel(const SsmArgs a, int row_blocks) {
  constexpr int ROWS = 32 * R;
  constexpr int NP = 32 * NI;   // N rounded up
  __shared__ __align__(16) float sB[kTok][NP];
  __shared__ __align__(16) float sC[kTok][NP];
  __shared__ float sx[kTok][ROWS];
  __shared__ float sy[kTok][ROWS];
  __shared__ float sdec[kTok], sdt[kTok];

  const int rb = (int)(blockIdx.x % row_blocks);
  const long long rest = blockIdx.x / row_blocks;
  const long long head = rest % a.H, s = rest / a.H;
  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, s, &bad);
  if (bad && threadIdx.x == 0) atomicOr(&a.status->flags, bad);
  if (!q.run || q.len <= 0) return;

  const bool packed = a.seqs.offsets != nullptr;
  const long long g = head / (a.H / a.G);
  const T* x = static_cast<const T*>(a.x) + (packed ? q.start * a.x_tok : s * a.x_seq) + head * a.P;
  const T* dt = static_cast<const T*>(a.dt) + (packed ? q.start * a.dt_tok : s * a.dt_seq) + head;
  const T* B = static_cast<const T*>(a.B) + (packed ? q.start * a.B_tok : s * a.B_seq) + g * a.N;
  const T* C = static_cast<const T*>(a.C) + (packed ? q.start * a.C_tok : s * a.C_seq) + g * a.N;
  const T* z = a.z ? static_cast<const T*>(a.z) + (packed ? q.start * a.z_tok : s * a.z_seq) + head * a.P : nullptr;
  T* y = static_cast<T*>(a.y) + (packed ? q.start * a.y_tok : s * a.y_seq) + head * a.P;
  const float A = a.A[head], D = a.D ? a.D[head] : 0.f, bias = a.dt_bias ? a.dt_bias[head] : 0.f;

  const int tid = threadIdx.x, lane = tid & 7, grp = tid >> 3;   // grp: row within 32
  const long long p0 = (long long)rb * ROWS;
  const int N = (int)a.N;
  const bool vec = (N & 3) == 0;   // rows of the state are then 16-byte aligned (its base is)

  float h[R][NI][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long p = p0 + 32 * r + grp;
    const float* src = a.state ? a.state + ((q.slot * a.H + head) * a.P + p) * N : nullptr;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 32 * i + 4 * lane;
      if (src && p < a.P && vec && n < N) {
        const float4 v = *reinterpret_cast<const float4*>(src + n);
        h[r][i][0] = v.x; h[r][i][1] = v.y; h[r][i][2] = v.z; h[r][i][3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[r][i][j] = src && p < a.P && n + j < N ? src[n + j] : 0.f;
      }
    }
  }
  for (long long t0 = 0; t0 < q.len; t0 += kTok) {
    const int n_tok = (int)(q.len - t0 < kTok ? q.len - t0 : kTok);
    if (t0 > 0) __syncthreads();   // the previous tokens' y has been written out
    for (int e = tid; e < n_tok * NP; e += kThreads) {
      const int t = e / NP, n = e - t * NP;
      sB[t][n] = n < N ? to_f32<T>(B[(t0 + t) * a.B_tok + n]) : 0.f;
      sC[t][n] = n < N ? to_f32<T>(C[(t0 + t) * a.C_tok + n]) : 0.f;
    }
    for (int e = tid; e < n_tok * ROWS; e += kThreads) {
      const int t = e / ROWS, p = e - t * ROWS;
      sx[t][p] = p0 + p < a.P ? to_f32<T>(x[(t0 + t) * a.x_tok + p0 + p]) : 0.f;
    }
    if (tid < n_tok) {
      const float step = time_step(to_f32<T>(dt[(t0 + tid) * a.dt_tok]), bias, a.softplus);
      sdt[tid] = step;
      sdec[tid] = expf(A * step);
    }
    __syncthreads();
    for (int t = 0; t < n_tok; ++t) {
      const float dec = sdec[t], step = sdt[t];
      float acc[R], in[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r] = 0.f;
        in[r] = step * sx[t][32 * r + grp];
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float4 b = *reinterpret_cast<const float4*>(&sB[t][32 * i + 4 * lane]);
        const float4 c = *reinterpret_cast<const float4*>(&sC[t][32 * i + 4 * lane]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          h[r][i][0] = fmaf(dec, h[r][i][0], in[r] * b.x);
          h[r][i][1] = fmaf(dec, h[r][i][1], in[r] * b.y);
          h[r][i][2] = fmaf(dec, h[r][i][2], in[r] * b.z);
          h[r][i][3] = fmaf(dec, h[r][i][3], in[r] * b.w);
          acc[r] = fmaf(h[r][i][0], c.x, acc[r]);
          acc[r] = fmaf(h[r][i][1], c.y, acc[r]);
          acc[r] = fmaf(h[r][i][2], c.z, acc[r]);
          acc[r] = fmaf(h[r][i][3], c.w, acc[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        if (lane == 0) sy[t][32 * r + grp] = acc[r];
      }
    }
    __syncthreads();
    for (int e = tid; e < n_tok * ROWS; e += kThreads) {
      const int t = e / ROWS, p = e - t * ROWS;
      if (p0 + p >= a.P) continue;
      float v = fmaf(D, sx[t][p], sy[t][p]);
      if (z) v *= silu<sizeof(T) == 2>(to_f32<T>(z[(t0 + t) * a.z_tok + p0 + p]));
      y[(t0 + t) * a.y_tok + p0 + p] = from_f32<T>(v);
    }
  }
  if (!a.state) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long p = p0 + 32 * r + grp;
    if (p >= a.P) continue;
    float* dst = a.state + ((q.slot * a.H + head) * a.P + p) * N;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 32 * i + 4 * lane;
      if (vec && n < N) {
        *reinterpret_cast<float4*>(dst + n) = make_float4(h[r][i][0], h[r][i][1], h[r][i][2], h[r][i][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) dst[n + j] = h[r][i][j];
      }
    }
  }
}

template <typename T, int NI, int R>
cudaError_t launch(const SsmArgs& a, cudaStream_t s) {
  const long long blocks = (a.P + 32 * R - 1) / (32 * R);
  const long long ctas = blocks * a.H * a.seqs.n_seq;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  ssm_steps_kernel<T, NI, R><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (int)blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const SsmArgs& a, cudaStream_t s) {
  if (a.N <= 32) return launch<T, 1, 1>(a, s);
  if (a.N <= 64) return launch<T, 2, 1>(a, s);
  if (a.N <= 128) return launch<T, 4, 1>(a, s);
  return launch<T, 8, 1>(a, s);
}

}  // namespace

cudaError_t launch_ssm_steps(const SsmArgs& a, bool bf16, int sm_count, cudaStream_t s) {
  (void)sm_count;
  return bf16 ? by_states<__nv_bfloat16>(a, s) : by_states<float>(a, s);
}

}  // namespace vla
