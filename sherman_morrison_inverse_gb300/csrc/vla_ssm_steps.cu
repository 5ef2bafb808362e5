// Selective state space scan, token by token (the decay is one number a head):
//   s_t = softplus(dt_t + bias),  h_t = exp(A s_t) h_{t-1} + s_t x_t B_t^T,
//   y_t = (h_t C_t + D x_t) * silu(z_t),   h in R^{P x N}, B_t, C_t in R^N shared by H / G heads.
//
// Rows of h never meet, so a CTA takes ROWS = 32 R of the P rows of one (sequence, head) and keeps
// them in registers: 8 lanes a row, lane j holding the states 32 i + 4 j .. + 3 (i < NI), so that a
// row of the state moves as 128-byte pieces.  This is the form for what the single-token form
// (vla_ssm_token.cu) and the tensor-core form (vla_ssm_prompt.cu) do not take: float32 input and
// output, short prompts, odd sizes and alignments.
//
// The recurrence itself is one fused multiply-add a token deep; what would make a token slow is
// everything around it.  So 16 tokens are staged in shared memory at a time, the next 16 are on their
// way in registers meanwhile, and the sums over N of 8 tokens are folded together: each step of the
// butterfly halves the tokens a lane carries, 7 shuffles for 8 tokens.  With many heads the kernel
// is bound by its 3 float32 operations a state element and token (in packed pairs).
//
// Few CTAs and a long sequence: it is cut into segments, one CTA each.  A first launch forms what
// every segment but a sequence's last adds to the state, the second starts each segment from those,
// joined in a fixed order.  Everything is float32 and every sum has a fixed order: the same bits
// every time.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 16;   // tokens staged in shared memory at a time
constexpr int kFold = 8;   // tokens whose sums are folded together
constexpr long long kSegMin = 192;   // shorter sequences are not cut (32 heads of 64 x 64: 128 tokens 19.0 us whole and
                                     // 18.5 cut, 192 tokens 27 and 26, 512 tokens 67 and 44)

// Floats of one (sequence, head, row block) in the workspace: nseg states of `per` floats (the last
// segment's place holds the state before the sequence), then the segments' decays; whole 16 bytes.
__host__ __device__ constexpr long long ws_floats(int nseg, int per) { return (long long)nseg * per + (nseg + 3) / 4 * 4; }

// FULL: outputs and the final state; else what the segment adds to the state.
template <typename T, int NI, int R, bool FULL>
__global__ void __launch_bounds__(kThreads) ssm_steps_kernel(const SsmArgs a, int row_blocks, int nseg, long long seg_len) {
  constexpr int ROWS = 32 * R;
  constexpr int NP = 32 * NI;   // N rounded up
  constexpr int EB = kTok * NP / kThreads, EX = kTok * ROWS / kThreads;   // staged values a thread
  __shared__ __align__(16) float sB[kTok][NP];
  __shared__ __align__(16) float sC[FULL ? kTok : 1][NP];
  __shared__ float sx[kTok][ROWS];
  __shared__ float sy[FULL ? kTok : 1][ROWS + 4];
  __shared__ float sdec[kTok], sdt[kTok];

  const int rb = (int)(blockIdx.x % row_blocks);
  long long rest = blockIdx.x / row_blocks;
  const long long head = rest % a.H;
  rest /= a.H;
  const int seg = (int)(rest % nseg);
  const long long s = rest / nseg;
  unsigned int bad = 0;
  const SeqRange q = seq_range(a.seqs, s, &bad);
  if (bad && threadIdx.x == 0 && FULL) atomicOr(&a.status->flags, bad);
  const long long t_begin = seg * seg_len;
  const long long t_end = t_begin + seg_len < q.len ? t_begin + seg_len : q.len;
  const bool last = t_end == q.len;
  if (!q.run || t_begin >= q.len || (!FULL && last)) return;

  const bool packed = a.seqs.offsets != nullptr;
  const long long g = head / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid & 7, grp = tid >> 3;   // grp: row within 32
  const long long p0 = (long long)rb * ROWS;
  const int N = (int)a.N;
  const T* x = static_cast<const T*>(a.x) + (packed ? q.start * a.x_tok : s * a.x_seq) + head * a.P + p0;
  const T* dt = static_cast<const T*>(a.dt) + (packed ? q.start * a.dt_tok : s * a.dt_seq) + head;
  const T* B = static_cast<const T*>(a.B) + (packed ? q.start * a.B_tok : s * a.B_seq) + g * a.N;
  const T* C = static_cast<const T*>(a.C) + (packed ? q.start * a.C_tok : s * a.C_seq) + g * a.N;
  const T* z = a.z ? static_cast<const T*>(a.z) + (packed ? q.start * a.z_tok : s * a.z_seq) + head * a.P + p0 : nullptr;
  T* y = static_cast<T*>(a.y) + (packed ? q.start * a.y_tok : s * a.y_seq) + head * a.P + p0;
  const float A = a.A[head], D = a.D ? a.D[head] : 0.f, bias = a.dt_bias ? a.dt_bias[head] : 0.f;
  const int rows = (int)(a.P - p0 < ROWS ? a.P - p0 : ROWS);

  constexpr int PER = R * NI * 4 * kThreads;
  float* ws = nseg > 1 ? a.ws + ((s * a.H + head) * row_blocks + rb) * ws_floats(nseg, PER) : nullptr;
  const bool from_ws = FULL && q.len > seg_len;

  uint64_t h[R][NI][2];   // pairs of states
  const bool vec = (N & 3) == 0;   // rows of the state are then 16-byte aligned (its base is)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = 32 * r + grp;
    const float* src = a.state && seg == 0 && !from_ws ? a.state + ((q.slot * a.H + head) * a.P + p0 + p) * N : nullptr;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 32 * i + 4 * lane;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (src && p < rows && vec && n < N) {
        v = *reinterpret_cast<const float4*>(src + n);
      } else if (src && p < rows) {
        if (n < N) v.x = src[n];
        if (n + 1 < N) v.y = src[n + 1];
        if (n + 2 < N) v.z = src[n + 2];
        if (n + 3 < N) v.w = src[n + 3];
      }
      h[r][i][0] = pair(v.x, v.y);
      h[r][i][1] = pair(v.z, v.w);
    }
  }
  auto ws_at = [&](int j, int r, int i) {   // 4 values of this thread in segment j's state
    return reinterpret_cast<float4*>(ws + (long long)j * PER) + (r * NI + i) * kThreads + tid;
  };
  if (!FULL && seg == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float4 v;
        unpair(h[r][i][0], v.x, v.y);
        unpair(h[r][i][1], v.z, v.w);
        *ws_at(nseg - 1, r, i) = v;
      }
  }
  if (from_ws) {
    const float* dec = ws + (long long)nseg * PER;
    for (int j = 0; j < (seg == 0 ? 1 : seg); ++j) {
      // segment 0 starts from the state before the sequence; its result holds that state's rest
      const float d = j == 0 ? 0.f : dec[j];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 e = *ws_at(seg == 0 ? nseg - 1 : j, r, i);
          h[r][i][0] = fma2(pair(d, d), h[r][i][0], pair(e.x, e.y));
          h[r][i][1] = fma2(pair(d, d), h[r][i][1], pair(e.z, e.w));
        }
    }
  }

  // the next tokens, on their way
  T nB[EB], nC[FULL ? EB : 1], nx[EX], nz[FULL ? EX : 1];
  float ndt = 0.f;
  const T none = from_f32<T>(0.f);
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int k = 0; k < EB; ++k) {
      const int e = k * kThreads + tid, t = e / NP, n = e - t * NP;
      const bool in = t0 + t < t_end && n < N;
      nB[k] = in ? B[(t0 + t) * a.B_tok + n] : none;
      if (FULL) nC[k] = in ? C[(t0 + t) * a.C_tok + n] : none;
    }
#pragma unroll
    for (int k = 0; k < EX; ++k) {
      const int e = k * kThreads + tid, t = e / ROWS, p = e - t * ROWS;
      const bool in = t0 + t < t_end && p < rows;
      nx[k] = in ? x[(t0 + t) * a.x_tok + p] : none;
      if (FULL) nz[k] = in && z ? z[(t0 + t) * a.z_tok + p] : none;
    }
    if (tid < kTok && t0 + tid < t_end) ndt = to_f32<T>(dt[(t0 + tid) * a.dt_tok]);
  };
  fetch(t_begin);
  float log_total = 0.f;
  for (long long t0 = t_begin; t0 < t_end; t0 += kTok) {
    const int n_tok = (int)(t_end - t0 < kTok ? t_end - t0 : kTok);
    T zz[FULL ? EX : 1];
#pragma unroll
    for (int k = 0; k < EB; ++k) {
      const int e = k * kThreads + tid;
      (&sB[0][0])[e] = to_f32<T>(nB[k]);
      if (FULL) (&sC[0][0])[e] = to_f32<T>(nC[k]);
    }
#pragma unroll
    for (int k = 0; k < EX; ++k) {
      (&sx[0][0])[k * kThreads + tid] = to_f32<T>(nx[k]);
      if (FULL) zz[k] = nz[k];
    }
    if (tid < kTok) {   // a token behind the end leaves the state as it is
      const float step = tid < n_tok ? time_step(ndt, bias, a.softplus) : 0.f;
      sdt[tid] = step;
      sdec[tid] = tid < n_tok ? expf(A * step) : 1.f;
      if (!FULL) log_total += tid < n_tok ? A * step : 0.f;
    }
    __syncthreads();
    if (t0 + kTok < t_end) fetch(t0 + kTok);
    for (int tb = 0; tb < n_tok; tb += kFold) {
      float acc[R][kFold];
#pragma unroll
      for (int j = 0; j < kFold; ++j) {
        const int t = tb + j;
        const float dec = sdec[t], step = sdt[t];
        const uint64_t dec2 = pair(dec, dec);
        uint64_t in2[R], sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float in = step * sx[t][32 * r + grp];
          in2[r] = pair(in, in);
          sum[r] = 0;   // two zeros
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(&sB[t][32 * i + 4 * lane]);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            h[r][i][0] = fma2(dec2, h[r][i][0], mul2(in2[r], pair(b.x, b.y)));
            h[r][i][1] = fma2(dec2, h[r][i][1], mul2(in2[r], pair(b.z, b.w)));
          }
          if (FULL) {
            const float4 c = *reinterpret_cast<const float4*>(&sC[t][32 * i + 4 * lane]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              sum[r] = fma2(h[r][i][0], pair(c.x, c.y), sum[r]);
              sum[r] = fma2(h[r][i][1], pair(c.z, c.w), sum[r]);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float e, f;
          unpair(sum[r], e, f);
          acc[r][j] = e + f;
        }
      }
      if constexpr (FULL) {
        // lane bits 4, 2, 1 choose the half of the tokens a lane keeps: token tb + lane is left
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int j = 0; j < o; ++j) {
              const float keep = up ? acc[r][j + o] : acc[r][j], send = up ? acc[r][j] : acc[r][j + o];
              acc[r][j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          }
          sy[tb + lane][32 * r + grp] = acc[r][0];
        }
      }
    }
    __syncthreads();
    if (FULL) {
#pragma unroll
      for (int k = 0; k < EX; ++k) {
        const int e = k * kThreads + tid, t = e / ROWS, p = e - t * ROWS;
        if (t >= n_tok || p >= rows) continue;
        float v = fmaf(D, sx[t][p], sy[t][p]);
        if (z) v *= silu<sizeof(T) == 2>(to_f32<T>(zz[k]));
        y[(t0 + t) * a.y_tok + p] = from_f32<T>(v);
      }
      __syncthreads();   // the staged tokens may be replaced
    }
  }
  if (!FULL) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float4 v;
        unpair(h[r][i][0], v.x, v.y);
        unpair(h[r][i][1], v.z, v.w);
        *ws_at(seg, r, i) = v;
      }
    if (tid < 32) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) log_total += __shfl_xor_sync(0xffffffffu, log_total, o);
      if (tid == 0) ws[(long long)nseg * PER + seg] = expf(log_total);
    }
    return;
  }
  if (!a.state || !last) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = 32 * r + grp;
    if (p >= rows) continue;
    float* dst = a.state + ((q.slot * a.H + head) * a.P + p0 + p) * N;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 32 * i + 4 * lane;
      float4 v;
      unpair(h[r][i][0], v.x, v.y);
      unpair(h[r][i][1], v.z, v.w);
      if (vec && n < N) {
        *reinterpret_cast<float4*>(dst + n) = v;
      } else {
        if (n < N) dst[n] = v.x;
        if (n + 1 < N) dst[n + 1] = v.y;
        if (n + 2 < N) dst[n + 2] = v.z;
        if (n + 3 < N) dst[n + 3] = v.w;
      }
    }
  }
}

template <typename T, int NI, int R>
cudaError_t launch(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  const long long ctas = p.row_blocks * a.H * a.seqs.n_seq * p.nseg;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (p.nseg > 1) {
    ssm_steps_kernel<T, NI, R, false><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (int)p.row_blocks, p.nseg, p.seg_len);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  ssm_steps_kernel<T, NI, R, true><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (int)p.row_blocks, p.nseg, p.seg_len);
  return cudaGetLastError();
}

template <typename T, int NI>
cudaError_t by_rows(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  return p.rows == 64 ? launch<T, NI, 2>(a, p, s) : launch<T, NI, 1>(a, p, s);
}

template <typename T>
cudaError_t by_states(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  switch (p.ni) {
    case 1: return by_rows<T, 1>(a, p, s);
    case 2: return by_rows<T, 2>(a, p, s);
    case 4: return by_rows<T, 4>(a, p, s);
    default: return launch<T, 8, 1>(a, p, s);
  }
}

}  // namespace

// 64 rows a CTA share what is staged where that still leaves two CTAs an SM; segments where there is
// not one for each of four on every SM.
StepsPlan ssm_steps_plan(long long n_seq, long long max_len, long long H, long long P, long long N, int sm_count) {
  StepsPlan p{};
  p.ni = N <= 32 ? 1 : N <= 64 ? 2 : N <= 128 ? 4 : 8;
  const long long heads = n_seq * H;
  p.rows = p.ni < 8 && P > 32 && heads * ((P + 63) / 64) >= 2LL * sm_count ? 64 : 32;
  p.row_blocks = (P + p.rows - 1) / p.rows;
  p.nseg = 1;
  p.seg_len = max_len > 0 ? max_len : 1;
  const long long ctas = heads * p.row_blocks;
  if (max_len >= kSegMin && ctas > 0 && ctas * 3 <= 4LL * sm_count) {
    long long k = 4LL * sm_count / ctas;
    if (k > max_len / 64) k = max_len / 64;
    p.seg_len = ((max_len + k - 1) / k + kTok - 1) / kTok * kTok;
    p.nseg = (int)((max_len + p.seg_len - 1) / p.seg_len);
    if (p.nseg > 1)
      p.ws_bytes = (size_t)ctas * ws_floats(p.nseg, p.rows / 32 * p.ni * 4 * kThreads) * sizeof(float);
  }
  return p;
}

cudaError_t launch_ssm_steps(const SsmArgs& a, const StepsPlan& p, bool bf16, cudaStream_t s) {
  return bf16 ? by_states<__nv_bfloat16>(a, p, s) : by_states<float>(a, p, s);
}

}  // namespace vla
