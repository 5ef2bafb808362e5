// Selective state space scan, token by token (the decay is one number a head):
//   s_t = softplus(dt_t + bias),  h_t = exp(A s_t) h_{t-1} + s_t x_t B_t^T,
//   y_t = (h_t C_t + D x_t) * silu(z_t),   h in R^{P x N}, B_t, C_t in R^N shared by H / G heads.
//
// Rows of h never meet, so a CTA takes some of the P rows of one (sequence, head) and keeps them in
// registers.  This is the form for what the single-token form (vla_ssm_token.cu) and the tensor-core
// form (vla_ssm_prompt.cu) do not take: float32 input and output, short prompts, odd sizes and
// alignments.
//
// A token costs three float32 operations a state element (in packed pairs): with many heads that is
// what bounds the kernel.  So a thread has a tile of 4 rows x 8 states: B and C, which every row needs,
// are read from shared memory once for 4 rows (one row a thread: shared memory bounds it, 253 us
// instead of 157 for a sequence of 2048 tokens with 32 heads of 64 x 128), and the sums over N of 4
// tokens x 4 rows are folded together, each step of the butterfly halving the sums a lane carries.
// Tokens are staged 8 at a time in two buffers, one barrier for 8 tokens, the next 8 on their way in
// registers.  8 sequences of 1024 tokens, 32 heads of 64 x 128, float32: 431 us, 0.42 us a token with two CTAs on
// most SMs, the float32 pipe 65 % busy there (53 % over all SMs: 256 CTAs on 152).
// Few CTAs: a thread has one row and four times as many CTAs a shorter step each.
//
// Few CTAs and a long sequence: it is cut into segments, one CTA each.  A first launch forms what
// every segment but a sequence's last adds to the state, the second starts each segment from those,
// joined in a fixed order.  Everything is float32 and every sum has a fixed order: the same bits
// every time.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kTok = 8;    // tokens staged in shared memory at a time
constexpr long long kSeg = 32;       // tokens of a segment at least (4 sequences of 513 tokens, 8 heads of 64 x 64: 16 tokens
                                     // 33.2 us, 32 30.7, 64 37.7, 128 47.1)
constexpr long long kSegMin = 96;    // shorter sequences are not cut (one sequence, 8 heads of 64 x 64: 96 tokens 12.6 us
                                     // whole and 11.3 cut, 192 tokens 23.1 and 13.3)

// Threads of a CTA: 16 groups of LPR lanes, or 8 of 32.
constexpr int cta_threads(int lpr) { return lpr == 8 ? 128 : 256; }

// Floats of one (sequence, head, row block) in the workspace: nseg states of `per` floats (the last
// segment's place holds the state before the sequence), then the segments' decays; whole 16 bytes.
__host__ __device__ constexpr long long ws_floats(int nseg, int per) { return (long long)nseg * per + (nseg + 3) / 4 * 4; }

// A thread has R rows and 4 NI states of each, LPR lanes a row (N <= 4 NI LPR).
// FULL: outputs and the final state; else what the segment adds to the state.
template <typename T, int LPR, int NI, int R, bool FULL>
__global__ void __launch_bounds__(cta_threads(LPR), 512 / cta_threads(LPR))
    ssm_steps_kernel(const SsmArgs a, int row_blocks, int nseg, long long seg_len) {
  constexpr int kThreads = cta_threads(LPR);
  constexpr int ROWS = kThreads / LPR * R;
  constexpr int NP = 4 * NI * LPR;   // N rounded up
  constexpr int kFold = R == 1 ? 8 : 4;   // tokens whose sums are folded together
  constexpr int EB = kTok * NP / kThreads, EX = (kTok * ROWS + kThreads - 1) / kThreads;   // staged values a thread
  static_assert(kTok % kFold == 0 && (kTok * ROWS) % 32 == 0, "");
  __shared__ __align__(16) float sB[2][kTok][NP];
  __shared__ __align__(16) float sC[FULL ? 2 : 1][FULL ? kTok : 1][NP];
  __shared__ __align__(16) float sx[2][kTok][ROWS];
  __shared__ float sz[FULL ? 2 : 1][FULL ? kTok : 1][ROWS];
  __shared__ __align__(8) float2 sdec[2][kTok];   // decay, time step

  if (!FULL) all_started();
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
  if (!q.run || t_begin >= q.len || (!FULL && last)) {
    if (FULL && nseg > 1) wait_for_first();
    return;
  }

  const bool packed = a.seqs.offsets != nullptr;
  const long long g = head / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid % LPR, grp = tid / LPR;   // rows R grp .. of the block
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
      const bool in = t < kTok && t0 + t < t_end && p < rows;
      nx[k] = in ? x[(t0 + t) * a.x_tok + p] : none;
      if (FULL) nz[k] = in && z ? z[(t0 + t) * a.z_tok + p] : none;
    }
    if (tid < kTok && t0 + tid < t_end) ndt = to_f32<T>(dt[(t0 + tid) * a.dt_tok]);
  };
  fetch(t_begin);

  constexpr int PER = R * NI * 4 * kThreads;
  float* ws = nseg > 1 ? a.ws + ((s * a.H + head) * row_blocks + rb) * ws_floats(nseg, PER) : nullptr;
  const bool from_ws = FULL && q.len > seg_len;

  uint64_t h[R][NI][2];   // pairs of states
  const bool vec = (N & 3) == 0;   // rows of the state are then 16-byte aligned (its base is)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = R * grp + r;
    const float* src = a.state && seg == 0 && !from_ws ? a.state + ((q.slot * a.H + head) * a.P + p0 + p) * N : nullptr;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 4 * LPR * i + 4 * lane;
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
    wait_for_first();
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

  float log_total = 0.f;
  int buf = 0;
  for (long long t0 = t_begin; t0 < t_end; t0 += kTok, buf ^= 1) {
    const int n_tok = (int)(t_end - t0 < kTok ? t_end - t0 : kTok);
#pragma unroll
    for (int k = 0; k < EB; ++k) {
      const int e = k * kThreads + tid;
      (&sB[buf][0][0])[e] = to_f32<T>(nB[k]);
      if (FULL) (&sC[buf][0][0])[e] = to_f32<T>(nC[k]);
    }
#pragma unroll
    for (int k = 0; k < EX; ++k) {
      const int e = k * kThreads + tid;
      if (kTok * ROWS % kThreads == 0 || e < kTok * ROWS) {
        (&sx[buf][0][0])[e] = to_f32<T>(nx[k]);
        if (FULL) (&sz[buf][0][0])[e] = to_f32<T>(nz[k]);
      }
    }
    if (tid < kTok) {   // a token behind the end leaves the state as it is
      const float step = tid < n_tok ? time_step(ndt, bias, a.softplus) : 0.f;
      sdec[buf][tid] = make_float2(tid < n_tok ? expf(A * step) : 1.f, step);
      if (!FULL) log_total += tid < n_tok ? A * step : 0.f;
    }
    __syncthreads();   // also: nobody reads the other buffer any more
    if (t0 + kTok < t_end) fetch(t0 + kTok);
    for (int tb = 0; tb < n_tok; tb += kFold) {
      float acc[R * kFold];
#pragma unroll
      for (int j = 0; j < kFold; ++j) {
        const int t = tb + j;
        const float2 ds = sdec[buf][t];
        const uint64_t dec2 = pair(ds.x, ds.x);
        uint64_t in2[R], sum[R];
        const Vec<float, R> xs = ld_vec<float, R>(&sx[buf][t][R * grp]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float in = ds.y * xs.v[r];
          in2[r] = pair(in, in);
          sum[r] = 0;   // two zeros
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(&sB[buf][t][4 * LPR * i + 4 * lane]);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            h[r][i][0] = fma2(dec2, h[r][i][0], mul2(in2[r], pair(b.x, b.y)));
            h[r][i][1] = fma2(dec2, h[r][i][1], mul2(in2[r], pair(b.z, b.w)));
          }
          if (FULL) {
            const float4 c = *reinterpret_cast<const float4*>(&sC[buf][t][4 * LPR * i + 4 * lane]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              sum[r] = i == 0 ? mul2(h[r][i][0], pair(c.x, c.y)) : fma2(h[r][i][0], pair(c.x, c.y), sum[r]);
              sum[r] = fma2(h[r][i][1], pair(c.z, c.w), sum[r]);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float e, f;
          unpair(sum[r], e, f);
          acc[r * kFold + j] = e + f;
        }
      }
      if constexpr (FULL) {
        // a lane's bits, from the highest, choose the half of the sums it keeps: of sum r kFold + j
        // the lanes r kFold + j over LPR / (R kFold) are left, or each lane has several
        constexpr int SUMS = R * kFold;
#pragma unroll
        for (int o = LPR / 2, n = SUMS / 2; o > 0; o >>= 1, n >>= 1) {
          if (n > 0) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int k = 0; k < n; ++k) {
              const float keep = up ? acc[k + n] : acc[k], send = up ? acc[k] : acc[k + n];
              acc[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          } else {
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
          }
        }
        constexpr int LEFT = SUMS > LPR ? SUMS / LPR : 1, COPIES = LPR > SUMS ? LPR / SUMS : 1;
        const int first = lane / COPIES * LEFT;
#pragma unroll
        for (int k = 0; k < LEFT; ++k) {
          const int t = tb + (first + k) % kFold, p = R * grp + (first + k) / kFold;
          if (t < n_tok && p < rows && lane % COPIES == 0) {
            float v = fmaf(D, sx[buf][t][p], acc[k]);
            if (z) v *= silu<sizeof(T) == 2>(sz[buf][t][p]);
            y[(t0 + t) * a.y_tok + p] = from_f32<T>(v);
          }
        }
      }
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
  if (nseg > 1) wait_for_first();   // the call ends after both
  if (!a.state || !last) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = R * grp + r;
    if (p >= rows) continue;
    float* dst = a.state + ((q.slot * a.H + head) * a.P + p0 + p) * N;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int n = 4 * LPR * i + 4 * lane;
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

template <typename T, int LPR, int NI, int R>
cudaError_t launch(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  const long long ctas = p.row_blocks * a.H * a.seqs.n_seq * p.nseg;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  constexpr int threads = cta_threads(LPR);
  if (p.nseg > 1) {
    ssm_steps_kernel<T, LPR, NI, R, false><<<(unsigned int)ctas, threads, 0, s>>>(a, (int)p.row_blocks, p.nseg, p.seg_len);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.overlap)
      return launch_second(ssm_steps_kernel<T, LPR, NI, R, true>, (unsigned int)ctas, threads, 0, s, a,
                           (int)p.row_blocks, p.nseg, p.seg_len);
  }
  ssm_steps_kernel<T, LPR, NI, R, true><<<(unsigned int)ctas, threads, 0, s>>>(a, (int)p.row_blocks, p.nseg, p.seg_len);
  return cudaGetLastError();
}

template <typename T, int LPR, int NI>
cudaError_t by_rows(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  return p.rows > cta_threads(LPR) / LPR ? launch<T, LPR, NI, 4>(a, p, s) : launch<T, LPR, NI, 1>(a, p, s);
}

template <typename T>
cudaError_t by_states(const SsmArgs& a, const StepsPlan& p, cudaStream_t s) {
  switch (p.ni) {
    case 1: return by_rows<T, 8, 1>(a, p, s);
    case 2: return by_rows<T, 8, 2>(a, p, s);
    case 4: return by_rows<T, 16, 2>(a, p, s);
    default: return by_rows<T, 32, 2>(a, p, s);
  }
}

}  // namespace

// Four rows a thread where that still gives every SM a CTA (16 sequences of 40 tokens, 16 heads of 64 x 64:
// 14.8 us, one row 22.1; one sequence of 128 tokens, 32 heads, uncut: 28.2 us, one row 16.2); segments where
// there is not a CTA for each place on the SMs.
StepsPlan ssm_steps_plan(long long n_seq, long long max_len, long long H, long long P, long long N, int sm_count) {
  StepsPlan p{};
  p.ni = N <= 32 ? 1 : N <= 64 ? 2 : N <= 128 ? 4 : 8;
  const int lpr = p.ni <= 2 ? 8 : p.ni == 4 ? 16 : 32;
  const long long heads = n_seq * H, segs = max_len >= kSegMin ? max_len / kSeg : 1;
  const int narrow = cta_threads(lpr) / lpr, wide = 4 * narrow;
  p.rows = P > narrow && heads * ((P + wide - 1) / wide) * segs >= sm_count ? wide : narrow;
  p.row_blocks = (P + p.rows - 1) / p.rows;
  p.nseg = 1;
  p.seg_len = max_len > 0 ? max_len : 1;
  const long long ctas = heads * p.row_blocks, most = 4LL * sm_count * 128 / cta_threads(lpr);
  if (max_len >= kSegMin && ctas > 0 && ctas * 3 <= most) {
    long long k = most / ctas;
    if (k > max_len / kSeg) k = max_len / kSeg;
    p.seg_len = ((max_len + k - 1) / k + kTok - 1) / kTok * kTok;
    p.nseg = (int)((max_len + p.seg_len - 1) / p.seg_len);
    // the second launch's CTAs wait beside the first's where there is room for both (8 heads of 64 x 64, 1000
    // tokens: 27.2 us, 25.5 beside it); where there is not, the places they get are uneven (4 sequences
    // of 513 tokens: 30.5 us, 33.3 beside it)
    p.overlap = 2 * ctas * p.nseg <= most;
    if (p.nseg > 1)
      p.ws_bytes = (size_t)ctas * ws_floats(p.nseg, p.rows * 4 * lpr * (p.ni == 1 ? 1 : 2)) * sizeof(float);
  }
  return p;
}

cudaError_t launch_ssm_steps(const SsmArgs& a, const StepsPlan& p, bool bf16, cudaStream_t s) {
  return bf16 ? by_states<__nv_bfloat16>(a, p, s) : by_states<float>(a, p, s);
}

}  // namespace vla
