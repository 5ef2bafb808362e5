// Selective state space scan of one token a sequence: h = exp(A s) h + s x B^T, y = (h C + D x) silu(z).
//
// The float32 state is read and written once (8 P N bytes a head; everything else is P and N values)
// and that is all the time there is: memory bound, or, for a sequence or two, one trip to memory
// and back.  A warp takes whole rows of the state, 16 bytes a lane, LPR lanes a row, all of its
// rows in flight before the first is used; B, C, the time step and x are loaded once a warp and
// the rows' sums over N are folded together (each step of the butterfly halves the rows a
// lane carries), no shared memory and no barrier.
// 128 sequences, 64 heads of 64 x 128: 86 us, 6.26 TB/s, 92 % of a plain copy's rate.  One sequence:
// 2.6 us on the GPU, which is about what a kernel of one trip to memory takes; the call takes 15 to 18 us on the host.
#include "vla_layer.cuh"

namespace vla {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p, bool vec) {
  if (vec) {
    const Vec<T, 4> v = ld_vec<T, 4>(p);
    return make_float4(to_f32<T>(v.v[0]), to_f32<T>(v.v[1]), to_f32<T>(v.v[2]), to_f32<T>(v.v[3]));
  }
  return make_float4(to_f32<T>(p[0]), to_f32<T>(p[1]), to_f32<T>(p[2]), to_f32<T>(p[3]));
}

// N <= 4 LPR K4, N a multiple of 4.  A warp has NPASS (32 / LPR) rows.
template <typename T, int LPR, int K4, int NPASS>
__global__ void __launch_bounds__(kThreads) ssm_token_kernel(const SsmArgs a, unsigned int row_blocks, bool vec) {
  constexpr int RPP = 32 / LPR, ROWS = RPP * NPASS;
  constexpr int XW = (ROWS + 31) / 32;
  const int lane = threadIdx.x & 31;
  const unsigned int task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned int rb = task % row_blocks, sh = task / row_blocks;
  const unsigned int H = (unsigned int)a.H, head = sh % H;
  const long long s = sh / H;
  if (s >= a.seqs.n_seq) return;
  const long long slot = a.seqs.slots ? a.seqs.slots[s] : s;
  const int N = (int)a.N, P = (int)a.P;
  const int n0 = (lane % LPR) * 4, sub = lane / LPR;
  const int p0 = (int)rb * ROWS;
  const unsigned int g = head / (H / (unsigned int)a.G);

  const T* x = static_cast<const T*>(a.x) + s * a.x_seq + (long long)head * P;
  const T* B = static_cast<const T*>(a.B) + s * a.B_seq + (long long)g * N;
  const T* C = static_cast<const T*>(a.C) + s * a.C_seq + (long long)g * N;
  const float dt = to_f32<T>(static_cast<const T*>(a.dt)[s * a.dt_seq + head]);
  const float A = a.A[head], bias = a.dt_bias ? a.dt_bias[head] : 0.f, D = a.D ? a.D[head] : 0.f;
  float xr[XW];
#pragma unroll
  for (int i = 0; i < XW; ++i) {
    const int p = p0 + 32 * i + lane;
    xr[i] = 32 * i + lane < ROWS && p < P ? to_f32<T>(x[p]) : 0.f;
  }
  float4 b[K4], c[K4];
#pragma unroll
  for (int k = 0; k < K4; ++k) {
    const int n = n0 + 4 * LPR * k;
    b[k] = c[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < N) {
      b[k] = load4<T>(B + n, vec);
      c[k] = load4<T>(C + n, vec);
    }
  }
  if (slot < 0) return;
  if (slot >= a.seqs.n_slots) {
    if (lane == 0) atomicOr(&a.status->flags, kStatusIndex);
    return;
  }
  float* state = a.state ? a.state + ((slot * a.H + head) * P + p0) * N : nullptr;
  float4 h[NPASS][K4];
#pragma unroll
  for (int i = 0; i < NPASS; ++i) {
    const int r = RPP * i + sub;
#pragma unroll
    for (int k = 0; k < K4; ++k) {
      const int n = n0 + 4 * LPR * k;
      h[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (state && p0 + r < P && n < N) h[i][k] = *reinterpret_cast<const float4*>(state + (long long)r * N + n);
    }
  }
  const float step = time_step(dt, bias, a.softplus), dec = expf(A * step);
  float v[NPASS];
#pragma unroll
  for (int i = 0; i < NPASS; ++i) {
    const int r = RPP * i + sub;
    const float in = step * __shfl_sync(0xffffffffu, xr[RPP * i / 32], r & 31);
    v[i] = 0.f;
#pragma unroll
    for (int k = 0; k < K4; ++k) {
      float4& q = h[i][k];
      q.x = fmaf(dec, q.x, in * b[k].x);
      q.y = fmaf(dec, q.y, in * b[k].y);
      q.z = fmaf(dec, q.z, in * b[k].z);
      q.w = fmaf(dec, q.w, in * b[k].w);
      v[i] = fmaf(q.x, c[k].x, v[i]);
      v[i] = fmaf(q.y, c[k].y, v[i]);
      v[i] = fmaf(q.z, c[k].z, v[i]);
      v[i] = fmaf(q.w, c[k].w, v[i]);
      const int n = n0 + 4 * LPR * k;
      if (state && p0 + r < P && n < N) *reinterpret_cast<float4*>(state + (long long)r * N + n) = q;
    }
  }
  // sums over the LPR lanes of a row: lane bits choose which half of the passes a lane keeps
  int pass = 0, cnt = NPASS, spare = 0;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    if (cnt > 1) {
      cnt >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < NPASS / 2; ++j) {
        if (j >= cnt) break;
        const float keep = up ? v[j + cnt] : v[j], send = up ? v[j] : v[j + cnt];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      if (up) pass += cnt;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      spare |= lane & o;
    }
  }
  const T* z = a.z ? static_cast<const T*>(a.z) + s * a.z_seq + (long long)head * P : nullptr;
  T* y = static_cast<T*>(a.y) + s * a.y_seq + (long long)head * P;
#pragma unroll
  for (int j = 0; j < NPASS; ++j) {
    if (j >= cnt) break;
    const int r = RPP * (pass + j) + sub;
    float xv = __shfl_sync(0xffffffffu, xr[0], r & 31);
    if (XW > 1) {
      const float other = __shfl_sync(0xffffffffu, xr[XW - 1], r & 31);
      if (r >= 32) xv = other;
    }
    if (spare || p0 + r >= P) continue;
    float o = fmaf(D, xv, v[j]);
    if (z) o *= silu<sizeof(T) == 2>(to_f32<T>(z[p0 + r]));
    y[p0 + r] = from_f32<T>(o);
  }
}

template <typename T, int LPR, int K4, int NPASS>
cudaError_t launch(const SsmArgs& a, cudaStream_t s) {
  constexpr int ROWS = 32 / LPR * NPASS;
  const long long blocks = (a.P + ROWS - 1) / ROWS, tasks = blocks * a.H * a.seqs.n_seq;
  const long long ctas = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL || tasks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C);
  const bool vec = (at | (unsigned long long)(a.B_seq | a.C_seq) * sizeof(T)) % (4 * sizeof(T)) == 0;
  ssm_token_kernel<T, LPR, K4, NPASS><<<(unsigned int)ctas, kThreads, 0, s>>>(a, (unsigned int)blocks, vec);
  return cudaGetLastError();
}

// 8 vectors a lane in flight; 2 where that would leave SMs without their fill of warps.
template <typename T, int LPR, int K4>
cudaError_t by_size(const SsmArgs& a, int sm_count, cudaStream_t s) {
  const long long warps = a.seqs.n_seq * a.H * ((a.P * LPR * K4 + 255) / 256);
  return warps >= 16LL * sm_count ? launch<T, LPR, K4, 8 / K4>(a, s) : launch<T, LPR, K4, 2 / K4>(a, s);
}

template <typename T>
cudaError_t by_states(const SsmArgs& a, int sm_count, cudaStream_t s) {
  if (a.N <= 16) return by_size<T, 4, 1>(a, sm_count, s);
  if (a.N <= 32) return by_size<T, 8, 1>(a, sm_count, s);
  if (a.N <= 64) return by_size<T, 16, 1>(a, sm_count, s);
  if (a.N <= 128) return by_size<T, 32, 1>(a, sm_count, s);
  return by_size<T, 32, 2>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_ssm_token(const SsmArgs& a, bool bf16, int sm_count, cudaStream_t s, bool* used) {
  *used = a.seqs.offsets == nullptr && a.seqs.max_len == 1 && a.N % 4 == 0 && a.N <= 256 && a.H <= 0x7fffffffLL &&
          a.P <= 0x7fffffffLL / 256;
  if (!*used) return cudaSuccess;
  return bf16 ? by_states<__nv_bfloat16>(a, sm_count, s) : by_states<float>(a, sm_count, s);
}

}  // namespace vla
