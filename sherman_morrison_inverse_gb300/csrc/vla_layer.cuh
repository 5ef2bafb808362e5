// Shared by the operators of a state space layer (short convolution, selective scan, norm): the
// description of a batch of sequences, its checked device-side reading, and 16-byte vectors.
#pragma once

#include <cuda_fp8.h>

#include "vla_internal.cuh"

namespace vla {

constexpr unsigned int kStatusIndex = 4u;   // VLA_STATUS_INDEX

// A batch of sequences over token rows.  Dense (offsets == NULL): n_seq sequences of T tokens.
// Packed: sequence s is the rows [offsets[s], offsets[s + 1]) of a buffer of T rows.
struct Seqs {
  const int* offsets;
  const int* slots;     // state of sequence s; NULL: s itself; negative: the sequence is skipped
  long long n_seq;
  long long T;
  long long max_len;    // no sequence is longer (packed); T (dense)
  long long n_slots;
};

struct SeqRange {
  long long start;   // packed: first row of the sequence; dense: 0
  long long len;
  long long slot;
  bool run;
};

// What sequence s covers.  Offsets or slots outside their ranges come back as a sequence that is
// not run, with kStatusIndex for the status: the kernels read and write nothing for it.
__device__ __forceinline__ SeqRange seq_range(const Seqs& q, long long s, unsigned int* bad) {
  SeqRange r{0, q.T, s, true};
  if (q.offsets) {
    const long long b = q.offsets[s], e = q.offsets[s + 1];
    r.start = b;
    r.len = e - b;
    if (b < 0 || e < b || e > q.T || r.len > q.max_len) {
      *bad |= kStatusIndex;
      r.run = false;
    }
  }
  if (q.slots) r.slot = q.slots[s];
  if (r.slot < 0) r.run = false;
  if (r.slot >= q.n_slots) {
    *bad |= kStatusIndex;
    r.run = false;
  }
  return r;
}

// VEC consecutive values of T as one memory access (VEC * sizeof(T) in {2, 4, 8, 16}).
template <int BYTES> struct RawVec;
template <> struct RawVec<2> { using type = unsigned short; };
template <> struct RawVec<4> { using type = uint32_t; };
template <> struct RawVec<8> { using type = uint2; };
template <> struct RawVec<16> { using type = uint4; };

template <typename T, int VEC>
union Vec {
  typename RawVec<(int)sizeof(T) * VEC>::type raw;
  T v[VEC];
  __device__ Vec() {}
};

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> ld_vec(const T* p) {
  Vec<T, VEC> r;
  r.raw = *reinterpret_cast<const decltype(r.raw)*>(p);
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void st_vec(T* p, const Vec<T, VEC>& x) {
  *reinterpret_cast<decltype(x.raw)*>(p) = x.raw;
}

// Pairs of float32 in one 64-bit register, and their packed arithmetic (one instruction a pair).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two bfloat16 of one 32-bit word (a in the low half), and back.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// x * sigmoid(x) of a pair with approximate exponential and reciprocal (a few ulp of float32).
// e^-x overflows to infinity below -88: the reciprocal is then 0 and the result -0.
__device__ __forceinline__ uint64_t silu2(uint64_t x) {
  const float l = -1.44269504088896341f;
  float a, b;
  unpair(mul2(x, pair(l, l)), a, b);
  unpair(add2(pair(ex2(a), ex2(b)), pair(1.f, 1.f)), a, b);
  return mul2(x, pair(rcp(a), rcp(b)));
}

// x * sigmoid(x).  float32 results keep expf and the rounded division; a result that is rounded to
// bfloat16 takes the approximate ones (a few ulp of float32).
template <bool FAST>
__device__ __forceinline__ float silu(float x) {
  return FAST ? __fdividef(x, 1.f + __expf(-x)) : x / (1.f + expf(-x));
}

struct ConvArgs {
  const void* x;
  const float* w;      // [C, K]
  const float* bias;   // [C] or NULL
  void* state;         // [n_slots, K - 1, C] or NULL
  void* y;
  Seqs seqs;
  long long C;
  long long x_seq, x_tok, y_seq, y_tok;   // strides in elements (channels are adjacent)
  int K;
  bool silu;
  int sm_count;
  DevStatus* status;
};
cudaError_t launch_short_conv(const ConvArgs& a, bool bf16, cudaStream_t s);

struct SsmArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;         // [H] or NULL
  const void* z;          // or NULL
  const float* dt_bias;   // [H] or NULL
  float* state;           // [n_slots, H, P, N] or NULL
  void* y;
  Seqs seqs;
  long long H, P, G, N;
  long long x_seq, x_tok, dt_seq, dt_tok, B_seq, B_tok, C_seq, C_tok, z_seq, z_tok, y_seq, y_tok;
  bool softplus;
  float* ws;              // segments' states
  DevStatus* status;
};
// One token a sequence; *used = false: not this form's call, nothing was launched.
cudaError_t launch_ssm_token(const SsmArgs& a, bool bf16, int sm_count, cudaStream_t s, bool* used);
// Token by token, any sizes.
struct StepsPlan {
  int ni;                         // 32 ni >= N states a row
  int rows;                       // rows of the state a CTA
  long long row_blocks;
  int nseg;                       // segments a sequence is cut into
  long long seg_len;              // tokens a segment
  size_t ws_bytes;
  bool overlap;                   // the second launch starts beside the first
};
StepsPlan ssm_steps_plan(long long n_seq, long long max_len, long long H, long long P, long long N, int sm_count);
cudaError_t launch_ssm_steps(const SsmArgs& a, const StepsPlan& plan, bool bf16, cudaStream_t s);

struct NormArgs {
  const void* x;
  const float* w;
  void* residual;   // or NULL
  void* y;
  float* scale;     // [rows] or [rows, ceil(D / 128)]; NULL without quantisation
  long long rows, D, x_row, res_row, y_row;
  float eps;
  int group;        // 0 or 128
  int out;          // vla_out_t
  bool res_bf16;
  int sm_count;
};
cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t s);

// The time step of a head: softplus(x) = log(1 + e^x), which is x itself from 20 on (e^-20 is below
// half an ulp of 20 in float32).
__device__ __forceinline__ float time_step(float x, float bias, bool softplus) {
  x += bias;
  return softplus && x <= 20.f ? log1pf(expf(x)) : x;
}

// A launch in two parts: the second's CTAs start as SMs become free, once every CTA of the first is
// running (all_started there), and wait for the first's results where they read them.
__device__ __forceinline__ void all_started() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_first() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_second(void (*kern)(P...), unsigned int ctas, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3((unsigned int)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, static_cast<A&&>(args)...);
}

}  // namespace vla
