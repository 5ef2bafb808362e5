// Shared by the operators of a state space layer (short convolution, selective scan, norm): the
// description of a batch of sequences, its checked device-side reading, and 16-byte vectors.
#pragma once

#include <cuda_fp8.h>

#include "vla_internal.cuh"

namespace vla {

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
  float* ws;              // segments' states (see vla_ssm_prompt.cu)
  DevStatus* status;
};
cudaError_t launch_ssm_steps(const SsmArgs& a, bool bf16, int sm_count, cudaStream_t s);

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
};
cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t s);

// The time step of a head: softplus(x) = log(1 + e^x), which is x itself from 20 on (e^-20 is below
// half an ulp of 20 in float32).
__device__ __forceinline__ float time_step(float x, float bias, bool softplus) {
  x += bias;
  return softplus && x <= 20.f ? log1pf(expf(x)) : x;
}

}  // namespace vla
