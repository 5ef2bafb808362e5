// C entry points of the state space layer's operators: argument checks and dispatch.
#include "vla.h"
#include "vla_handle.cuh"
#include "vla_layer.cuh"
#include "vla_ssm_prompt.cuh"

#include <exception>

using namespace vla::api;

namespace {

constexpr long long kMaxStates = 256;     // N of the scan
constexpr long long kMaxWidth = 32768;    // D of the norm

// Checks a batch of sequences and fills it in.  state: whether the call carries states.
vla_err_t check_seqs(vla_handle_t h, const std::string& f, long long n_seq, long long T, long long max_len,
                     const int* offsets, const int* slots, long long n_slots, bool state, vla::Seqs* q) {
  if (n_seq < 0 || T < 0 || max_len < 0 || n_slots < 0)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (n_seq > 0x7fffffffLL || T > 0x7fffffffLL)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": n_seq and T must be below 2^31");
  if (slots && !state) return fail(h, VLA_ERR_INVALID_ARG, f + ": slots without a state");
  if (state && !slots && n_slots < n_seq)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": fewer states than sequences");
  q->offsets = offsets;
  q->slots = slots;
  q->n_seq = n_seq;
  q->T = T;
  q->max_len = offsets ? (max_len < T ? max_len : T) : T;
  q->n_slots = state ? n_slots : n_seq;
  return VLA_OK;
}

// Which form runs can hang on the operands' alignment: the workspace serves either.
size_t ws_need(const vla::PromptPlan& prompt, const vla::StepsPlan& steps) {
  return prompt.fits && prompt.ws_bytes > steps.ws_bytes ? prompt.ws_bytes : steps.ws_bytes;
}

// Whether pointers (NULL among them) are aligned to values of `size` bytes.
template <typename... P>
bool to_values(size_t size, P... p) { return ((reinterpret_cast<uintptr_t>(p) | ...) & (size - 1)) == 0; }
size_t size_of(vla_dtype_t t) { return t == VLA_BF16 ? 2 : 4; }

bool stride_ok(long long v) { return v >= 0 && v < (1LL << 40); }

// Rows of an output must not overlap: a stride that the call uses is at least a row's width.
bool out_ok(const vla::Seqs& q, long long seq, long long tok, long long width) {
  const bool uses_tok = q.offsets ? q.T > 1 : q.max_len > 1;
  const bool uses_seq = !q.offsets && q.n_seq > 1;
  return !(uses_tok && tok < width) && !(uses_seq && seq < width);
}

}  // namespace

extern "C" {

vla_err_t vla_short_conv(vla_handle_t h, const void* x, const float* w, const float* bias, void* state, void* y,
                         long long n_seq, long long T, long long max_len, const int* offsets, const int* slots,
                         long long n_slots, long long C, int K, const long long* strides, int silu,
                         vla_dtype_t io_dtype, void* stream) try {
  const std::string f = "vla_short_conv";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (io_dtype != VLA_F32 && io_dtype != VLA_BF16) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (C < 0 || C > 0x7fffffffLL) return fail(h, VLA_ERR_INVALID_ARG, f + ": C out of range");
  if (K < 2 || K > 4) return fail(h, VLA_ERR_UNSUPPORTED, f + ": built for 2, 3 or 4 taps");
  vla::ConvArgs a{};
  vla_err_t err = check_seqs(h, f, n_seq, T, max_len, offsets, slots, n_slots, state != nullptr, &a.seqs);
  if (err != VLA_OK) return err;
  if (n_seq == 0 || T == 0 || C == 0 || a.seqs.max_len == 0) return VLA_OK;
  if (!x || !w || !y || !strides) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(io_dtype), x, state, y) || !to_values(4, w, bias, offsets, slots))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  for (int i = 0; i < 4; ++i)
    if (!stride_ok(strides[i])) return fail(h, VLA_ERR_INVALID_ARG, f + ": stride out of range");
  if (!out_ok(a.seqs, strides[2], strides[3], C))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of y overlap");
  a.x = x; a.w = w; a.bias = bias; a.state = state; a.y = y;
  a.C = C; a.K = K; a.silu = silu != 0;
  a.sm_count = h->sm_count;
  // a dense batch of one sequence or one token never uses the other stride: 0 keeps it from
  // deciding the vector width
  a.x_seq = offsets || n_seq == 1 ? 0 : strides[0]; a.x_tok = a.seqs.max_len == 1 && !offsets ? 0 : strides[1];
  a.y_seq = offsets || n_seq == 1 ? 0 : strides[2]; a.y_tok = a.seqs.max_len == 1 && !offsets ? 0 : strides[3];
  a.status = h->status;
  cudaError_t e = on_device(h->device, [&]() {
    return vla::launch_short_conv(a, io_dtype == VLA_BF16, static_cast<cudaStream_t>(stream));
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_short_conv: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_ssm_scan(vla_handle_t h, const void* x, const void* dt, const float* A, const void* B, const void* C,
                       const float* D, const void* z, const float* dt_bias, float* state, void* y,
                       long long n_seq, long long T, long long max_len, const int* offsets, const int* slots,
                       long long n_slots, long long H, long long P, long long G, long long N,
                       const long long* strides, int softplus, vla_dtype_t io_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) try {
  const std::string f = "vla_ssm_scan";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (io_dtype != VLA_F32 && io_dtype != VLA_BF16) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (H < 0 || P < 0 || G < 0 || N < 0 || H > 0x7fffffffLL || P > 0x7fffffffLL)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": size out of range");
  vla::SsmArgs a{};
  vla_err_t err = check_seqs(h, f, n_seq, T, max_len, offsets, slots, n_slots, state != nullptr, &a.seqs);
  if (err != VLA_OK) return err;
  if (n_seq == 0 || T == 0 || H == 0 || P == 0 || a.seqs.max_len == 0) return VLA_OK;
  if (G == 0 || H % G != 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": H must be a multiple of G");
  if (N == 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": N must be positive");
  if (N > kMaxStates) return fail(h, VLA_ERR_UNSUPPORTED, f + ": built for N up to 256");
  if (!x || !dt || !A || !B || !C || !y || !strides) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(io_dtype), x, dt, B, C, z, y) || !to_values(4, A, D, dt_bias, offsets, slots))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if (state && !aligned16(state)) return fail(h, VLA_ERR_INVALID_ARG, f + ": state must be 16-byte aligned");
  for (int i = 0; i < 12; ++i)
    if (!stride_ok(strides[i])) return fail(h, VLA_ERR_INVALID_ARG, f + ": stride out of range");
  if (!out_ok(a.seqs, strides[10], strides[11], H * P))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of y overlap");
  a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.dt_bias = dt_bias; a.state = state; a.y = y;
  a.H = H; a.P = P; a.G = G; a.N = N;
  a.x_seq = strides[0]; a.x_tok = strides[1]; a.dt_seq = strides[2]; a.dt_tok = strides[3];
  a.B_seq = strides[4]; a.B_tok = strides[5]; a.C_seq = strides[6]; a.C_tok = strides[7];
  a.z_seq = strides[8]; a.z_tok = strides[9]; a.y_seq = strides[10]; a.y_tok = strides[11];
  a.softplus = softplus != 0;
  a.status = h->status;
  const bool bf16 = io_dtype == VLA_BF16;
  const vla::PromptPlan plan = vla::ssm_prompt_plan(n_seq, offsets ? T : n_seq * T, a.seqs.max_len, H, P, N, bf16, h->sm_count);
  const vla::StepsPlan steps = vla::ssm_steps_plan(n_seq, a.seqs.max_len, H, P, N, h->sm_count);
  const size_t need = ws_need(plan, steps);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": workspace missing, misaligned or smaller than vla_ssm_workspace says");
  a.ws = static_cast<float*>(workspace);
  cudaError_t e = on_device(h->device, [&]() {
    bool used = false;
    cudaError_t r = cudaSuccess;
    r = vla::launch_ssm_token(a, bf16, h->sm_count, static_cast<cudaStream_t>(stream), &used);
    if (r != cudaSuccess || used) return r;
    if (plan.fits) r = vla::launch_ssm_prompt(a, plan, static_cast<cudaStream_t>(stream), &used);
    if (r != cudaSuccess || used) return r;
    return vla::launch_ssm_steps(a, steps, bf16, static_cast<cudaStream_t>(stream));
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_ssm_scan: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_ssm_workspace(vla_handle_t h, long long n_seq, long long T, long long max_len, int packed, long long H,
                            long long P, long long N, vla_dtype_t io_dtype, size_t* bytes) try {
  const std::string f = "vla_ssm_workspace";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!bytes) return fail(h, VLA_ERR_INVALID_ARG, f + ": bytes is NULL");
  if (n_seq < 0 || T < 0 || max_len < 0 || H < 0 || P < 0 || N < 0)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (io_dtype != VLA_F32 && io_dtype != VLA_BF16) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (packed && max_len > T) max_len = T;
  const long long len = packed ? max_len : T;
  *bytes = ws_need(vla::ssm_prompt_plan(n_seq, packed ? T : n_seq * T, len, H, P, N, io_dtype == VLA_BF16, h->sm_count),
                   vla::ssm_steps_plan(n_seq, len, H, P, N, h->sm_count));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_rms_norm(vla_handle_t h, const void* x, const float* w, void* residual, void* y, float* scale,
                       long long rows, long long D, long long x_row, long long res_row, long long y_row, float eps,
                       int group, vla_out_t out, vla_dtype_t io_dtype, vla_dtype_t res_dtype, void* stream) try {
  const std::string f = "vla_rms_norm";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (io_dtype != VLA_F32 && io_dtype != VLA_BF16) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (residual && res_dtype != VLA_F32 && res_dtype != VLA_BF16)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown res_dtype");
  if (out != VLA_OUT_IO && out != VLA_OUT_E4M3 && out != VLA_OUT_INT8)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown output type");
  if (group != 0 && group != 128) return fail(h, VLA_ERR_INVALID_ARG, f + ": group must be 0 (a row) or 128");
  if (!(eps >= 0.f)) return fail(h, VLA_ERR_INVALID_ARG, f + ": eps must be >= 0 (NaN rejected)");
  if (rows < 0 || D < 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (!stride_ok(x_row) || !stride_ok(res_row) || !stride_ok(y_row))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": stride out of range");
  if (rows == 0 || D == 0) return VLA_OK;
  if (D > kMaxWidth) return fail(h, VLA_ERR_UNSUPPORTED, f + ": built for D up to 32768");
  if (!x || !w || !y || (out != VLA_OUT_IO && !scale)) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(io_dtype), x) || !to_values(out == VLA_OUT_IO ? size_of(io_dtype) : 1, y) ||
      !to_values(size_of(res_dtype), residual) || !to_values(4, w, scale))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if (rows > 1 && (y_row < D || (residual && res_row < D)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of y or the residual overlap");
  vla::NormArgs a{};
  a.x = x; a.w = w; a.residual = residual; a.y = y; a.scale = scale;
  a.rows = rows; a.D = D; a.x_row = x_row; a.res_row = res_row; a.y_row = y_row;
  a.eps = eps; a.group = out == VLA_OUT_IO ? 0 : group; a.out = out; a.res_bf16 = res_dtype == VLA_BF16;
  a.sm_count = h->sm_count;
  cudaError_t e = on_device(h->device, [&]() {
    return vla::launch_rms_norm(a, io_dtype == VLA_BF16, static_cast<cudaStream_t>(stream));
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_rms_norm: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

}  // extern "C"
