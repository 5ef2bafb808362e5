// Operands of the tensor-core products: those that TMA cannot read as they are (float32, as three bfloat16 terms; rows off
// 16-byte boundaries) are copied to the workspace first, memory bound, 10 bytes a float32 value; tensor maps.
#include "vla_gemm.cuh"

namespace vla {
namespace gemm {
namespace {

// One row piece of 8 values a thread.  x1 = x rounded, x2 = x - x1 rounded, x3 = x - x1 - x2 rounded: the differences
// are exact.  A value beyond bfloat16's range, an infinity or a NaN has only its first term.
template <typename I>
__global__ void __launch_bounds__(256) pack_kernel(const Copies c) {
  all_started();   // the products
  const Operand& o = c.o[blockIdx.y];
  const long long across = (o.cols + 7) / 8, all = o.rows * across;
  const bool vec = ((reinterpret_cast<uintptr_t>(o.p) | (uintptr_t)(o.row * o.size)) & 15u) == 0;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const long long r = i / across, at = (i - r * across) * 8;
    const I* p = static_cast<const I*>(o.p) + r * o.row + at;
    const int left = o.cols - at < 8 ? (int)(o.cols - at) : 8;
    if constexpr (sizeof(I) == 4) {
      float v[8];
      if (vec && left == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.f;
      }
      Vec<__nv_bfloat16, 8> t[3];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[0].v[j] = __float2bfloat16_rn(v[j]);
        float rest = v[j] - __bfloat162float(t[0].v[j]);
        if (!isfinite(rest)) rest = 0.f;
        t[1].v[j] = __float2bfloat16_rn(rest);
        t[2].v[j] = __float2bfloat16_rn(rest - __bfloat162float(t[1].v[j]));
      }
      __nv_bfloat16* to = static_cast<__nv_bfloat16*>(c.to[blockIdx.y]);
#pragma unroll
      for (int k = 0; k < 3; ++k) st_vec<__nv_bfloat16, 8>(to + (k * o.rows + r) * o.out_row + at, t[k]);
    } else {
      Vec<I, 8> t;
#pragma unroll
      for (int j = 0; j < 8; ++j) t.v[j] = p[j < left ? j : 0];   // the row's end is not read by anyone
      st_vec<I, 8>(static_cast<I*>(c.to[blockIdx.y]) + r * o.out_row + at, t);
    }
  }
}

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

}  // namespace

Operand operand(const void* p, long long side, long long kd, long long row, bool mn, int size) {
  Operand o{};
  o.p = p;
  o.size = size;
  o.mn = mn;
  o.rows = mn ? kd : side;
  o.cols = mn ? side : kd;
  o.row = row;
  o.out_row = (o.cols + 15) / 16 * 16;
  if (o.rows == 1) o.row = o.out_row;   // not used
  o.pack = size == 4 || (reinterpret_cast<uintptr_t>(p) & 15u) || o.row * size % 16 || o.row < o.cols;
  o.bytes = o.pack ? (size_t)o.rows * o.out_row * (size == 4 ? 6 : size) : 0;
  return o;
}

bool encode(CUtensorMap* m, const Operand& o, const void* base, int box_x, int box_y) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const int size = o.size == 1 ? 1 : 2;
  const cuuint64_t row = (cuuint64_t)((o.pack ? o.out_row : o.row) * size);
  const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, o.size == 4 ? 3ull : 1ull};
  const cuuint64_t strides[2] = {row, row * (cuuint64_t)o.rows};
  const cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, o.size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t pack(const Copies& c, int sm_count, cudaStream_t s) {
  long long most = 0;
  for (int i = 0; i < c.count; ++i) {
    const long long ctas = (c.o[i].rows * ((c.o[i].cols + 7) / 8) + 255) / 256;
    if (ctas > most) most = ctas;
  }
  const long long cap = 16LL * sm_count;
  const dim3 grid((unsigned int)(most < cap ? most : cap), (unsigned int)c.count);
  if (c.o[0].size == 4) pack_kernel<float><<<grid, 256, 0, s>>>(c);
  else if (c.o[0].size == 2) pack_kernel<unsigned short><<<grid, 256, 0, s>>>(c);
  else pack_kernel<unsigned char><<<grid, 256, 0, s>>>(c);
  return cudaGetLastError();
}

GemmArgs args_of(const ProductArgs& p) {
  GemmArgs g{};
  g.M = p.M;
  g.N = p.N;
  g.out = p.out;
  g.status = p.status;
  const size_t size = p.out.y_bf16 ? 2 : 4;
  auto aligned = [&](const void* x, long long row, size_t to) {
    return ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)((size_t)row * size)) & (to - 1)) == 0;
  };
  g.part_row = (p.N + 7) / 8 * 8;
  g.direct = p.N * size % 32 == 0 && aligned(p.out.y, p.out.y_row, 32) && (!p.out.pre || aligned(p.out.pre, p.out.pre_row, 32)) &&
             (!p.out.residual || aligned(p.out.residual, p.out.res_row, 32)) &&
             ((reinterpret_cast<uintptr_t>(p.out.bias) | reinterpret_cast<uintptr_t>(p.out.w_scale)) & 15u) == 0;
  g.y_vec = aligned(p.out.y, p.out.y_row, 4 * size);
  g.res_vec = aligned(p.out.residual, p.out.res_row, 4 * size);
  g.pre_vec = aligned(p.out.pre, p.out.pre_row, 4 * size);
  return g;
}

}  // namespace gemm
}  // namespace vla
