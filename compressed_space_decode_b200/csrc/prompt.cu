// prompt.cu -- isoquant_prompt_attend: attention of packed prompts to
// themselves on uncompressed queries, keys and values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "isoquant_internal.cuh"

namespace isoquant {
namespace {

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

struct PromptArgs {
  const void *q, *k, *v;
  void *out;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu_seqlens;
  int n_tok, batch, Hq, H, G, causal;
  float scale;
  uint32_t *status;
};

// One warp per (token, query head): four coordinates per lane, the running
// maximum and sum of the softmax in fp32.
template <typename T>
__global__ void __launch_bounds__(256) k_prompt_rows(const PromptArgs p) {
  pdl_trigger();
  pdl_wait();
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(p.n_tok) * p.Hq) return;
  const int hq = static_cast<int>(w % p.Hq), t = static_cast<int>(w / p.Hq), h = hq / p.G;
  int begin = -1, end = 0;
  for (int b = 0; b < p.batch; ++b) {
    const int x = p.cu_seqlens[b], y = p.cu_seqlens[b + 1];
    if (x < 0 || y < x || y > p.n_tok) {
      if (lane == 0) set_status(p.status, ISOQUANT_DEVERR_SEQ_RANGE);
    } else if (t >= x && t < y) {
      begin = x;
      end = p.causal ? t + 1 : y;
    }
  }
  if (begin < 0) return;
  const uint2 qw = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.q) + t * p.q_stride + hq * kD + 4 * lane);
  const float2 q0 = unpack2(qw.x, T()), q1 = unpack2(qw.y, T());
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = begin; j < end; ++j) {
    const uint2 kw = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.k) + j * p.k_stride + h * kD + 4 * lane);
    const uint2 vw = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p.v) + j * p.v_stride + h * kD + 4 * lane);
    const float2 k0 = unpack2(kw.x, T()), k1 = unpack2(kw.y, T()), v0 = unpack2(vw.x, T()), v1 = unpack2(vw.y, T());
    float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s), a = __expf(m - mn), e = __expf(s - mn);
    m = mn;
    l = l * a + e;
    o[0] = o[0] * a + e * v0.x; o[1] = o[1] * a + e * v0.y;
    o[2] = o[2] * a + e * v1.x; o[3] = o[3] * a + e * v1.y;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + w * kD + 4 * lane) =
      make_uint2(pack2(o[0] * inv, o[1] * inv, T()), pack2(o[2] * inv, o[3] * inv, T()));
}

}  // namespace

cudaError_t launch_prompt_attend(const isoquant_ctx *ctx, const void *q, const void *k, const void *v, int dtype,
                                 int n_tok, int num_q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                 const int32_t *cu_seqlens, int batch, int causal, float scale, void *out,
                                 cudaStream_t stream) {
  PromptArgs p{q, k, v, out, q_stride, k_stride, v_stride, cu_seqlens, n_tok, batch, num_q_heads, ctx->num_kv_heads,
               num_q_heads / ctx->num_kv_heads, causal, scale, ctx->status};
  const int64_t rows = static_cast<int64_t>(n_tok) * num_q_heads;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8)), block(256);
  return dtype == ISOQUANT_BF16 ? launch_pdl(k_prompt_rows<__nv_bfloat16>, grid, block, 0, stream, p)
                                : launch_pdl(k_prompt_rows<__half>, grid, block, 0, stream, p);
}

}  // namespace isoquant
