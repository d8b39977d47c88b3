// dense.cu -- isoquant_dense_prep: appends to the paged cache of 16-bit keys
// and values, with the position rotation of keys and queries.
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

// ------------------------------------------------------------------ append
struct DensePrepArgs {
  const void *k, *v, *q;
  void *k_out, *q_out, *data;  // k_out, data may be null
  const int64_t *slots, *k_pos, *q_pos;
  const float *table;  // null: no rotation
  int64_t num_pos;
  int rot, inter;
  int n_tok, n_rows, H, Hq;
  int num_pages, ps_shift;
  uint32_t q_items, k_items;  // items of the query rows, of the keys (and of the values)
  uint32_t *status;
};

// Eight lanes take a vector, 32 bytes each: the lanes below rot / 16 hold the
// two 8-coordinate chunks whose coordinates pair up (c and c + rot / 16, or
// adjacent ones if interleaved), the others two chunks that stay.
struct LanePart {
  int c0, c1;          // its chunks
  bool rotates;
  float c[8], s[8];    // cosines and sines (interleaved: four per chunk)
};

__device__ __forceinline__ void lane_part(const DensePrepArgs &g, int64_t pos, int l8, LanePart &p) {
  const int hp = g.table ? g.rot >> 4 : 0;
  p.rotates = l8 < hp;
  p.c0 = !p.rotates || g.inter ? 2 * l8 : l8;
  p.c1 = !p.rotates || g.inter ? 2 * l8 + 1 : l8 + hp;
  if (p.rotates) {
    const float4 *row = reinterpret_cast<const float4 *>(g.table + pos * g.rot + 8 * l8);
    const float4 *rs = reinterpret_cast<const float4 *>(g.table + pos * g.rot + (g.rot >> 1) + 8 * l8);
    const float4 a = row[0], b = row[1], d = rs[0], e = rs[1];
    p.c[0] = a.x; p.c[1] = a.y; p.c[2] = a.z; p.c[3] = a.w; p.c[4] = b.x; p.c[5] = b.y; p.c[6] = b.z; p.c[7] = b.w;
    p.s[0] = d.x; p.s[1] = d.y; p.s[2] = d.z; p.s[3] = d.w; p.s[4] = e.x; p.s[5] = e.y; p.s[6] = e.z; p.s[7] = e.w;
  }
}

// a' = a c - b s, b' = b c + a s in fp32 (one fma after one product), rounded
// once to T.
template <typename T>
__device__ __forceinline__ void rotate_part(const LanePart &p, int inter, uint4 &x, uint4 &y) {
  uint32_t *xw = reinterpret_cast<uint32_t *>(&x), *yw = reinterpret_cast<uint32_t *>(&y);
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack2(xw[i], T()), b = unpack2(yw[i], T());
      xw[i] = pack2(fmaf(a.x, p.c[i], -(a.y * p.s[i])), fmaf(a.y, p.c[i], a.x * p.s[i]), T());
      yw[i] = pack2(fmaf(b.x, p.c[4 + i], -(b.y * p.s[4 + i])), fmaf(b.y, p.c[4 + i], b.x * p.s[4 + i]), T());
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack2(xw[i], T()), b = unpack2(yw[i], T());
    xw[i] = pack2(fmaf(a.x, p.c[2 * i], -(b.x * p.s[2 * i])), fmaf(a.y, p.c[2 * i + 1], -(b.y * p.s[2 * i + 1])), T());
    yw[i] = pack2(fmaf(b.x, p.c[2 * i], a.x * p.s[2 * i]), fmaf(b.y, p.c[2 * i + 1], a.y * p.s[2 * i + 1]), T());
  }
}

// An item is HC heads of one token's queries, keys or values; its eight lanes
// load the table row once for all of them.
template <typename T, int HC>
__global__ void __launch_bounds__(256) k_dense_prep(const DensePrepArgs g) {
  pdl_trigger();
  pdl_wait();
  uint32_t item = blockIdx.x * 32u + (threadIdx.x >> 3);
  const int l8 = threadIdx.x & 7;
  int kind = 0;  // 0: queries, 1: keys, 2: values
  if (item >= g.q_items) {
    item -= g.q_items;
    kind = 1;
    if (item >= g.k_items) {
      item -= g.k_items;
      kind = 2;
      if (item >= g.k_items || g.data == nullptr) return;
    }
  }
  const int heads = kind == 0 ? g.Hq : g.H;
  const uint32_t per = (static_cast<uint32_t>(heads) + HC - 1) / HC;
  const int64_t row = item / per;
  const int h0 = static_cast<int>(item - static_cast<uint32_t>(row) * per) * HC;

  int64_t slot = -1;
  if (kind != 0 && g.data != nullptr) slot = g.slots[row];
  int64_t pos = 0;
  bool bad = false;
  if (g.table != nullptr && (kind == 0 || slot >= 0 || g.k_out != nullptr)) {
    pos = kind == 0 ? g.q_pos[row] : g.k_pos[row];
    bad = pos < 0 || pos >= g.num_pos;
    if (bad && l8 == 0) set_status(g.status, ISOQUANT_DEVERR_POS_RANGE);
  }
  const int64_t page = slot >> g.ps_shift;
  bool store = slot >= 0 && !bad;
  if (store && page >= g.num_pages) {
    if (l8 == 0) set_status(g.status, ISOQUANT_DEVERR_SLOT_RANGE);
    store = false;
  }
  T *out = kind == 0 ? static_cast<T *>(g.q_out) : kind == 1 ? static_cast<T *>(g.k_out) : nullptr;
  if (!store && out == nullptr) return;
  LanePart p;
  p.rotates = false;
  p.c0 = 2 * l8;
  p.c1 = 2 * l8 + 1;
  if (kind != 2 && !bad) lane_part(g, pos, l8, p);

  const T *src = static_cast<const T *>(kind == 0 ? g.q : kind == 1 ? g.k : g.v) + (row * heads + h0) * kD;
  uint4 x[HC], y[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (h0 + i < heads) {
      x[i] = *reinterpret_cast<const uint4 *>(src + i * kD + 8 * p.c0);
      y[i] = *reinterpret_cast<const uint4 *>(src + i * kD + 8 * p.c1);
    }
  }
  const int off = static_cast<int>(slot & ((1 << g.ps_shift) - 1));
  T *dst = static_cast<T *>(g.data) +
           (((page * 2 + (kind == 2)) * g.H + h0) * (int64_t(1) << g.ps_shift) + off) * kD;
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (h0 + i < heads) {
      if (p.rotates) rotate_part<T>(p, g.inter, x[i], y[i]);
      if (bad) x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
      if (store) {
        T *d = dst + (static_cast<int64_t>(i) << g.ps_shift) * kD;
        *reinterpret_cast<uint4 *>(d + 8 * p.c0) = x[i];
        *reinterpret_cast<uint4 *>(d + 8 * p.c1) = y[i];
      }
      if (out != nullptr) {
        T *o = out + (row * heads + h0 + i) * kD;
        *reinterpret_cast<uint4 *>(o + 8 * p.c0) = x[i];
        *reinterpret_cast<uint4 *>(o + 8 * p.c1) = y[i];
      }
    }
  }
}

int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

}  // namespace

cudaError_t launch_dense_prep(const isoquant_ctx *ctx, const isoquant_dense_cache *cache, const void *k,
                              const void *v, int n_tok, const int64_t *slot_mapping, const int64_t *k_pos,
                              const void *q, int dtype, int n_rows, int num_q_heads, const int64_t *q_pos,
                              const isoquant_rope *rope, void *k_out, void *q_out, cudaStream_t stream) {
  DensePrepArgs g{};
  g.k = k; g.v = v; g.q = q; g.k_out = k_out; g.q_out = q_out;
  g.slots = slot_mapping; g.k_pos = k_pos; g.q_pos = q_pos;
  if (cache != nullptr) {
    g.data = cache->data;
    g.num_pages = cache->num_pages;
    g.ps_shift = shift_of(cache->page_size);
  }
  if (rope != nullptr) {
    g.table = rope->cos_sin;
    g.num_pos = rope->num_positions;
    g.rot = rope->rot_dim;
    g.inter = rope->interleaved;
  }
  g.n_tok = n_tok; g.n_rows = n_rows; g.H = ctx->num_kv_heads; g.Hq = num_q_heads;
  g.status = ctx->status;
  // four heads per item where that still fills the SMs with work
  const int64_t vectors = static_cast<int64_t>(n_rows) * g.Hq + 2 * static_cast<int64_t>(n_tok) * g.H;
  const int hc = vectors * 8 >= static_cast<int64_t>(ctx->num_sms) * 2048 * 4 ? 4 : 1;
  g.q_items = static_cast<uint32_t>(n_rows) * ((g.Hq + hc - 1) / hc);
  g.k_items = static_cast<uint32_t>(n_tok) * ((g.H + hc - 1) / hc);
  const int64_t items = static_cast<int64_t>(g.q_items) + (cache != nullptr ? 2 : 1) * static_cast<int64_t>(g.k_items);
  const dim3 grid(static_cast<unsigned>((items + 31) / 32)), block(256);
  if (dtype == ISOQUANT_BF16)
    return hc == 4 ? launch_pdl(k_dense_prep<__nv_bfloat16, 4>, grid, block, 0, stream, g)
                   : launch_pdl(k_dense_prep<__nv_bfloat16, 1>, grid, block, 0, stream, g);
  return hc == 4 ? launch_pdl(k_dense_prep<__half, 4>, grid, block, 0, stream, g)
                 : launch_pdl(k_dense_prep<__half, 1>, grid, block, 0, stream, g);
}

}  // namespace isoquant
