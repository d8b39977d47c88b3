// attend16.cu -- attention on 16-bit queries, keys and values, head dim 128:
// isoquant_prompt_attend (packed prompts to themselves) and
// isoquant_dense_attend (newest tokens over the paged 16-bit cache, split over
// the context and joined).
//
// A row tile is up to 128 query rows of one KV head: `tok` consecutive tokens
// times the group's heads, so that the heads that share keys share each key
// tile.  Keys and values come as tiles of 128 tokens.  k_attend16 (prompts, and
// more than 64 rows over the cache), for a tile: S = Q K^T (8 products of 16
// dims), an online softmax of S's rows, O += P V (8 products of 16 tokens).
//   * S[128 x 128] fp32 sits in tensor memory, lane = row.  A softmax thread
//     owns a row: it takes its 128 scores into registers, and writes the
//     weights P (16-bit pairs) over S's columns, from where they are the A
//     operand of P V: neither S nor P passes through shared memory.
//   * Two S/P/O sets ("sides"), each with a warpgroup of softmax threads, so
//     that the tensor cores work for one side while the other's softmax runs.
//     Prompts: the sides are two neighbouring row tiles that share the key
//     tiles.  Cache: the sides take alternate key tiles of the same rows
//     and are merged at the end of the sequence's part.
//   * A warp per side issues the side's products in the order S(i), PV(i),
//     S(i + 1), so a completed S(i + 1) also says that PV(i) is done, and a
//     softmax thread may rescale its O row then.  The two warps take turns: a
//     warp's waits overlap the other's products, and the sides' products do
//     not interleave (prompt of 8192 tokens: 500 us with turns, 630 without,
//     490 to 530 with one warp for both, whose waits the tensor cores idle for).
//   * Weights are taken against a reference that may lag behind the row's
//     maximum.  Only when a tile's weights sum to more than 2^8 (2^15 in fp16's
//     form, scaled by 2^7) the row's maximum is computed, the tile redone and
//     O rescaled; sums are fp32, so a lagging reference loses nothing, and
//     most tiles need no maximum (7.96 -> 7.25 ms for a prompt of 32768).
//   * A loader warp brings Q, K and V by TMA with the 128-byte swizzle that the
//     products read, into a ring of 32 KB slots.  Over prompts it also takes
//     the work of CTAs that have not started (cluster launch control), so that
//     the next piece's loads overlap this one's epilogue.
//   * A guard warp sees, before they are used, to value tiles that not every
//     row sees whole: rows behind the last visible token are cleared
//     (neighbouring sequences, padding, stale pages: 0 x NaN would be NaN) and
//     non-finite elements taken out; the rows that do see such an element get
//     it added at the end.  Of tokens that every row sees they stay in: a sum
//     that comes out NaN is looked up in the values then.
// Prompts of 32768 tokens, 32 and 8 heads: 1040 (power-capped) to 1240 TFLOP/s.  What bounds
// it: the products' issue.  In isolation the 16 products of a side and tile
// take 1027 cycles; here 1690, their warps sharing issue slots and tensor
// memory with the softmax (removing the exponentials gains 3 %, the copies 2 %).
// Weights keep 8 bits (bf16) or 11 (fp16) in the prompts' product with V: a
// second operand for the remainders would be half as many products again.
// Over the cache, which is bound by its bytes, bf16 weights keep 16; fp16's 11
// are off by no more than the result's own rounding.
// All waits are bounded; after one expires every role leaves its loop.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "isoquant_internal.cuh"
#include "tcgen05.cuh"

namespace isoquant {
namespace {

constexpr int kTile = 128;                  // rows of a row tile, tokens of a key tile
constexpr int kTileBytes = kTile * kD * 2;  // 32 KB
constexpr int kMaxSlots = 5;
// warps 0 and 1 issue products, then these, then the sides' softmax warps
constexpr int kLoadWarp = 2, kGuardWarp = 3;
constexpr int kKeySlots = 2;                // of a ring; the others hold values
constexpr int kRowSlots = 5;                // of k_attend16
constexpr int kThreads16 = 3 * 128;         // k_attend16: two sides
// shared memory behind the tiles
constexpr int kOffBad = 0;                      // first token with +inf, -inf, NaN of each dim
constexpr int kOffBar = kOffBad + 3 * kD * 4;   // barriers
constexpr int kOffFlags = kOffBar + 304;
constexpr int kOffLoc = kOffFlags + 48;         // cache: the CTA's part, then locate's scratch; prompts: two jobs
constexpr int kTailBytes = kOffLoc + 160;
constexpr int kOffMl = kTailBytes;              // k_attend16: side 1's (reference, sum) of each row

struct Attend16 {
  int H, Hq, G, GB, chunks, tok, R, B, nq, causal;  // GB: heads of a row tile (G, or 128 of a larger group)
  int rts;                                          // cache: row tiles of a sequence and KV head
  int sides;                                        // prompts: row tiles of a job (1: the sides share its key tiles)
  float c;                                          // softmax scale * log2(e)
  const int32_t *cu;                                // prompts
  int n_tok;
  const int32_t *page_table, *seq_lens;             // cache
  int max_pages, num_pages, ps_shift;
  const uint16_t *values;                           // the cache, or the prompts' V with tokens v_stride apart
  int64_t v_stride;
  float *records;
  int2 *plan;
  int n_cta, row_stride;                            // records: rows rounded up to 2
  int slots, q_half;                                // ring slots, bytes of a 64-dim half of a Q buffer
  void *out;
  uint32_t *status;
  int device;
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// maximum of three that keeps a NaN
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ __nv_bfloat16 to16(float x, __nv_bfloat16) { return __float2bfloat16_rn(x); }
__device__ __forceinline__ __half to16(float x, __half) { return __float2half_rn(x); }
// A sum without the non-finite values that guard_tile took out of dim d: with
// those that a row seeing `lim` tokens sees.
__device__ __forceinline__ float with_nonfinite(float o, const int *bad, int d, int lim) {
  if (bad[d] < lim) o += INFINITY;
  if (bad[kD + d] < lim) o -= INFINITY;
  return bad[2 * kD + d] < lim ? NAN : o;
}

__device__ __forceinline__ void fetch_map(const CUtensorMap &map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
}

// shared-memory matrix descriptor, 128-byte swizzle, strides in 16-byte units
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lbo) << 16) |
         (static_cast<uint64_t>(sbo) << 32) | (1ull << 46) | (2ull << 61);
}
// no swizzle: 8 x 16-byte pieces, `lbo` and `sbo` units apart along the two axes
__device__ __forceinline__ uint64_t desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lbo) << 16) |
         (static_cast<uint64_t>(sbo) << 32) | (1ull << 46);
}
// A, B of type T (bf16 or fp16, both the same), fp32 accumulator, 128 x n;
// mn: the operand's 16-bit elements run along M or N, not K
template <typename T>
__device__ constexpr uint32_t idesc16(int n, int a_mn, int b_mn) {
  constexpr uint32_t t = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | ((static_cast<uint32_t>(n) >> 3) << 17) | ((128u >> 4) << 24);
}
// The whole warp runs the issuing code; the thread with `issue` set issues.
// Only a descriptor's low word changes from product to product (addresses stay
// below 2^18), so the high words are converted once: the fewer instructions
// a product takes, the less its warp's neighbours delay it.
__device__ __forceinline__ void mma_ss(uint32_t issue, uint32_t d, uint64_t a, uint32_t a_add, uint64_t b,
                                       uint32_t b_add, uint32_t idesc, uint32_t acc) {
  const uint32_t al = static_cast<uint32_t>(a) + a_add, ah = static_cast<uint32_t>(a >> 32);
  const uint32_t bl = static_cast<uint32_t>(b) + b_add, bh = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %8, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, {%7, %7, %7, %7}, p;\n\t}\n" ::"r"(d),
      "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"(acc), "r"(0u), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t issue, uint32_t d, uint32_t a, uint64_t b, uint32_t b_add,
                                       uint32_t idesc, uint32_t acc) {
  const uint32_t bl = static_cast<uint32_t>(b) + b_add, bh = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, {%6, %6, %6, %6}, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(bl), "r"(bh), "r"(idesc), "r"(acc), "r"(0u), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// Asks the hardware for a CTA of this grid that has not started (it then never
// will); the answer's 16 bytes complete on `bar`.  One thread.
__device__ __forceinline__ void steal_request(uint4 *answer, uint64_t *bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_addr(answer)),
               "r"(smem_addr(bar))
               : "memory");
}
// the answer: false if none was left, else the block's index
__device__ __forceinline__ bool steal_answer(const uint4 *answer, uint32_t &block) {
  const uint64_t lo = reinterpret_cast<const volatile uint64_t *>(answer)[0],
                 hi = reinterpret_cast<const volatile uint64_t *>(answer)[1];
  uint32_t got, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n mov.b128 r, {%2, %3};\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(got), "=r"(x)
      : "l"(lo), "l"(hi));
  block = x;
  return got != 0;
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// The reference passed by 2^kLazy moves; fp16 weights are held times 2^7 so
// that those far below the maximum keep their bits (2^15 at most).
constexpr float kLazy = 8.f;
// The reference is kept as the score itself: c s - (c times reference rounded)
// is off by that rounding, up to 2^9 for logarithms of 2^33.  It scales a row's
// weights alike, so it cancels while it fits the exponents; from here on the
// difference of the scores is taken first.
constexpr float kLarge = 1048576.f;  // rounded within 2^-4
template <typename T>
constexpr float kShift = std::is_same<T, __half>::value ? 7.f : 0.f;

// One key tile of a softmax thread's row: scores at tensor-memory columns ts,
// of which the first `vis` count, become weights 2^(c (s - ref)) at the same
// columns; with kLo the weights' remainders follow as a second operand.
// any_large: whether a row of the warp has a large reference.
template <typename T, bool kLo>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, float c, int vis, bool first, float &ref,
                                             float &l, bool &any_large) {
  constexpr float kMost = kShift<T> == 0.f ? 256.f : 32768.f;  // 2^(8 + shift)
  const float2 c2 = make_float2(c, c);
  float sum;
  uint32_t w[64], e[kLo ? 64 : 1];
  bool move = first || (ref == -INFINITY && vis > 0), moved = move, again = __any_sync(0xffffffffu, move);
  while (true) {
    float s[4][32];
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_ld32_async(ts + 32 * k, s[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_arrived(s[k]);
    if (__any_sync(0xffffffffu, vis < kTile)) {
#pragma unroll
      for (int i = 0; i < kTile; ++i)
        if (i >= vis) s[i >> 5][i & 31] = -INFINITY;
    }
    if (again) {
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kTile; i += 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = max3_nan(mx[j], s[i >> 5][(i + j) & 31], s[i >> 5][(i + j + 4) & 31]);
      }
      const float mt = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]);
      const bool up = move && !(mt <= ref);
      const float corr = up ? ex2f((ref - mt) * c) : 1.f;
      if (up) ref = mt;
      any_large = __any_sync(0xffffffffu, fabsf(ref * c) > kLarge && ref != -INFINITY);
      l *= corr;
      if (!first) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float o[32];
          tmem_ld32(to + 32 * k, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= corr;
          tmem_st32(to + 32 * k, o);
        }
      }
    }
    // (NaN for a NaN or +inf)
    float sub = ref == -INFINITY ? 0.f : (ref * c - kShift<T>) + (ref - ref);
    if (any_large) {
      const float off = ref == -INFINITY ? 0.f : -ref;
      sub = -kShift<T>;
#pragma unroll
      for (int i = 0; i < kTile; i += 2) {
        const float2 v = __fadd2_rn(make_float2(s[i >> 5][i & 31], s[i >> 5][(i & 31) + 1]), make_float2(off, off));
        s[i >> 5][i & 31] = v.x;
        s[i >> 5][(i & 31) + 1] = v.y;
      }
    }
    const float2 n2 = make_float2(-sub, -sub);
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < kTile; i += 2) {
      const float2 y = __ffma2_rn(make_float2(s[i >> 5][i & 31], s[i >> 5][(i & 31) + 1]), c2, n2);
      const float2 p = make_float2(ex2f(y.x), ex2f(y.y));
      part[(i >> 1) & 1] = __fadd2_rn(part[(i >> 1) & 1], p);
      const uint32_t hi = pack16(p.x, p.y, T());
      w[i >> 1] = hi;
      if constexpr (kLo) e[i >> 1] = pack16(p.x - __uint_as_float(hi << 16), p.y - __uint_as_float(hi & 0xffff0000u), T());
    }
    sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
    move = !moved && !(sum <= kMost);  // a NaN moves too
    moved |= move;
    again = __any_sync(0xffffffffu, move);
    if (!again) break;
  }
  l += sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t part[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) part[i] = w[16 * k + i];
    tmem_st16u(ts + 16 * k, part);
    if constexpr (kLo) {
#pragma unroll
      for (int i = 0; i < 16; ++i) part[i] = e[16 * k + i];
      tmem_st16u(ts + 64 + 16 * k, part);
    }
  }
  tmem_stored();
}

// ---------------------------------------------------------------- the work
// A segment: one sequence's (row tile, KV head) and a run of its key tiles.
struct Segment {
  int b, h;
  int row0;         // first token of the row tile (of side 0) in its sequence's queries
  int chunk;        // heads chunk * 128 .. of a group above 128
  int kv0;          // prompts: first token of the sequence
  int rows;         // prompts: tokens of the sequence; cache: nq
  int shift;        // row of query token i sees tokens below i + shift (causal)
  int cap;          // no row sees more
  int j0, n[2];     // first key tile, tiles of each side (cache: n[0] = all, split even and odd)
  int id;           // cache: segment number
  bool whole;       // cache: all of the sequence's tiles
  bool starts;      // cache: from tile 0
  // tokens that query token i sees
  __device__ int limit(int i, int causal) const { return causal ? max(0, min(cap, i + shift)) : cap; }
};

// cache: tiles of a row tile (one at least: its rows have to be written)
struct Unit {
  int b, rt, L, cap, row0, chunk, nt;
  __device__ void set(const Attend16 &p, int u) {
    b = p.rts == 1 ? u : u / p.rts;
    rt = u - b * p.rts;
    L = p.seq_lens[b];
    // (places behind a row's last tile are counted in 32 bits too)
    const int64_t room = min(static_cast<int64_t>(p.max_pages) << p.ps_shift, static_cast<int64_t>(INT_MAX - 2 * kTile));
    cap = max(0, static_cast<int>(min(static_cast<int64_t>(L), room)));
    row0 = p.chunks == 1 ? rt * p.tok : rt / p.chunks * p.tok;
    chunk = p.chunks == 1 ? 0 : rt % p.chunks;
    const int last = min(p.nq, row0 + p.tok) - 1;
    const int64_t hz = p.causal ? min(static_cast<int64_t>(cap), static_cast<int64_t>(L) - p.nq + last + 1) : cap;
    nt = max(1, static_cast<int>((hz + kTile - 1) / kTile));
  }
};

// a / b for a >= 0, b > 0: 32-bit division where it does (a 64-bit one takes
// some hundred cycles, and a call of few tiles waits for a handful of them)
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The CTA's part [gs, ge) of all tiles, and the (unit, tile offset) where it
// starts.  loc: {gs, ge, unit, offset, total}; ends with __syncthreads.
template <int NT>
__device__ void locate16(const Attend16 &p, int64_t *loc, int64_t *scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int U = p.B * p.rts;
  const int u0 = static_cast<int>(div64(static_cast<int64_t>(U) * tid, NT)),
            u1 = static_cast<int>(div64(static_cast<int64_t>(U) * (tid + 1), NT));
  int64_t mine = 0;
  Unit un;
  for (int u = u0; u < u1; ++u) {
    un.set(p, u);
    mine += static_cast<int64_t>(un.nt) * p.H;
    if (blockIdx.x == 0 && un.cap < un.L) set_status(p.status, ISOQUANT_DEVERR_PAGE_RANGE);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const int64_t excl = before + incl - mine;
  const int64_t N = min(static_cast<int64_t>(p.n_cta), total), c = blockIdx.x;
  const int64_t gs = c < N ? div64(total * c, N) : 0, ge = c < N ? div64(total * (c + 1), N) : 0;
  if (tid == 0) {
    loc[0] = gs;
    loc[1] = ge;
    loc[4] = total;
  }
  if (gs < ge && excl <= gs && gs < excl + mine) {
    int64_t run = excl;
    for (int u = u0; u < u1; ++u) {
      un.set(p, u);
      const int64_t n = static_cast<int64_t>(un.nt) * p.H;
      if (gs < run + n) {
        loc[2] = u;
        loc[3] = gs - run;
        break;
      }
      run += n;
    }
  }
  __syncthreads();
}

// cache: the segments of a CTA's part, in the same order for every role
struct Walk16 {
  int64_t g, ge;
  Unit un;
  int u, h, j;
  __device__ Walk16(const Attend16 &p, const int64_t *loc) {
    g = loc[0];
    ge = loc[1];
    if (g < ge) {
      u = static_cast<int>(loc[2]);
      un.set(p, u);
      h = static_cast<int>(div64(loc[3], un.nt));
      j = static_cast<int>(loc[3] - static_cast<int64_t>(h) * un.nt);
    }
  }
  __device__ bool next(const Attend16 &p, Segment &s) {
    if (g >= ge) return false;
    if (j == un.nt) {
      j = 0;
      if (++h == p.H) {
        h = 0;
        un.set(p, ++u);
      }
    }
    s.b = un.b;
    s.h = h;
    s.row0 = un.row0;
    s.chunk = un.chunk;
    s.kv0 = 0;
    s.rows = p.nq;
    s.shift = un.L - p.nq + 1;
    s.cap = un.cap;
    s.j0 = j;
    s.n[0] = static_cast<int>(min(static_cast<int64_t>(un.nt - j), ge - g));
    s.n[1] = 0;
    s.id = u * p.H + h;
    s.starts = j == 0;
    j += s.n[0];
    g += s.n[0];
    s.whole = s.starts && j == un.nt;
    return true;
  }
};

// prompts: sequence and pair of row tiles of a job, found by one warp.  The KV
// heads of a pair are next to one another.  Up to 32 sequences: the pairs with
// the most keys first, so that what ends last is short (16 ragged prompts of 1
// to 511 tokens: 39 -> 35 us); more: sequence by sequence, each from its last pair (the most
// keys) to its first, found by reading the bounds from the front (1000 prompts
// of 1 to 64 tokens: 0.7 us each, 4000: 2.4, 100: 0.35).  false: no work.
__device__ bool find_prompt(const Attend16 &p, uint32_t job, Segment &s) {
  const int lane = threadIdx.x & 31;
  const int item = static_cast<int>(job / p.H);
  s.h = static_cast<int>(job % p.H);
  int before = 0, highest = 0;
  bool found = false;
  for (int b0 = 0; b0 < p.B && (!found || job == 0); b0 += 32) {  // job 0 looks at all bounds
    const int b = b0 + lane;
    const int x = b < p.B ? p.cu[b] : 0, y = b < p.B ? p.cu[b + 1] : 0;
    // the sequences lie one behind another: none starts before an earlier bound
    int top = b < p.B ? x : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, top, o);
      if (lane >= o) top = max(top, t);
    }
    const int earlier = max(highest, top);
    const bool good = x >= 0 && y >= x && y <= p.n_tok && x >= earlier;
    if (b < p.B && !good && job == 0) set_status(p.status, ISOQUANT_DEVERR_SEQ_RANGE);
    const int pairs = b < p.B && good ? (y - x + p.sides * p.tok - 1) / (p.sides * p.tok) : 0;
    if (p.B <= 32) {
      if (item >= __reduce_add_sync(0xffffffffu, pairs)) return false;
      int pair = 0;
      bool mine;
      if (p.causal) {
        // the highest place t so that more than `item` pairs stand at t or above
        int t = 0, high = __reduce_max_sync(0xffffffffu, pairs);
        while (high - t > 1) {
          const int mid = (t + high) >> 1;
          if (__reduce_add_sync(0xffffffffu, max(0, pairs - mid)) > item) t = mid;
          else high = mid;
        }
        const int rank = item - __reduce_add_sync(0xffffffffu, max(0, pairs - t - 1));
        const unsigned there = __ballot_sync(0xffffffffu, pairs > t);
        mine = pairs > t && __popc(there & ((1u << lane) - 1u)) == rank;
        pair = t;
      } else {
        int before_me = 0;  // pairs of longer sequences
        for (int j = 0; j < p.B; ++j) {
          const int other = __shfl_sync(0xffffffffu, pairs, j);
          if (other > pairs || (other == pairs && j < lane)) before_me += other;
        }
        mine = item >= before_me && item < before_me + pairs;
        pair = item - before_me;
      }
      const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      s.b = src;
      s.kv0 = __shfl_sync(0xffffffffu, x, src);
      s.rows = __shfl_sync(0xffffffffu, y - x, src);
      s.row0 = __shfl_sync(0xffffffffu, pair, src) * p.sides * p.tok;
      found = true;
      break;
    }
    int incl = pairs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int first = before + incl - pairs;
    const unsigned hit = __ballot_sync(0xffffffffu, item >= first && item < first + pairs);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s.b = b0 + src;
      s.kv0 = __shfl_sync(0xffffffffu, x, src);
      s.rows = __shfl_sync(0xffffffffu, y - x, src);
      const int pair = __shfl_sync(0xffffffffu, first + pairs - 1 - item, src);
      s.row0 = pair * p.sides * p.tok;
      found = true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    highest = max(highest, __shfl_sync(0xffffffffu, max(top, y), 31));
  }
  if (!found) return false;
  s.chunk = 0;
  s.shift = 1;
  s.cap = s.rows;
  s.j0 = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int lo = s.row0 + x * p.tok, hi = min(s.rows, lo + p.tok);
    s.n[x] = x < p.sides && lo < s.rows ? ((p.causal ? hi : s.rows) + kTile - 1) / kTile : 0;
  }
  if (p.sides == 1) {
    s.n[1] = s.n[0] >> 1;
    s.n[0] -= s.n[1];
  }
  return true;
}

// 16-bit patterns whose exponent is all ones
template <typename T>
__device__ __forceinline__ uint32_t exponent_mask() {
  return std::is_same<T, __nv_bfloat16>::value ? 0x7F807F80u : 0x7C007C00u;
}

// The non-finite values of a head's tokens [t0, end), all of them in the
// sequence: lane l has dims 8 (l mod 16) .. + 7, three bits a dim (+inf, -inf,
// NaN).  The products lose an infinity where its weight, or a bf16 weight's
// remainder, is zero or negative (0 x inf); a sum that came out NaN looks here
// what it should be.  Rare, and kept out of line so that it costs the loops
// nothing; one whole warp.  values: the head's first value vector, of token 0 or
// page 0; stride: elements from token to token, or page to page.
template <bool kPaged>
__device__ __noinline__ uint32_t values_seen(const int32_t *pages, int num_pages, int ps_shift,
                                             const uint16_t *values, int64_t stride, int t0, int end, uint32_t mask) {
  const int lane = threadIdx.x & 31;
  values += 8 * (lane & 15);
  constexpr int kAtOnce = 8;
  constexpr uint32_t kNans = 0x924924u;  // a lane's dims all NaN: no token changes that
  uint32_t kinds = 0;
  for (int first = t0; first < end && !__all_sync(0xffffffffu, (kinds & kNans) == kNans); first += 2 * kAtOnce) {
    uint4 v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int t = first + 2 * i + (lane >> 4);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (t < end) {
        int64_t at = t * stride;
        if constexpr (kPaged) {
          const int page = pages[t >> ps_shift];
          at = (page < 0 || page >= num_pages ? 0 : page * stride) + (t & ((1 << ps_shift) - 1)) * kD;
        }
        v[i] = *reinterpret_cast<const uint4 *>(values + at);
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t x = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
        if ((x & mask) == mask) kinds |= ((x & 0x7fffu) != mask ? 4u : 1u << (x >> 15)) << (3 * e);
      }
    }
    kinds |= __shfl_xor_sync(0xffffffffu, kinds, 16);
  }
  return kinds;
}
template <typename T, bool kPaged>
__device__ __forceinline__ uint32_t values_seen(const Attend16 &p, const Segment &s, int t0, int end) {
  const uint32_t mask = exponent_mask<T>() & 0xffffu;
  if constexpr (kPaged)
    return values_seen<true>(p.page_table + static_cast<int64_t>(s.b) * p.max_pages, p.num_pages, p.ps_shift,
                             p.values + (static_cast<int64_t>(p.H + s.h) << p.ps_shift) * kD,
                             (static_cast<int64_t>(2 * p.H) << p.ps_shift) * kD, t0, end, mask);
  else
    return values_seen<false>(nullptr, 0, 0, p.values + s.kv0 * p.v_stride + static_cast<int64_t>(s.h) * kD,
                              p.v_stride, t0, end, mask);
}
// dim d's three bits of what values_seen returned
__device__ __forceinline__ uint32_t kinds_of(uint32_t seen, int d) {
  return (__shfl_sync(0xffffffffu, seen, d >> 3) >> (3 * (d & 7))) & 7u;
}
__device__ __forceinline__ float nonfinite_sum(uint32_t kinds) {
  return kinds == 1u ? INFINITY : kinds == 2u ? -INFINITY : NAN;
}

// Every wait of a warp: false once it, or any other of the CTA, gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Attend16 &p, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.status, abort));
}

// The barriers of a CTA: ring slots filled (for a tile that the guard sees to
// first: loaded), freed; queries there and used; a side's or tile's scores
// there and read, weights, products; the sides' hand-overs; all products.
struct Bars {
  uint64_t full[kMaxSlots], loaded[kMaxSlots], freed[kMaxSlots];
  uint64_t q_full[2], q_free[2], s_full[2], s_free[2], p_full[2], o_done[2], turn[2], job_full[2], job_free[2];
  uint64_t side1, seg_done, mma_done, stolen;
  __device__ void init(int slot_users, int q_users, int p_count, int seg_count, int readers) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&loaded[i], 1);
      mbar_init(&freed[i], slot_users);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], q_users);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], p_count);
      mbar_init(&p_full[i], p_count);
      mbar_init(&o_done[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&job_full[i], 1);
      mbar_init(&job_free[i], readers);
    }
    mbar_init(&side1, seg_count);
    mbar_init(&seg_done, seg_count);
    mbar_init(&mma_done, 2);
    mbar_init(&stolen, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
};
static_assert(sizeof(Bars) <= 304, "room for the barriers");
// A prompt's piece of work as the loader hands it to the other warps.
struct Job {
  int kv0, rows, row0, h, n0, n1, end, pad;
};
// what the roles of a CTA share beside the barriers
struct Flags {
  uint32_t tmem;
  int abort;
  int nonfinite;  // the segment, counted from 1, that the guard's marks belong to
  // Segments behind each reader of the marks: a softmax warp of k_attend16, a
  // side of k_cols16.  Each has a count of its own: readers are up to two
  // segments apart (one without tiles of a segment passes it at once), so a
  // sum would let one stand for another.
  int done[8];
};
static_assert(sizeof(Flags) <= 48, "room for the flags");

// The ring: tile t's keys lie in slot t mod kKeySlots, its values in one of the
// other slots in turn.  use: how often the slot was used before.
__device__ __forceinline__ uint32_t key_slot(uint32_t t) { return t % kKeySlots; }
__device__ __forceinline__ uint32_t key_use(uint32_t t) { return t / kKeySlots; }
__device__ __forceinline__ uint32_t value_slot(uint32_t t, int slots) { return kKeySlots + t % (slots - kKeySlots); }
__device__ __forceinline__ uint32_t value_use(uint32_t t, int slots) { return t / (slots - kKeySlots); }

__device__ __forceinline__ float *record(const Attend16 &p, int i) {
  return p.records + i * (static_cast<int64_t>(p.row_stride) * (kD + 2));
}

// Tensor memory of COLS columns, the barriers and the guard's marks; the
// caller's next __syncthreads makes them visible.
template <uint32_t COLS>
__device__ __forceinline__ void start_cta(Bars &bars, Flags *flags, int *bad, int slot_users, int q_users,
                                          int p_count, int seg_count, int readers) {
  if (threadIdx.x < 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&flags->tmem)),
                 "r"(COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
    tc_fence_before();
  }
  if (threadIdx.x == 32) {
    bars.init(slot_users, q_users, p_count, seg_count, readers);
    flags->abort = flags->nonfinite = 0;
    for (int i = 0; i < 8; ++i) flags->done[i] = 0;
  }
  for (int i = threadIdx.x; i < 3 * kD; i += blockDim.x) bad[i] = INT_MAX;
}
// the products must complete before tensor memory is released
template <uint32_t COLS>
__device__ __forceinline__ void end_cta(Bars &bars, Flags *flags, const Attend16 &p) {
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    mbar_wait(&bars.mma_done, 0, p.status, nullptr);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(flags->tmem), "r"(COLS));
  }
}

// f(segment, number) for each segment of the CTA's part, until f says stop
template <typename F>
__device__ __forceinline__ void cache_segments(const Attend16 &p, const int64_t *loc, F &&f) {
  Walk16 wk(p, loc);
  Segment s;
  for (uint32_t k = 0; wk.next(p, s); ++k)
    if (!f(s, k)) return;
}
// the token below which every row of the segment sees all, and the first that none sees
__device__ __forceinline__ int all_see(const Attend16 &p, const Segment &s) { return s.limit(s.row0, p.causal); }
__device__ __forceinline__ int none_sees(const Attend16 &p, const Segment &s, int tokens) {
  return s.limit(min(s.rows, s.row0 + tokens) - 1, p.causal);
}

// The loader warp's ring: begin() waits until a slot is free and says which
// barrier the tile's copies complete on.
struct Loader {
  const Attend16 &p;
  Bars &bars;
  volatile int *abort;
  bool ok = true;
  // lane i: slot i's uses, those that the guard sees to, and whether the last was one
  uint32_t uses = 0, guards = 0;
  bool guarded = false;
  uint32_t queries = 0;  // lane i: loads into query buffer i
  __device__ Loader(const Attend16 &p_, Bars &b, volatile int *a) : p(p_), bars(b), abort(a) {}
  __device__ uint64_t *begin(uint32_t slot, uint32_t use, bool guard, uint32_t bytes) {
    if (use > 0) ok = ok && warp_wait(&bars.freed[slot], (use - 1) & 1u, p, abort);
    if (!ok) return nullptr;
    const uint32_t lane = threadIdx.x & 31;
    uint64_t *bar = guard ? &bars.loaded[slot] : &bars.full[slot];
    if (lane == slot) {
      guarded = guard;
      ++uses;
      guards += guard;
    }
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    return bar;
  }
  // Waits until query buffer qb, used `use` times before, is free: true for the
  // lane that loads it (box after box on bars.q_full[qb]).
  __device__ bool begin_queries(uint32_t qb, uint32_t use) {
    if (use > 0) ok = ok && warp_wait(&bars.q_free[qb], (use - 1) & 1u, p, abort);
    const uint32_t lane = threadIdx.x & 31;
    if (ok && lane == qb) ++queries;
    if (ok && lane == 0) mbar_arrive_expect_tx(&bars.q_full[qb], static_cast<uint32_t>(p.R * kD * 2));
    return ok && lane == 0;
  }
  // The last copies have landed before the CTA ends, whoever of it gave up (else
  // those that use them wait for them anyway).
  __device__ void drain() {
    const uint32_t lane = threadIdx.x & 31, n = guarded ? guards : uses;
    if (n > 0) mbar_wait(guarded ? &bars.loaded[lane] : &bars.full[lane], (n - 1) & 1u, p.status, nullptr);
    if (queries > 0) mbar_wait(&bars.q_full[lane], (queries - 1) & 1u, p.status, nullptr);
    __syncwarp();
  }
};

// Tokens of a copied box, which a page of any size holds whole (16 x 32768
// tokens: 8 tokens a box 287 us, 16 188, 32 162, 128 161).
constexpr int kBox = 32;
// The loader warp over the cache: the segments' queries into q_bufs buffers
// whose 64-dim halves are p.q_half bytes, key and value tiles into the ring.
__device__ void load_cache(const Attend16 &p, const int64_t *loc, const CUtensorMap &mq, const CUtensorMap &mk,
                           uint32_t sq, uint32_t sr, int q_bufs, Bars &bars, volatile int *abort) {
  const int lane = threadIdx.x & 31;
  Loader ld(p, bars, abort);
  uint32_t t = 0;  // tiles so far
  cache_segments(p, loc, [&](const Segment &s, uint32_t k) {
    const uint32_t qb = k % q_bufs;
    if (ld.begin_queries(qb, k / q_bufs)) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        tma_3d(sq + (2 * qb + hf) * p.q_half, &mq, 64 * hf, s.h * p.G + s.chunk * kTile, s.b * p.nq + s.row0,
               &bars.q_full[qb]);
    }
    __syncwarp();
    const int end = none_sees(p, s, p.tok), all = all_see(p, s);
    // lane 2 i + hf loads half hf of the tile's i-th box
    constexpr int box = kBox, boxes = kTile / box;
    const int hf = lane & 1, part = lane >> 1;
    auto page_of = [&](int i) {  // this lane's page of tile i: -1 if nothing of it is seen, -2 if it is none
      const int at = (s.j0 + i) * kTile + part * box;
      if (i >= s.n[0] || part >= boxes || at >= end) return -1;
      const int page = p.page_table[static_cast<int64_t>(s.b) * p.max_pages + (at >> p.ps_shift)];
      return page < 0 || page >= p.num_pages ? -2 : page;
    };
    int ahead = page_of(0);
    for (int i = 0; i < s.n[0] && ld.ok; ++i, ++t) {
      int page = ahead;
      ahead = page_of(i + 1);
      if (page == -2) {
        set_status(p.status, ISOQUANT_DEVERR_PAGE_RANGE);
        page = 0;
      }
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * box * 128u;
      const int t0 = (s.j0 + i) * kTile;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t sl = kv ? value_slot(t, p.slots) : key_slot(t);
        uint64_t *bar = ld.begin(sl, kv ? value_use(t, p.slots) : key_use(t), kv && t0 + kTile > all, bytes);
        if (page >= 0 && ld.ok) {
          // one row per token: below 2^31 rows, checked on the host
          const int off = (t0 + part * box) & ((1 << p.ps_shift) - 1);
          const int row = ((page * 2 + kv) * p.H + s.h) * (1 << p.ps_shift) + off;
          tma_2d(sr + sl * kTileBytes + hf * (kTileBytes / 2) + part * box * 128, &mk, 64 * hf, row, bar);
        }
        __syncwarp();
      }
    }
    return ld.ok;
  });
  ld.drain();
}

// The guard warp on a value tile (tokens from t0 on) of segment k: rows that
// no query row sees are cleared, non-finite elements of rows that some see
// are taken out and their first token noted for this segment.  readers: bit i
// set if done[i] counts a reader of the marks.  false: gave up waiting.
template <typename T>
__device__ __forceinline__ bool guard_tile(const Attend16 &p, uint8_t *tile, int t0, int all, int none, int k,
                                           uint32_t readers, int *bad, Flags *flags) {
  const uint32_t mask = exponent_mask<T>();
  const int lane = threadIdx.x & 31;
  auto at = [&](int r) {  // this lane's 16 bytes of row r
    const int c = lane & 15;
    return reinterpret_cast<uint4 *>(tile + (c >> 3) * (kTileBytes / 2) + r * 128 + (c & 7) * 16);
  };
  bool any = false;
#pragma unroll 4
  for (int r = max(0, all - t0) + (lane >> 4); r < kTile; r += 2) {
    if (t0 + r >= none) {
      *at(r) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 v = *at(r);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        any |= (w[i] & mask & 0xffffu) == (mask & 0xffffu) || (w[i] & mask & 0xffff0000u) == (mask & 0xffff0000u);
    }
  }
  if (!__any_sync(0xffffffffu, any)) return true;
  // rare: an earlier segment's marks must have been read before they go
  volatile int *marked = &flags->nonfinite, *done = flags->done, *abort = &flags->abort;
  const int before = *marked;
  if (before != k + 1) {
    const bool reader = (readers >> lane) & 1u;
    const uint64_t start = global_ns();
    while (!__all_sync(0xffffffffu, !reader || done[lane] >= before)) {
      const bool late = global_ns() - start >= kWaitLimitNs;
      if (late) set_status(p.status, ISOQUANT_DEVERR_WAIT_TIMEOUT);
      if (late) *abort = 1;
      if (__any_sync(0xffffffffu, *abort != 0)) return false;
      __nanosleep(200);
    }
    for (int e = lane; e < 3 * kD; e += 32) bad[e] = INT_MAX;
    __syncwarp();
  }
  for (int r = max(0, all - t0) + (lane >> 4); r < min(kTile, none - t0); r += 2) {
    uint4 v = *at(r);
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
    // the chunk lies where the row's swizzle put it
    const int dim0 = ((lane & 15) >> 3) * 64 + (((lane & 7) ^ (r & 7)) * 8);
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu, m = mask & 0xffffu;
      if ((x & m) != m) continue;
      const int kind = (x & 0x7fffu) != m ? 2 : (x >> 15);
      atomicMin(&bad[kind * kD + dim0 + e], t0 + r);
      w[e >> 1] &= ~(0xffffu << (16 * (e & 1)));
    }
    *at(r) = v;
  }
  __syncwarp();
  if (lane == 0) *marked = k + 1;
  return true;
}

// A loaded tile: seen to, then handed on.  phases: bit i = parity of slot i's loads.
template <typename T>
__device__ __forceinline__ bool guard_slot(const Attend16 &p, uint32_t sl, uint32_t &phases, uint8_t *ring_base, int t0,
                                           int all, int none, int k, uint32_t readers, int *bad, Bars &bars,
                                           Flags *flags) {
  const bool ok = warp_wait(&bars.loaded[sl], (phases >> sl) & 1u, p, &flags->abort);
  phases ^= 1u << sl;
  if (!ok || !guard_tile<T>(p, ring_base + sl * kTileBytes, t0, all, none, k, readers, bad, flags)) return false;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.full[sl]);
  return true;
}

// The guard warp over the cache.
template <typename T>
__device__ void guard_cache(const Attend16 &p, const int64_t *loc, uint8_t *ring_base, uint32_t readers, int *bad,
                            Bars &bars, Flags *flags) {
  uint32_t phases = 0, t = 0;
  cache_segments(p, loc, [&](const Segment &s, uint32_t k) {
    const int all = all_see(p, s), none = none_sees(p, s, p.tok), n = s.n[0];
    bool ok = true;
    for (int i = max(0, all / kTile - s.j0); i < n && ok; ++i)
      ok = guard_slot<T>(p, value_slot(t + i, p.slots), phases, ring_base, (s.j0 + i) * kTile, all, none, k, readers,
                         bad, bars, flags);
    t += n;
    return ok;
  });
}

// The segment that starts in this CTA's part and goes on in the CTAs behind,
// for the combine kernel (one thread).
__device__ void write_plan(const Attend16 &p, const int64_t *loc) {
  const int64_t ge = loc[1], total = loc[4];
  int2 plan = make_int2(-1, 0);
  Walk16 wk(p, loc);
  Segment s;
  while (wk.next(p, s)) {
    if (s.starts && !s.whole) {
      const int64_t N = min(static_cast<int64_t>(p.n_cta), total);
      const int64_t last = ge + (wk.un.nt - wk.j) - 1;  // the segment's last tile
      plan = make_int2(s.id, static_cast<int>(div64((last + 1) * N + total - 1, total) - 1));
    }
  }
  p.plan[blockIdx.x] = plan;
}

// kPaged: the cache's form for more than 64 rows, else prompts.  kAlternate: the
// sides take alternate key tiles of the same rows (the cache, few prompts),
// else key tiles in common and rows of their own.  kLo: bf16
// weights as two operands (16 bits), so that the result is off by one rounding.
template <typename T, bool kPaged, bool kAlternate>
__global__ void __launch_bounds__(kThreads16, 1)
    k_attend16(const Attend16 p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv) {
  constexpr bool kLo = kPaged && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *ring_base = smem + 4 * p.q_half, *tail = ring_base + p.slots * kTileBytes;
  int *bad = reinterpret_cast<int *>(tail + kOffBad);
  float2 *ml = reinterpret_cast<float2 *>(tail + kOffMl);
  Bars &bars = *reinterpret_cast<Bars *>(tail + kOffBar);
  Flags *flags = reinterpret_cast<Flags *>(tail + kOffFlags);
  volatile int *abort = &flags->abort, *nonfinite = &flags->nonfinite;
  int64_t *loc = reinterpret_cast<int64_t *>(tail + kOffLoc);
  uint4 *stolen = reinterpret_cast<uint4 *>(tail + kOffLoc + 2 * sizeof(Job));
  const int row_warps = (p.R + 31) / 32;  // warps of a side that hold rows
  // a segment's key tiles
  auto tiles = [&](const Segment &s) {
    return kPaged ? s.n[0] : kAlternate ? s.n[0] + s.n[1] : max(s.n[0], s.n[1]);
  };

  start_cta<512>(bars, flags, bad, 2, kPaged ? 2 : 1, row_warps, row_warps, 3 + 2 * row_warps);
  if (tid == 64) {
    fetch_map(mq);
    fetch_map(mk);
    if (!kPaged) fetch_map(mv);
  }
  pdl_trigger();
  pdl_wait();
  if constexpr (kPaged) locate16<kThreads16>(p, loc, loc + 8);
  else __syncthreads();
  Job *jobs = reinterpret_cast<Job *>(loc);
  tc_fence_after();
  const uint32_t tmem = flags->tmem;
  auto for_segments = [&](auto &&f) {
    if constexpr (kPaged) {
      cache_segments(p, loc, f);
    } else {
      for (uint32_t k = 0;; ++k) {
        if (!warp_wait(&bars.job_full[k & 1], (k >> 1) & 1u, p, abort)) return;
        const Job jb = jobs[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.job_free[k & 1]);
        if (jb.end) return;
        Segment s{};
        s.h = jb.h;
        s.kv0 = jb.kv0;
        s.rows = s.cap = jb.rows;
        s.row0 = jb.row0;
        s.shift = 1;
        s.n[0] = jb.n0;
        s.n[1] = jb.n1;
        if (!f(s, k)) return;
      }
    }
  };

  // registers of the four helper warps go to the softmax threads:
  // 256 x 208 + 128 x 80 of the 384 x 168 at launch
  if (warp < 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------------------- products
    // Each side has a warp that issues its products: issuing takes as long as
    // the tensor cores need, so one warp's waits and commits would be time
    // that they idle (one issuing warp for both: 490 us for a prompt of 8192
    // tokens, 32 and 8 heads).
    const int x = warp;
    const uint32_t issue = lane == 0;
    uint32_t n_p = 0, n_q = 0, t = 0, n_turn = 0;  // weights, queries, tiles, turns so far
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && warp_wait(bar, parity, p, abort); };
    // Both warps go through all tiles: what only the other side uses is passed,
    // so that each sees every phase of a slot.
    auto keys = [&](uint32_t tile) {
      wait(&bars.full[key_slot(tile)], key_use(tile) & 1u);
      return key_slot(tile);
    };
    auto values = [&](uint32_t tile) {
      const uint32_t sl = value_slot(tile, kRowSlots);
      wait(&bars.full[sl], value_use(tile, kRowSlots) & 1u);
      return sl;
    };
    auto commit = [&](uint64_t *bar) {
      if (ok) umma_commit_by(issue, bar);
    };
    auto arrive = [&](uint64_t *bar) {
      if (ok && issue) mbar_arrive(bar);
    };
    const uint64_t dK = desc128(smem_addr(ring_base), 1, 64),
                   dV = desc128(smem_addr(ring_base), kTileBytes / 32, 64), dQ = desc128(smem_addr(smem), 1, 64);
    auto issue_s = [&](int qb, uint32_t sl) {
      if (!ok) return;
      tc_fence_after();
      const uint64_t a = dQ + static_cast<uint64_t>(qb) * (kTileBytes >> 4), b = dK + sl * (kTileBytes >> 4);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        mma_ss(issue, tmem + 128 * x, a, (q >> 2) * (kTileBytes >> 5) + 2 * (q & 3), b,
               (q >> 2) * (kTileBytes >> 5) + 2 * (q & 3), idesc16<T>(kTile, 0, 0), q > 0);
      umma_commit_by(issue, &bars.s_full[x]);
    };
    auto issue_pv = [&](uint32_t sl, bool first) {
      if (!ok) return;
      tc_fence_after();
      const uint64_t b = dV + sl * (kTileBytes >> 4);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        mma_ts(issue, tmem + 256 + 128 * x, tmem + 128 * x + 8 * q, b, 128 * q, idesc16<T>(kTile, 0, 1),
               !first || q > 0);
      if constexpr (kLo) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          mma_ts(issue, tmem + 256 + 128 * x, tmem + 128 * x + 64 + 8 * q, b, 128 * q, idesc16<T>(kTile, 0, 1), 1);
      }
    };
    for_segments([&](const Segment &s, uint32_t k) {
      const int qb = kPaged ? k & 1 : x, n = tiles(s);
      if (kPaged || s.n[x] > 0) wait(&bars.q_full[qb], (kPaged ? k >> 1 : n_q++) & 1u);
      if (kPaged && x >= n) arrive(&bars.q_free[qb]);
      // this side's tiles: each second, or the first s.n[x]
      const int first = kAlternate ? x : 0, step = kAlternate ? 2 : 1, last = kAlternate ? n : s.n[x];
      auto mine = [&](int i) { return i < last && (!kAlternate || (i & 1) == x); };
      for (int i = 0; i < n + step && ok; ++i) {
        // the product of tile i - step, then the scores of tile i: both tiles first
        const bool has_v = i >= step;
        uint32_t v_slot = 0, k_slot = 0;
        if (has_v) v_slot = values(t + i - step);
        if (i < n) k_slot = keys(t + i);
        if (has_v && mine(i - step)) wait(&bars.p_full[x], n_p++ & 1u);
        // the sides take turns
        if (x == 1 || n_turn > 0) wait(&bars.turn[x], (n_turn - (x == 0)) & 1u);
        ++n_turn;
        if (has_v) {
          if (mine(i - step)) {
            issue_pv(v_slot, i - step == first);
            commit(&bars.freed[v_slot]);
            if (i >= last) commit(&bars.o_done[x]);
          } else {
            arrive(&bars.freed[v_slot]);
          }
        }
        if (i < n) {
          if (mine(i)) {
            issue_s(qb, k_slot);
            commit(&bars.freed[k_slot]);
            if (i + step >= last) commit(&bars.q_free[qb]);
          } else {
            arrive(&bars.freed[k_slot]);
          }
        }
        arrive(&bars.turn[1 - x]);
      }
      t += n;
      return ok;
    });
    umma_commit_by(issue, &bars.mma_done);
  } else if (warp == kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if constexpr (kPaged) {
      load_cache(p, loc, mq, mk, smem_addr(smem), smem_addr(ring_base), 2, bars, abort);
    } else {
      const uint32_t sq = smem_addr(smem), sr = smem_addr(ring_base);
      Loader ld(p, bars, abort);
      uint32_t t = 0, n_q0 = 0, n_q1 = 0;
      uint32_t job = blockIdx.x;
      bool more = true;
      for (uint32_t k = 0; ld.ok; ++k) {
        Segment s{};
        more = more && find_prompt(p, job, s);
        // (jobs without work come last)
        if (k > 1) ld.ok = warp_wait(&bars.job_free[k & 1], ((k >> 1) + 1) & 1u, p, abort);
        if (!ld.ok) break;
        if (lane == 0) {
          jobs[k & 1] = Job{s.kv0, s.rows, s.row0, s.h, s.n[0], s.n[1], !more, 0};
          mbar_arrive(&bars.job_full[k & 1]);
          // the next CTA that has not started, if any: its work becomes this CTA's
          if (more) steal_request(stolen, &bars.stolen);
        }
        __syncwarp();
        if (!more) break;
        // box of a Q tile: 64 dims x G heads x tok tokens
        auto load_q = [&](int x) {
          if (s.n[x] == 0) return;
          uint32_t &n_q = x ? n_q1 : n_q0;
          if (ld.begin_queries(x, n_q++)) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              tma_3d(sq + (2 * x + hf) * p.q_half, &mq, 64 * hf, s.h * p.G, s.kv0 + s.row0 + (kAlternate ? 0 : x * p.tok),
                     &bars.q_full[x]);
          }
          __syncwarp();
        };
        const int n = tiles(s), all = all_see(p, s);
        for (int j = 0; j < n && ld.ok; ++j, ++t) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t sl = kv ? value_slot(t, kRowSlots) : key_slot(t);
            uint64_t *bar =
                ld.begin(sl, kv ? value_use(t, kRowSlots) : key_use(t), kv && (j + 1) * kTile > all, kTileBytes);
            if (lane == 0 && ld.ok) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                tma_3d(sr + sl * kTileBytes + hf * (kTileBytes / 2), kv ? &mv : &mk, 64 * hf, s.h, s.kv0 + j * kTile,
                       bar);
            }
            __syncwarp();
            if (j == 0 && kv == 0) {
              load_q(0);
              load_q(1);
            }
          }
        }
        // the answer (waited for even if this CTA gave up: it is a copy into its memory)
        const bool there = __all_sync(0xffffffffu, mbar_wait(&bars.stolen, k & 1u, p.status, nullptr));
        more = there && steal_answer(stolen, job);
        ld.ok = ld.ok && there;
      }
      ld.drain();
    }
  } else if (warp == kGuardWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // who reads the marks: side 0, which merges the sides, or both
    const uint32_t side = (1u << row_warps) - 1u, readers = kAlternate ? side : side | side << 4;
    if constexpr (kPaged) {
      guard_cache<T>(p, loc, ring_base, readers, bad, bars, flags);
    } else {
      uint32_t phases = 0, t = 0;
      for_segments([&](const Segment &s, uint32_t k) {
        const int all = all_see(p, s), none = none_sees(p, s, p.sides * p.tok), n = tiles(s);
        bool ok = true;
        for (int j = all / kTile; j < n && ok; ++j)
          ok = guard_slot<T>(p, value_slot(t + j, kRowSlots), phases, ring_base, j * kTile, all, none, k, readers, bad,
                             bars, flags);
        t += n;
        return ok;
      });
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp >> 2) - 1, r = tid & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + 128 * x;
    const int r_tok = r / p.GB, r_head = r - r_tok * p.GB;
    uint32_t n_s = 0, n_o1 = 0, n_o = 0;
    bool ok = true;
    // one row's sum of products, times f; a NaN of the sum stays in `worst`
    auto finish = [&](float (&o)[32], float f, float &worst) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        o[i] *= f;
        o[i + 1] *= f;
        worst = max3_nan(worst, o[i], o[i + 1]);
      }
    };
    auto passed = [&](uint32_t k) {  // segment k's marks have been read
      __syncwarp();
      if (lane == 0) *const_cast<volatile int *>(&flags->done[warp - 4]) = static_cast<int>(k) + 1;
    };
    // Non-finite values, added where the row was stored: those that the guard
    // took out, and infinities that the products lost (rare: a loop that takes
    // no room in the code above).  sum: of the row's weights; a row without
    // weight is zero and stays so.
    auto repair = [&](const Segment &s, uint32_t k, bool valid, int lim, float sum, float worst, bool whole, auto *dst) {
      const bool marked = *nonfinite == static_cast<int>(k) + 1, lost = valid && sum == sum && isnan(worst);
      const bool any_lost = __any_sync(0xffffffffu, lost);
      if (!marked && !any_lost) return;
      const int t0 = s.j0 * kTile, end = min(all_see(p, s), t0 + tiles(s) * kTile);
      const uint32_t seen = any_lost ? values_seen<T, kPaged>(p, s, t0, end) : 0;
      for (int d = 0; d < kD; ++d) {
        const uint32_t kinds = kinds_of(seen, d);
        if (!valid) continue;
        float y = static_cast<float>(dst[d]);
        if (lost && kinds != 0 && isnan(y)) y = nonfinite_sum(kinds);
        if (marked) y = with_nonfinite(y, bad, d, lim);
        dst[d] = whole && sum == 0.f ? 0.f : y;
      }
    };
    auto store16 = [&](T *dst, const float (&o)[32]) {
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        *reinterpret_cast<uint4 *>(dst + i) =
            make_uint4(pack16(o[i], o[i + 1], T()), pack16(o[i + 2], o[i + 3], T()), pack16(o[i + 4], o[i + 5], T()),
                       pack16(o[i + 6], o[i + 7], T()));
    };
    if ((warp & 3) < row_warps) for_segments([&](const Segment &s, uint32_t k) {
      const int n = kPaged ? (s.n[0] + 1 - x) >> 1 : s.n[x];
      const int qi = s.row0 + (kAlternate ? 0 : x * p.tok) + r_tok;
      const int hq = s.chunk * kTile + r_head;
      const bool valid = r < p.R && qi < s.rows && hq < p.G;
      const int lim = valid ? s.limit(qi, p.causal) : 0;
      float ref = -INFINITY, l = 0.f;
      bool any_large = false;
      for (int i = 0; i < n && ok; ++i) {
        const int t0 = (s.j0 + (kAlternate ? 2 * i + x : i)) * kTile;
        ok = warp_wait(&bars.s_full[x], n_s & 1u, p, abort);
        ++n_s;
        // Side 1's O and sums are merged by side 0 before it writes them again.
        // (Its scores are here, so side 0 is past segment k - 2 and the parity
        // is that of k - 1.)
        if (kAlternate && x == 1 && k > 0 && i == 0) ok = ok && warp_wait(&bars.seg_done, (k - 1) & 1u, p, abort);
        if (!ok) break;
        tc_fence_after();
        softmax_tile<T, kLo>(ts, to, p.c, lim - t0, i == 0, ref, l, any_large);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[x]);
      }
      if (!ok) return false;
      const float sub = ref * p.c - kShift<T>;  // (-inf if it saw nothing)
      if (!kAlternate) {
        if (n == 0) {
          passed(k);
          return true;
        }
        ok = warp_wait(&bars.o_done[x], n_o++ & 1u, p, abort);
        if (!ok) return false;
        tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;
        T *dst = static_cast<T *>(p.out) +
                 (static_cast<int64_t>(s.kv0 + qi) * p.Hq + static_cast<int64_t>(s.h) * p.G + hq) * kD;
        float worst = 0.f;
#pragma unroll
        for (int col = 0; col < kD; col += 32) {
          float o[32];
          tmem_ld32(to + col, o);
          finish(o, inv, worst);
          if (valid) store16(dst + col, o);
        }
        repair(s, k, valid, lim, l, worst, true, dst);
        tc_fence_before();
        passed(k);
      } else if (x == 1) {
        if (n > 0) ml[r] = make_float2(sub, l);
        __syncwarp();
        if (lane == 0 && n > 0) mbar_arrive(&bars.side1);
      } else {
        const bool both = tiles(s) > 1, whole = !kPaged || s.whole;
        ok = warp_wait(&bars.o_done[0], k & 1u, p, abort);
        if (both) {
          ok = ok && warp_wait(&bars.o_done[1], n_o1 & 1u, p, abort) &&
               warp_wait(&bars.side1, n_o1 & 1u, p, abort);
          ++n_o1;
        }
        if (!ok) return false;
        tc_fence_after();
        float m = sub, w0 = 1.f, w1 = 0.f;
        if (both) {
          const float2 other = ml[r];
          // a NaN reference weighs NaN
          m = fmaxf(sub, other.x);
          const float base = m == -INFINITY ? 0.f : m;
          w0 = ex2f(sub - base);
          w1 = ex2f(other.x - base);
          l = l * w0 + other.y * w1;
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        // whole: the result; else a record for the combine kernel
        float *rec = record(p, 2 * blockIdx.x + (s.starts ? 1 : 0));
        const int64_t row = kPaged ? static_cast<int64_t>(s.b) * p.nq + qi : s.kv0 + qi;
        T *dst = static_cast<T *>(p.out) + (row * p.Hq +
                                            static_cast<int64_t>(s.h) * p.G + hq) * kD;
        if (valid && !whole) *reinterpret_cast<float2 *>(rec + 2 * r) = make_float2(m, l);
        float worst = 0.f;
#pragma unroll
        for (int col = 0; col < kD; col += 32) {
          float o[32];
          tmem_ld32(to + col, o);
          if (both) {
            float o1[32];
            tmem_ld32(to + 128 + col, o1);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = o[i] * w0 + o1[i] * w1;
          }
          finish(o, whole ? inv : 1.f, worst);
          if (valid) {
            if (whole) {
              store16(dst + col, o);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(rec + 2 * p.row_stride + r * kD + col + i) =
                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        if (whole) repair(s, k, valid, lim, l, worst, true, dst);
        else repair(s, k, valid, lim, l, worst, false, rec + 2 * p.row_stride + r * kD);
        tc_fence_before();
        passed(k);
        if (lane == 0) mbar_arrive(&bars.seg_done);
      }
      return true;
    });
  }
  if constexpr (kPaged) {
    if (tid == 0) write_plan(p, loc);
  }
  end_cta<512>(bars, flags, p);
}

// ------------------------------------------------- cache, up to 64 query rows
// The same walk with tokens as the products' M: a step of a few query rows is
// bound by the bytes of the cache, and the form above would spend a softmax of
// 128 rows and two 128-row products on each key tile.  Here
//   S^T[128 tokens x NR rows] = K Q^T,  O^T[128 dims x 2 NR] += V^T [P | P'],
// with P the weights' 16-bit parts and, for bf16, P' their remainders in NR
// more columns, added at the end.  K and V are the A operands from shared
// memory (V read dims-major), Q and P the narrow B operands.  A softmax thread
// owns a token; two (four) sides share each tile and take 8 or 16 rows each.  No
// row spans a thread, so the rows' references are common to a side's 128
// threads (shared memory) and change only when some score passes one by 2^8
// (one barrier with a vote per tile); the sums stay with the threads until the
// segment ends.  S^T has two buffers: tile i + 1's scores are computed while
// tile i's weights are.  P goes to shared memory as 16-byte pieces,
// [8-row group][token].
template <typename T, int NR>
struct Cols {
  static constexpr bool kLo = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kSide = NR == 16 ? 8 : 16;      // rows of a side
  static constexpr int kThreads = (4 + NR / kSide * 4) * 32;
  static constexpr int kN = kLo ? 2 * NR : NR;         // columns of O^T
  static constexpr int kQBufs = NR == 64 ? 1 : 2;
  static constexpr int kPBufs = NR == 64 ? 1 : 2;  // (two for 64 rows fit, and gain nothing: 113 -> 114 us)
  // 16 x 32768 tokens: 4 and 5 slots 162 us; 4 long contexts: 222 and 221;
  // 16-token chunks: 113 and 109 (6 slots were slower: 200 when 4 were 186)
  static constexpr int kSlots = 4;
  static constexpr int kQBytes = NR * kD * 2;
  static constexpr int kPBytes = kN * kTile * 2;
  static constexpr int kP = kQBufs * kQBytes;
  static constexpr int kRing = kP + kPBufs * kPBytes;
  static constexpr int kTail = kRing + kSlots * kTileBytes;
  // Each row's reference, the score above which it moves, what is added to a
  // score's logarithm, what an O column is multiplied by, four warps' maxima
  // or sums, and what is taken from large scores.
  static constexpr int kRefs = kTail + kTailBytes + 64;  // (locate's scratch: a word of 8 bytes per warp)
  static constexpr int kLimits = kRefs + NR * 4;
  static constexpr int kSubs = kLimits + NR * 4;
  static constexpr int kFactor = kSubs + NR * 4;
  static constexpr int kPart = kFactor + NR * 4;
  static constexpr int kOff = kPart + 4 * NR * 4;
  static constexpr int kAnyOff = kOff + NR * 4;    // whether a side has such a row
  static constexpr int kBytes = kAnyOff + 16;
  static constexpr uint32_t kColO = 2 * NR;            // S^T buffers at 0 and NR
  static constexpr uint32_t kCols = kColO + kN <= 64 ? 64 : kColO + kN <= 128 ? 128 : 256;
  static_assert(kRing % 1024 == 0 && kBytes <= 227 * 1024 && kColO + kN <= kCols, "layout");
  static_assert(64 + kThreads / 32 * 8 <= 160 + 64, "locate's scratch");
};

// barrier of a side's 128 threads with a vote
__device__ __forceinline__ bool side_any(int x, bool v) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.u32 a, %2, 0;\n barrier.cta.red.or.pred b, %1, 128, a;\n selp.u32 %0, 1, 0, "
      "b;\n}\n"
      : "=r"(any)
      : "r"(x + 1), "r"(static_cast<uint32_t>(v))
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void side_sync(int x) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(x + 1) : "memory");
}
// maximum over a warp that keeps a NaN
__device__ __forceinline__ float warp_max_nan(float v) {
  float y;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}

// N columns of this thread's tensor-memory lane
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, float (&v)[N]) {
  if constexpr (N == 8) tmem_ld8(addr, v);
  else if constexpr (N == 16) tmem_ld16(addr, v);
  else tmem_ld32(addr, v);
}

template <typename T, int NR>
__global__ void __launch_bounds__(Cols<T, NR>::kThreads, 1)
    k_cols16(const Attend16 p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk) {
  using C = Cols<T, NR>;
  constexpr bool kLo = C::kLo;
  constexpr int SR = C::kSide;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *ring_base = smem + C::kRing, *tail = smem + C::kTail;
  int *bad = reinterpret_cast<int *>(tail + kOffBad);
  Bars &bars = *reinterpret_cast<Bars *>(tail + kOffBar);
  Flags *flags = reinterpret_cast<Flags *>(tail + kOffFlags);
  volatile int *abort = &flags->abort, *nonfinite = &flags->nonfinite;
  int64_t *loc = reinterpret_cast<int64_t *>(tail + kOffLoc);
  const int soft_warps = (p.R + SR - 1) / SR * 4;  // sides without rows rest

  start_cta<C::kCols>(bars, flags, bad, 1, 1, soft_warps, soft_warps, 1);
  // Q rows that no copy writes are zero
  for (int i = tid; i < C::kP / 16; i += C::kThreads) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (tid == 64) {
    fetch_map(mq);
    fetch_map(mk);
  }
  pdl_trigger();
  pdl_wait();
  locate16<C::kThreads>(p, loc, loc + 8);
  tc_fence_after();
  const uint32_t tmem = flags->tmem;

  if (warp < 2) {
    // ------------------------------------------------------------- products
    // warp 0 issues the scores, warp 1 the products with the values
    const uint32_t issue = lane == 0;
    uint32_t tiles = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && warp_wait(bar, parity, p, abort); };
    auto commit = [&](uint64_t *bar) {
      if (ok) umma_commit_by(issue, bar);
    };
    const uint64_t dK = desc128(smem_addr(ring_base), 1, 64),
                   dV = desc128(smem_addr(ring_base), kTileBytes / 32, 64), dQ = desc128(smem_addr(smem), 1, 64),
                   dP = desc_plain(smem_addr(smem + C::kP), 8, 128);
    cache_segments(p, loc, [&](const Segment &s, uint32_t k) {
      const int n = s.n[0];
      if (warp == 0) {
        const uint32_t qb = k % C::kQBufs, use = k / C::kQBufs;
        wait(&bars.q_full[qb], use & 1u);
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t sl = key_slot(tiles), buf = tiles & 1u;
          wait(&bars.full[sl], key_use(tiles) & 1u);
          if (tiles >= 2) wait(&bars.s_free[buf], ((tiles >> 1) + 1u) & 1u);
          if (ok) {
            tc_fence_after();
            const uint64_t a = dK + sl * (kTileBytes >> 4), b = dQ + qb * (C::kQBytes >> 4);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              mma_ss(issue, tmem + buf * NR, a, (q >> 2) * (kTileBytes >> 5) + 2 * (q & 3), b,
                     (q >> 2) * (C::kQBytes >> 5) + 2 * (q & 3), idesc16<T>(NR, 0, 0), q > 0);
          }
          commit(&bars.s_full[buf]);
          commit(&bars.freed[sl]);
          if (i == n - 1) commit(&bars.q_free[qb]);
          ++tiles;
        }
      } else {
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t sl = value_slot(tiles, C::kSlots), buf = tiles & 1u;
          wait(&bars.full[sl], value_use(tiles, C::kSlots) & 1u);
          wait(&bars.p_full[buf], (tiles >> 1) & 1u);
          if (ok) {
            tc_fence_after();
            const uint64_t a = dV + sl * (kTileBytes >> 4), b = dP + tiles % C::kPBufs * (C::kPBytes >> 4);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              mma_ss(issue, tmem + C::kColO, a, 128 * q, b, 16 * q, idesc16<T>(C::kN, 1, 1), i > 0 || q > 0);
          }
          commit(&bars.freed[sl]);
          commit(&bars.o_done[buf]);
          ++tiles;
        }
      }
      return ok;
    });
    umma_commit_by(issue, &bars.mma_done);
  } else if (warp == kLoadWarp) {
    load_cache(p, loc, mq, mk, smem_addr(smem), smem_addr(ring_base), C::kQBufs, bars, abort);
  } else if (warp == kGuardWarp) {
    guard_cache<T>(p, loc, ring_base, (1u << soft_warps / 4) - 1u, bad, bars, flags);
  } else {
    // -------------------------------------------------------------- softmax
    const int x = (warp >> 2) - 1, t = tid & (kTile - 1), row0 = x * SR;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + row0, to = tmem + lanes + C::kColO + row0;
    float *refs = reinterpret_cast<float *>(smem + C::kRefs) + row0;
    float *limits = reinterpret_cast<float *>(smem + C::kLimits) + row0;
    float *subs = reinterpret_cast<float *>(smem + C::kSubs) + row0;
    float *factor = reinterpret_cast<float *>(smem + C::kFactor) + row0;
    float *part = reinterpret_cast<float *>(smem + C::kPart) + 4 * row0;
    float *offs = reinterpret_cast<float *>(smem + C::kOff) + row0;
    int *any_off = reinterpret_cast<int *>(smem + C::kAnyOff) + x;
    bool large_rows = false;  // *any_off
    const int tok0 = row0 / p.GB, head0 = row0 - tok0 * p.GB;
    uint32_t n_s = 0;  // tiles so far
    bool ok = true;
    // Waits for the product of an earlier tile.  The tiles take the two barriers
    // in turn; that of two tiles before was waited for already (a tile's
    // weights wait below for the last reader of their buffer, or a later one),
    // so the parity names one phase.
    auto product = [&](uint32_t tile) { return warp_wait(&bars.o_done[tile & 1u], (tile >> 1) & 1u, p, abort); };
    // Every warp of a side goes through the same barriers, after a failed wait too.
    if (warp < 4 + soft_warps) cache_segments(p, loc, [&](const Segment &s, uint32_t k) {
      const int all = all_see(p, s), n = s.n[0];
      float2 l[SR / 2];
#pragma unroll
      for (int r = 0; r < SR / 2; ++r) l[r] = make_float2(0.f, 0.f);
      for (int i = 0; i < n; ++i) {
        const int tok = (s.j0 + i) * kTile + t;
        ok = ok && warp_wait(&bars.s_full[n_s & 1u], (n_s >> 1) & 1u, p, abort);
        tc_fence_after();
        float v[SR];
        tmem_ld_cols<SR>(ts + (n_s & 1u) * NR, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bars.s_free[n_s & 1u]);
        if ((s.j0 + i + 1) * kTile > all) {
          int qi = s.row0 + tok0, head = head0, lim = s.limit(qi, p.causal);
#pragma unroll
          for (int r = 0; r < SR; ++r) {
            if (tok >= lim) v[r] = -INFINITY;
            if (++head == p.GB) {
              head = 0;
              lim = s.limit(++qi, p.causal);
            }
          }
        }
        // has a score passed its row's limit?  A NaN has.
        bool stay = i > 0;
        if (i > 0) {
#pragma unroll
          for (int r = 0; r < SR; r += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(limits + r);
            stay = stay && v[r] <= f.x && v[r + 1] <= f.y && v[r + 2] <= f.z && v[r + 3] <= f.w;
          }
        }
        if (side_any(x, !stay)) {
          // the tile's maxima: over a warp's tokens, then over the four warps
#pragma unroll
          for (int r = 0; r < SR; ++r) {
            const float m = warp_max_nan(v[r]);
            if (lane == 0) part[(warp & 3) * SR + r] = m;
          }
          side_sync(x);
          if (t < SR) {
            const float m = max3_nan(max3_nan(part[t], part[SR + t], part[2 * SR + t]), part[3 * SR + t],
                                     part[3 * SR + t]);
            const float old = i == 0 ? -INFINITY : refs[t];
            const float lazy = fminf(kLazy / p.c, FLT_MAX);
            const bool up = !(m <= old + lazy);
            const float ref = up ? m : old;
            factor[t] = up ? ex2f((old - m) * p.c) : 1.f;
            refs[t] = ref;
            limits[t] = ref + lazy;  // (+inf stays: only a NaN is above)
            const bool large = fabsf(ref * p.c) > kLarge && ref != -INFINITY;
            offs[t] = large ? ref : 0.f;
            subs[t] = ref == -INFINITY ? 0.f : large ? kShift<T> : kShift<T> - ref * p.c;
            const bool any = __any_sync((1u << SR) - 1u, large);
            if (t == 0) *any_off = any;
          }
          side_sync(x);
          large_rows = *any_off != 0;
          if (i > 0) {
            // the last product must be done
            ok = ok && product(n_s - 1);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < SR; r += 2)
              l[r >> 1] = __fmul2_rn(l[r >> 1], *reinterpret_cast<const float2 *>(factor + r));
#pragma unroll
            for (int c = 0; c < (kLo ? 2 : 1); ++c) {
              float o[SR];
              tmem_ld_cols<SR>(to + c * NR, o);
#pragma unroll
              for (int r = 0; r < SR; ++r) o[r] *= factor[r];
              tmem_st_cols<SR>(to + c * NR, o);
            }
            tmem_stored();
          }
        }
        if (large_rows) {
#pragma unroll
          for (int r = 0; r < SR; ++r) v[r] -= offs[r];
        }
        uint32_t w[SR / 2], e[SR / 2];  // weights and their remainders, two rows each
#pragma unroll
        for (int r = 0; r < SR; r += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(subs + r);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int at = (r >> 1) + a;
            const float2 x2 = __ffma2_rn(make_float2(v[2 * at], v[2 * at + 1]), make_float2(p.c, p.c),
                                         a ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
            const float2 pr = make_float2(ex2f(x2.x), ex2f(x2.y));
            l[at] = __fadd2_rn(l[at], pr);
            w[at] = pack16(pr.x, pr.y, T());
            if constexpr (kLo)
              e[at] = pack16(pr.x - __uint_as_float(w[at] << 16), pr.y - __uint_as_float(w[at] & 0xffff0000u), T());
          }
        }
        // the last product that read this buffer of P
        if (n_s >= C::kPBufs) ok = ok && product(n_s - C::kPBufs);
        uint8_t *dst = smem + C::kP + n_s % C::kPBufs * C::kPBytes + (row0 >> 3) * (kTile * 16) + t * 16;
#pragma unroll
        for (int g = 0; g < SR / 8; ++g) {
          *reinterpret_cast<uint4 *>(dst + g * (kTile * 16)) = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
          if constexpr (kLo)
            *reinterpret_cast<uint4 *>(dst + (NR / 8 + g) * (kTile * 16)) =
                make_uint4(e[4 * g], e[4 * g + 1], e[4 * g + 2], e[4 * g + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bars.p_full[n_s & 1u]);
        ++n_s;
      }
      // the rows' sums over a warp's tokens, then over the four warps
      side_sync(x);  // the maxima of a last move have been read
#pragma unroll
      for (int r = 0; r < SR; ++r) {
        float a = r & 1 ? l[r >> 1].y : l[r >> 1].x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (lane == 0) part[(warp & 3) * SR + r] = a;
      }
      side_sync(x);
      float *rec = record(p, 2 * blockIdx.x + (s.starts ? 1 : 0));
      if (t < SR) {
        const float sum = (part[t] + part[SR + t]) + (part[2 * SR + t] + part[3 * SR + t]);
        factor[t] = !s.whole ? 1.f : sum != 0.f ? 1.f / sum : 0.f;
        if (!s.whole && row0 + t < p.R)
          *reinterpret_cast<float2 *>(rec + 2 * (row0 + t)) =
              make_float2(refs[t] * p.c - kShift<T>, sum);
      }
      ok = ok && product(n_s - 1);
      tc_fence_after();
      side_sync(x);
      // thread t: dim t of the side's rows
      float o[SR];
      auto load_o = [&]() {
        tmem_ld_cols<SR>(to, o);
        if constexpr (kLo) {
          float e[SR];
          tmem_ld_cols<SR>(to + NR, e);
#pragma unroll
          for (int r = 0; r < SR; ++r) o[r] += e[r];
        }
      };
      load_o();
      // infinities that the products lost
      bool lost = false;
#pragma unroll
      for (int r = 0; r < SR; ++r) lost |= isnan(o[r]);
      if (__any_sync(0xffffffffu, ok && lost)) {
        const int t0 = s.j0 * kTile;
        const uint32_t kinds = kinds_of(values_seen<T, true>(p, s, t0, min(all, t0 + n * kTile)), t);
        load_o();  // (rather than kept across the call)
#pragma unroll
        for (int r = 0; r < SR; ++r)
          if (isnan(o[r]) && kinds != 0) o[r] = nonfinite_sum(kinds);
      }
      if (ok) {
        int qi = s.row0 + tok0, head = head0;
        T *out = static_cast<T *>(p.out) + (static_cast<int64_t>(s.h) * p.G + s.chunk * kTile) * kD + t;
        const int heads = p.G - s.chunk * kTile;
#pragma unroll
        for (int r = 0; r < SR; ++r) {
          if (row0 + r < p.R && qi < s.rows && head < heads) {
            const bool zero = factor[r] == 0.f;  // every score -inf
            float y = zero ? 0.f : o[r] * factor[r];
            if (!zero && *nonfinite == static_cast<int>(k) + 1) y = with_nonfinite(y, bad, t, s.limit(qi, p.causal));
            if (s.whole) out[((static_cast<int64_t>(s.b) * p.nq + qi) * p.Hq + head) * kD] = to16(y, T());
            else rec[2 * p.row_stride + (row0 + r) * kD + t] = y;
          }
          if (++head == p.GB) {
            head = 0;
            ++qi;
          }
        }
      }
      tc_fence_before();
      side_sync(x);  // sums, factors and marks are read
      if (t == 0) *const_cast<volatile int *>(&flags->done[x]) = static_cast<int>(k) + 1;
      return true;
    });
  }
  if (tid == 0) write_plan(p, loc);
  end_cta<C::kCols>(bars, flags, p);
}

// Joins the records of each segment that spans CTAs: block (c, y) the rows 4 y
// .. of the one that starts in CTA c and goes on, one warp per row.  Record
// 2 c + 1 holds its first part, 2 k those of the CTAs k behind.
template <typename T>
__global__ void __launch_bounds__(128) k_combine16(const Attend16 p) {
  pdl_trigger();
  pdl_wait();
  const int2 plan = p.plan[blockIdx.x];
  if (plan.x < 0) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int u = plan.x / p.H, h = plan.x - u * p.H;
  const int b = u / p.rts, rt = u - b * p.rts;
  const int qi = rt / p.chunks * p.tok + r / p.GB, hq = rt % p.chunks * kTile + r % p.GB;
  if (r >= p.R || qi >= p.nq || hq >= p.G) return;
  const int first = blockIdx.x, count = plan.y - first + 1;
  auto rec = [&](int i) { return record(p, 2 * (first + i) + (i == 0 ? 1 : 0)); };
  float m = -INFINITY;
  for (int i = lane; i < count; i += 32) m = fmaxf(m, rec(i)[2 * r]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < count; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < count) {
      const float2 t = *reinterpret_cast<const float2 *>(rec(i0 + lane) + 2 * r);
      w = ex2f(t.x - base);
      l += w * t.y;
      // an infinite sum counts however small its weight: 0 x inf would be NaN
      // (a NaN weight's sum of weights is NaN too)
      w = fmaxf(w, __uint_as_float(1u));
    }
    const int top = min(32, count - i0);
#pragma unroll 8
    for (int i = 0; i < top; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float4 o = *reinterpret_cast<const float4 *>(rec(i0 + i) + 2 * p.row_stride + r * kD + 4 * lane);
      acc.x = fmaf(wi, o.x, acc.x); acc.y = fmaf(wi, o.y, acc.y);
      acc.z = fmaf(wi, o.z, acc.z); acc.w = fmaf(wi, o.w, acc.w);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (l == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);  // every score -inf
  const float inv = l != 0.f ? 1.f / l : 0.f;
  T *dst = static_cast<T *>(p.out) +
           ((static_cast<int64_t>(b) * p.nq + qi) * p.Hq + static_cast<int64_t>(h) * p.G + hq) * kD + 4 * lane;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack16(acc.x * inv, acc.y * inv, T()), pack16(acc.z * inv, acc.w * inv, T()));
}

// --------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's encoder, looked up once
EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *sym = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return static_cast<EncodeFn>(nullptr);
    return reinterpret_cast<EncodeFn>(sym);
  }();
  return fn;
}

// 64-dim boxes with the 128-byte swizzle
bool encode(CUtensorMap *map, int dtype, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box) {
  const cuuint32_t ones[3] = {1, 1, 1};
  const EncodeFn fn = encoder();
  return fn != nullptr &&
         fn(map, dtype == ISOQUANT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
            const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [tokens][heads][128], tokens `stride` elements apart; box_heads x box_tokens
bool encode_rows(CUtensorMap *map, int dtype, const void *base, int64_t tokens, int heads, int64_t stride,
                 int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {kD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {kD * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  return encode(map, dtype, 3, base, dims, strides, box);
}

void row_tiles(Attend16 &p, int group) {
  p.G = group;
  p.GB = group < kTile ? group : kTile;
  p.chunks = (group + kTile - 1) / kTile;
  p.tok = kTile / p.GB;
}

// A kernel's launch with its dynamic shared memory, allowed once per device.
template <auto kernel, typename... A>
cudaError_t launch_tiles(int device, int threads, int smem, unsigned grid, cudaStream_t stream, const A &...args) {
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (device >= 64 || !(allowed.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(kernel, dim3(grid), dim3(threads), smem, stream, args...);
}
static_assert(2 * kTileBytes + kRowSlots * kTileBytes + kOffMl + kTile * 8 <= 227 * 1024 && 64 + kThreads16 / 32 * 8 <= 160 &&
                  2 * sizeof(Job) + 16 <= 160,
              "shared memory of k_attend16");
int rows_smem(const Attend16 &p) { return 4 * p.q_half + p.slots * kTileBytes + kOffMl + kTile * 8; }

template <typename T, int NR>
cudaError_t launch_cols(Attend16 p, const CUtensorMap &mq, const CUtensorMap &mk, unsigned grid, cudaStream_t stream) {
  p.slots = Cols<T, NR>::kSlots;
  p.q_half = Cols<T, NR>::kQBytes / 2;
  return launch_tiles<k_cols16<T, NR>>(p.device, Cols<T, NR>::kThreads, Cols<T, NR>::kBytes, grid, stream, p, mq, mk);
}
template <typename T>
cudaError_t launch_cache(Attend16 p, const CUtensorMap &mq, const CUtensorMap &mk, unsigned grid,
                         cudaStream_t stream) {
  if (p.R <= 16) return launch_cols<T, 16>(p, mq, mk, grid, stream);
  if (p.R <= 32) return launch_cols<T, 32>(p, mq, mk, grid, stream);
  if (p.R <= 64) return launch_cols<T, 64>(p, mq, mk, grid, stream);
  p.slots = kRowSlots;
  p.q_half = kTileBytes / 2;
  return launch_tiles<k_attend16<T, true, true>>(p.device, kThreads16, rows_smem(p), grid, stream, p, mq, mk, mk);
}

template <typename T, bool kAlternate>
cudaError_t launch_prompt(const Attend16 &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                          unsigned grid, cudaStream_t stream) {
  return launch_tiles<k_attend16<T, false, kAlternate>>(p.device, kThreads16, rows_smem(p), grid, stream, p, mq, mk, mv);
}

// the cache's row tiles: rows, and the stride of a record's rows
void paged_rows(Attend16 &p, const AttendShape &s) {
  row_tiles(p, s.group);
  if (p.tok > s.nq) p.tok = s.nq;
  p.R = p.tok * p.GB;
  p.rts = (s.nq + p.tok - 1) / p.tok * p.chunks;
  p.row_stride = (p.R + 1) / 2 * 2;
}

size_t plan_bytes(int n_cta) { return (static_cast<size_t>(n_cta) * sizeof(int2) + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_prompt_attend(const isoquant_ctx *ctx, const void *q, const void *k, const void *v, int dtype,
                                 int n_tok, int num_q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                 const int32_t *cu_seqlens, int batch, int causal, float scale, void *out,
                                 cudaStream_t stream) {
  Attend16 p{};
  p.H = ctx->num_kv_heads;
  p.Hq = num_q_heads;
  row_tiles(p, p.Hq / p.H);
  p.R = p.tok * p.GB;
  p.B = batch;
  p.causal = causal;
  p.c = scale * 1.4426950408889634f;
  p.cu = cu_seqlens;
  p.n_tok = n_tok;
  p.slots = kRowSlots;
  p.q_half = kTileBytes / 2;
  p.values = static_cast<const uint16_t *>(v);
  p.v_stride = v_stride;
  p.out = out;
  p.status = ctx->status;
  p.device = ctx->device;
  CUtensorMap mq, mk, mv;
  if (!encode_rows(&mq, dtype, q, n_tok, p.Hq, q_stride, p.GB, p.tok) ||
      !encode_rows(&mk, dtype, k, n_tok, p.H, k_stride, 1, kTile) ||
      !encode_rows(&mv, dtype, v, n_tok, p.H, v_stride, 1, kTile))
    return cudaErrorInvalidValue;
  // jobs: no more than one per `sides` row tiles and one per sequence
  auto jobs = [&](int sides) { return (static_cast<int64_t>(n_tok) / (sides * p.tok) + batch) * p.H; };
  // Where two-sided jobs would leave SMs idle, jobs of one row tile whose key
  // tiles the sides share are half as long (7237 tokens, 2 and 1 heads, 57
  // jobs: 143 -> 81 us; 16384, 1 head, 65 jobs: 263 -> 169; 114 jobs of three
  // prompts: 41 -> 35), but read each key tile twice as often (136 short jobs
  // 17.9 -> 20.9, 252 jobs 56 -> 60, 316 jobs 73 -> 84).
  p.sides = jobs(2) < ctx->num_sms * 3 / 4 ? 1 : 2;
  const int64_t grid = jobs(p.sides);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(grid);
  const bool bf = dtype == ISOQUANT_BF16;
  if (p.sides == 1)
    return bf ? launch_prompt<__nv_bfloat16, true>(p, mq, mk, mv, g, stream)
              : launch_prompt<__half, true>(p, mq, mk, mv, g, stream);
  return bf ? launch_prompt<__nv_bfloat16, false>(p, mq, mk, mv, g, stream)
            : launch_prompt<__half, false>(p, mq, mk, mv, g, stream);
}

size_t dense_workspace_bytes(const isoquant_ctx *ctx, const AttendShape &s) {
  Attend16 p{};
  paged_rows(p, s);
  return plan_bytes(ctx->num_sms) +
         static_cast<size_t>(2) * ctx->num_sms * p.row_stride * (kD + 2) * sizeof(float);
}

cudaError_t launch_dense_attend(const isoquant_ctx *ctx, const isoquant_dense_cache *cache, const AttendShape &s,
                                const void *q, const int32_t *page_table, int max_pages, const int32_t *seq_lens,
                                float scale, void *ws, void *out, cudaStream_t stream) {
  Attend16 p{};
  p.H = s.kv_heads;
  p.Hq = s.q_heads;
  paged_rows(p, s);
  p.B = s.batch;
  p.nq = s.nq;
  p.causal = s.causal;
  p.c = scale * 1.4426950408889634f;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.max_pages = max_pages;
  p.num_pages = cache->num_pages;
  while ((1 << p.ps_shift) < cache->page_size) ++p.ps_shift;
  p.values = static_cast<const uint16_t *>(cache->data);
  p.n_cta = ctx->num_sms;
  p.plan = static_cast<int2 *>(ws);
  p.records = reinterpret_cast<float *>(static_cast<char *>(ws) + plan_bytes(p.n_cta));
  p.out = out;
  p.status = ctx->status;
  p.device = ctx->device;
  CUtensorMap mq, mk;
  const int64_t rows = static_cast<int64_t>(cache->num_pages) * 2 * p.H * cache->page_size;
  const cuuint64_t dims[2] = {kD, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {kD * 2};
  const cuuint32_t box[2] = {64, kBox};
  if (!encode_rows(&mq, cache->dtype, q, static_cast<int64_t>(s.batch) * s.nq, p.Hq,
                   static_cast<int64_t>(p.Hq) * kD, p.GB, p.tok) ||
      !encode(&mk, cache->dtype, 2, cache->data, dims, strides, box))
    return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(p.n_cta);
  const bool bf = cache->dtype == ISOQUANT_BF16;
  const cudaError_t e = bf ? launch_cache<__nv_bfloat16>(p, mq, mk, grid, stream)
                           : launch_cache<__half>(p, mq, mk, grid, stream);
  if (e != cudaSuccess) return e;
  const dim3 cg(grid, static_cast<unsigned>((p.R + 3) / 4)), block(128);
  return bf ? launch_pdl(k_combine16<__nv_bfloat16>, cg, block, 0, stream, p)
            : launch_pdl(k_combine16<__half>, cg, block, 0, stream, p);
}

}  // namespace isoquant
