// kernel_attention_rows.cu -- the kernels of qvg_attention_batch and
// qvg_attention_weights for few rows, and the merge of partial results.
//
// For a row r with query q (rotated to its position) and the keys k_j it sees
// (rotated to theirs; the reconstructed prefix and its own tail),
//   s_j = q.k_j / sqrt(d),  O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m).
// All rows of a K/V head (every sequence, every query head of the group) read
// the same prefix, so a key is reconstructed once for 16 of them.
//
// A warp takes 16 keys at a time and builds the tensor core's operands in the
// registers that need them (mma.sync m16n8k16, bf16 operands, fp32 sums): a
// lane reconstructs and rotates 32 channels of two keys, and 16 channels of
// four values.  The contraction over channels may run in any order, so lane
// 4g + c owns the 8-channel chunks c, c + 4, c + 8, c + 12 of key g: four lanes
// read 64 contiguous bytes of a centroid row.  In the product with V the lane
// owns chunks g and g + 8 of its keys.  With few rows nothing is shared
// between warps, so nothing goes through shared memory but the queries.
#include "batch.cuh"

namespace qvg {
namespace {

constexpr int kRwThreads = 128;                   // 4 warps, each with its own keys
constexpr int kRwRows = 16;                       // rows per CTA (the M of the product)
constexpr int kRwKeys = 16;                       // keys per warp and step
constexpr int kRwStep = kRwThreads / 32 * kRwKeys;   // keys per CTA and step
constexpr int kRwChunk = 64;                      // rows whose weights are added up at a time
constexpr int kRwQStride = kD + 8;                // padded row of Q in shared memory (bf16)

// D += A B, m16n8k16, bf16 operands
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The keys of a CTA: the prefix of head h, or the tail of sequence b.
struct Keys {
  int h, b;
  bool tail;
  int64_t n;                      // keys there are
};

// Reconstructed channels c0 .. c0+7 of a prefix token, as packed bf16 pairs:
// y = s q + m (or s (u - 2)), plus the centroids of stages T, ..., 1, each an
// fp32 add, then one rounding -- the arithmetic of qvg_dequant_fused.
template <int TT>
__device__ __forceinline__ uint4 rebuild8(const BatchParams& p, const float2* nlut, int w, int h, uint32_t tok, int c0,
                                          uint32_t code, float s, float m, const int* kk) {
  const float2 s2 = make_float2(s, s), m2 = make_float2(m, m);
  float2 y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 q = nlut[(code >> (4 * e)) & 0xFu];
    y[e] = p.sym ? __fmul2_rn(s2, q) : __ffma2_rn(s2, q, m2);
  }
  const int T = TT >= 0 ? TT : p.T;
  const __nv_bfloat16* tab = p.tab[w] + (int64_t)h * p.K * kD + c0;
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    const int k = TT >= 0 ? kk[t] : min((int)__ldg(p.assign[w] + ((int64_t)t * p.H + h) * p.Nk + tok), p.K - 1);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(tab + (int64_t)t * p.H * p.K * kD + (uint32_t)k * kD));
    y[0] = __fadd2_rn(y[0], make_float2(lo_f(v.x), hi_f(v.x)));
    y[1] = __fadd2_rn(y[1], make_float2(lo_f(v.y), hi_f(v.y)));
    y[2] = __fadd2_rn(y[2], make_float2(lo_f(v.z), hi_f(v.z)));
    y[3] = __fadd2_rn(y[3], make_float2(lo_f(v.w), hi_f(v.w)));
  }
  return make_uint4(pack2(y[0].x, y[0].y), pack2(y[1].x, y[1].y), pack2(y[2].x, y[2].y), pack2(y[3].x, y[3].y));
}

template <int TT>
__device__ __forceinline__ void load_assign(const BatchParams& p, int w, int h, uint32_t tok, int* kk) {
#pragma unroll
  for (int t = 0; t < TT; ++t) kk[t] = min((int)__ldg(p.assign[w] + ((int64_t)t * p.H + h) * p.Nk + tok), p.K - 1);
}

// The scale (or zero) bytes of a token, all d/G of them.
__device__ __forceinline__ uint4 load_groups(const uint8_t* base, int64_t tok, int ng) {
  uint4 r = make_uint4(0, 0, 0, 0);
  switch (ng) {
    case 1: r.x = __ldg(base + tok); break;
    case 2: r.x = __ldg(reinterpret_cast<const uint16_t*>(base) + tok); break;
    case 4: r.x = __ldg(reinterpret_cast<const uint32_t*>(base) + tok); break;
    case 8: { const uint2 v = __ldg(reinterpret_cast<const uint2*>(base) + tok); r.x = v.x; r.y = v.y; break; }
    default: r = __ldg(reinterpret_cast<const uint4*>(base) + tok);
  }
  return r;
}
// The byte of chunk 4i + c (channels 32i + 8c .. + 7).
__device__ __forceinline__ uint32_t chunk_byte(const uint4& r, int i, int c, int ng, int lgG) {
  uint32_t w;
  int sh;
  if (ng == 16) { w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; sh = 8 * c; }
  else if (ng == 8) { w = i < 2 ? r.x : r.y; sh = 8 * (2 * (i & 1) + (c >> 1)); }
  else { w = r.x; sh = 8 * ((32 * i) >> lgG); }
  return (w >> sh) & 0xFFu;
}

// One rotated key for lane 4g + c: pair u = 4i + e of its 16 channel pairs is
// operand register u & 1 of k-step u >> 1, as bf16 (hi) and, when PRECISE, the
// bf16 of what that rounding left (lo).  `use(i, hi, lo)` is called per chunk.
template <int TT, bool PRECISE, class F>
__device__ __forceinline__ void rotated_key(const BatchParams& p, const float2* nlut, const Keys& ks, int64_t key, int c,
                                            F&& use) {
  const bool in = key < ks.n;
  const int64_t tok = in ? key : ks.n - 1;
  const int64_t pos = raw_key_pos(p, ks.tail, ks.h, ks.b, tok);
  uint16_t code[4];
  uint4 sc = make_uint4(0, 0, 0, 0), ze = make_uint4(0, 0, 0, 0);
  int kk[TT > 0 ? TT : 1];
  const int ng = kD >> p.lgG;
  const int64_t row = (int64_t)ks.h * p.Nk + tok;
  const __nv_bfloat16* dense = nullptr;
  if (ks.tail) {
    dense = p.tail[0] + (((int64_t)ks.b * p.H + ks.h) * p.Nt + tok) * kD;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) code[i] = __ldg(reinterpret_cast<const uint16_t*>(p.codes[0] + row * (kD / 4)) + 4 * i + c);
    sc = load_groups(p.scale[0], row, ng);
    if (!p.sym) ze = load_groups(p.zero[0], row, ng);
    load_assign<TT>(p, 0, ks.h, (uint32_t)tok, kk);
  }
  const float4* turn = reinterpret_cast<const float4*>(p.rope + rope_row(p, pos) * (kD / 2));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c0 = 8 * (4 * i + c);
    uint4 v;
    if (ks.tail) {
      v = __ldg(reinterpret_cast<const uint4*>(dense + c0));
    } else {
      const float2 sm = e4m3_pair(chunk_byte(sc, i, c, ng, p.lgG) | (chunk_byte(ze, i, c, ng, p.lgG) << 8));
      v = rebuild8<TT>(p, nlut, 0, ks.h, (uint32_t)tok, c0, code[i], sm.x, sm.y, kk);
    }
    const float4 t0 = __ldg(turn + c0 / 4), t1 = __ldg(turn + c0 / 4 + 1);
    const float2 cs[4] = {make_float2(t0.x, t0.y), make_float2(t0.z, t0.w), make_float2(t1.x, t1.y), make_float2(t1.z, t1.w)};
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = lo_f(x[e]), b = hi_f(x[e]);
      const float u = a * cs[e].x - b * cs[e].y, w = a * cs[e].y + b * cs[e].x;
      hi[e] = pack2(u, w);
      if (PRECISE) lo[e] = pack2(u - lo_f(hi[e]), w - hi_f(hi[e]));
    }
    use(i, hi, lo);
  }
}

// Chunk g + 8 i of a value, as packed bf16 pairs (zero past the end: the
// memory behind a tail's last token may hold anything).
template <int TT>
__device__ __forceinline__ uint4 value8(const BatchParams& p, const float2* nlut, const Keys& ks, int64_t key, int g, int i) {
  const int c0 = 8 * (g + 8 * i);
  if (key >= ks.n) return make_uint4(0, 0, 0, 0);
  if (ks.tail)
    return __ldg(reinterpret_cast<const uint4*>(p.tail[1] + (((int64_t)ks.b * p.H + ks.h) * p.Nt + key) * kD + c0));
  const int64_t row = (int64_t)ks.h * p.Nk + key;
  const int ng = kD >> p.lgG;
  const uint32_t code = __ldg(reinterpret_cast<const uint16_t*>(p.codes[1] + row * (kD / 4)) + g + 8 * i);
  const int64_t at = row * ng + (c0 >> p.lgG);
  const float2 sm = e4m3_pair((uint32_t)__ldg(p.scale[1] + at) | (p.sym ? 0u : (uint32_t)__ldg(p.zero[1] + at) << 8));
  int kk[TT > 0 ? TT : 1];
  load_assign<TT>(p, 1, ks.h, (uint32_t)key, kk);
  return rebuild8<TT>(p, nlut, 1, ks.h, (uint32_t)key, c0, code, sm.x, sm.y, kk);
}

__device__ __forceinline__ void fill_nlut(const BatchParams& p, float2* nlut) {
  if (threadIdx.x < 16) {
    const float off = p.sym ? 2.0f : 0.0f;
    nlut[threadIdx.x] = make_float2((float)(threadIdx.x & 3u) - off, (float)(threadIdx.x >> 2) - off);
  }
}

// Rotated queries of rows r0 .. r0+15 (those below r1; zeros otherwise) to
// shared memory, bf16 and, when PRECISE, the bf16 of the rest.
template <bool PRECISE>
__device__ __forceinline__ void rotate_queries(const BatchParams& p, int h, int64_t r0, int64_t r1, __nv_bfloat16* hi,
                                               __nv_bfloat16* lo) {
  for (int e = threadIdx.x; e < kRwRows * kD / 8; e += kRwThreads) {
    const int r = e >> 4, c0 = 8 * (e & 15);
    uint4 v = make_uint4(0, 0, 0, 0);
    int64_t pos = 0;
    if (r0 + r < r1) {
      pos = query_pos(p, r0 + r);
      v = __ldg(reinterpret_cast<const uint4*>(p.Q + query_row(p, h, r0 + r) * kD + c0));
    }
    const float2* turn = p.rope + rope_row(p, pos) * (kD / 2) + c0 / 2;
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t wh[4], wl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cs = __ldg(turn + i);
      const float a = lo_f(x[i]), b = hi_f(x[i]);
      const float u = a * cs.x - b * cs.y, w = a * cs.y + b * cs.x;
      wh[i] = pack2(u, w);
      wl[i] = pack2(u - lo_f(wh[i]), w - hi_f(wh[i]));
    }
    *reinterpret_cast<uint4*>(hi + r * kRwQStride + c0) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
    if (PRECISE) *reinterpret_cast<uint4*>(lo + r * kRwQStride + c0) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
  }
}

// Operand A of k-step kk for lane 4g + c from the rows in shared memory.
__device__ __forceinline__ void query_frag(const __nv_bfloat16* q, int g, int c, int kk, uint32_t (&a)[4]) {
  const int ch = 8 * (4 * (kk >> 1) + c) + 4 * (kk & 1);
  const uint2 x = *reinterpret_cast<const uint2*>(q + g * kRwQStride + ch);
  const uint2 y = *reinterpret_cast<const uint2*>(q + (g + 8) * kRwQStride + ch);
  a[0] = x.x; a[1] = y.x; a[2] = x.y; a[3] = y.y;
}

// Which keys and rows a CTA has: prefix CTAs first (range fastest, then row
// tile, then head), then the tails' (range, row tile, head, sequence).
struct Place {
  Keys ks;
  int64_t k0, k1, r0, r1;         // keys [k0, k1), rows [r0, r1)
  int slot;                       // of the partial results
};
__device__ __forceinline__ Place place_of(const BatchParams& p, int64_t id) {
  Place a;
  const int64_t first_tail = (int64_t)p.S1 * p.tiles1 * p.H;
  a.ks.tail = id >= first_tail;
  const int64_t e = a.ks.tail ? id - first_tail : id;
  const int S = a.ks.tail ? p.S2 : p.S1;
  const int64_t tiles = a.ks.tail ? p.tiles2 : p.tiles1;
  const int range = (int)(e % S);
  const int64_t tile = e / S % tiles, unit = e / S / tiles;
  a.ks.h = (int)(unit % p.H);
  a.ks.b = (int)(unit / p.H);
  a.ks.n = a.ks.tail ? tail_length(p, a.ks.b) : p.Nk;
  a.slot = a.ks.tail ? p.slot2 + range : range;
  a.r0 = (a.ks.tail ? a.ks.b * p.RB : 0) + tile * kRwRows;
  a.r1 = a.ks.tail ? (a.ks.b + 1) * p.RB : p.R;
  const int64_t steps = (a.ks.n + kRwStep - 1) / kRwStep;
  a.k0 = steps * range / S * kRwStep;
  a.k1 = steps * (range + 1) / S * kRwStep;
  return a;
}

// Partial attention of 16 rows over a range of keys.  With VALUES the rows'
// unnormalised O, maximum and sum; without, the maximum and sum alone, from
// scores whose operands carry 16 bits of mantissa (three products: high x
// high, low x high, high x low), so that the sums are good to fp32.
template <int TT, bool VALUES>
__global__ void __launch_bounds__(kRwThreads) qvg_attention_rows(const BatchParams p) {
  __shared__ float2 nlut[16];
  __shared__ __align__(16) __nv_bfloat16 sq[2][kRwRows * kRwQStride];
  __shared__ float sO[VALUES ? kRwRows * (kD + 4) : 1];
  __shared__ float2 sml[4][kRwRows];
  const Place a = place_of(p, blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t R = p.R;
  fill_nlut(p, nlut);
  rotate_queries<!VALUES>(p, a.ks.h, a.r0, a.r1, sq[0], sq[1]);
  __syncthreads();
  uint32_t qh[8][4], ql[8][4];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    query_frag(sq[0], g, c, kk, qh[kk]);
    if (!VALUES) query_frag(sq[1], g, c, kk, ql[kk]);
  }
  int limit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = a.r0 + g + 8 * i;
    limit[i] = r < a.r1 ? row_limit(p, query_pos(p, r)) : kLimitNone;
  }
  float m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
  float o[VALUES ? 16 : 1][4];
  if (VALUES) {
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
  }
#pragma unroll 1
  for (int64_t k = a.k0 + warp * kRwKeys; k < a.k1; k += kRwStep) {
    if (k >= a.ks.n) break;
    float s[2][4];
    float mt[2] = {kNoMax, kNoMax};
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
      rotated_key<TT, !VALUES>(p, nlut, a.ks, k + 8 * nt + g, c, [&](int i, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
        mma16816(s[nt], qh[2 * i], hi[0], hi[1]);
        mma16816(s[nt], qh[2 * i + 1], hi[2], hi[3]);
        if (!VALUES) {
          mma16816(s[nt], ql[2 * i], hi[0], hi[1]);
          mma16816(s[nt], ql[2 * i + 1], hi[2], hi[3]);
          mma16816(s[nt], qh[2 * i], lo[0], lo[1]);
          mma16816(s[nt], qh[2 * i + 1], lo[2], lo[3]);
        }
      });
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool sees = mask_pos(p, a.ks.tail, a.ks.h, a.ks.b, k + 8 * nt + 2 * c + (e & 1), a.ks.n) <= limit[e >> 1];
        s[nt][e] = sees ? s[nt][e] * p.sl : -INFINITY;
        mt[e >> 1] = fmaxf(mt[e >> 1], s[nt][e]);
      }
    }
    float alpha[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 1));
      mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 2));
      const float mn = fmaxf(m[i], mt[i]);
      alpha[i] = ex2(m[i] - mn);
      m[i] = mn;
      l[i] *= alpha[i];
    }
    uint32_t pa[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float w0 = ex2(s[nt][2 * i] - m[i]), w1 = ex2(s[nt][2 * i + 1] - m[i]);
        if (VALUES) {                 // the sum of the rounded weights, the ones the product uses
          pa[2 * nt + i] = pack2(w0, w1);
          l[i] += lo_f(pa[2 * nt + i]) + hi_f(pa[2 * nt + i]);
        } else {
          l[i] += w0 + w1;
        }
      }
    if (VALUES) {
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= alpha[0]; o[n][1] *= alpha[0];
          o[n][2] *= alpha[1]; o[n][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 v = value8<TT>(p, nlut, a.ks, k + 8 * (e >> 1) + 2 * c + (e & 1), g, i);
          w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          mma16816(o[8 * i + 2 * n], pa, __byte_perm(w[0][n], w[1][n], 0x5410), __byte_perm(w[2][n], w[3][n], 0x5410));
          mma16816(o[8 * i + 2 * n + 1], pa, __byte_perm(w[0][n], w[1][n], 0x7632), __byte_perm(w[2][n], w[3][n], 0x7632));
        }
      }
    }
  }
  // the four warps' results joined
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c == 0) sml[warp][g + 8 * i] = make_float2(m[i], l[i]);
  }
  __syncthreads();
  float f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float M = kNoMax, L = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sml[w][g + 8 * i].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) L += sml[w][g + 8 * i].y * ex2(sml[w][g + 8 * i].x - M);
    f[i] = ex2(m[i] - M);
    const int64_t r = a.r0 + g + 8 * i;
    if (warp == 0 && c == 0 && r < a.r1) p.part_ml[((int64_t)a.slot * p.H + a.ks.h) * R + r] = make_float2(M, L);
  }
  if (VALUES) {
    constexpr int ST = kD + 4;
    for (int w = 0; w < 4; ++w) {
      if (warp == w) {
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = 64 * (n >> 3) + 8 * (2 * c + (e & 1)) + (n & 7);
            float* d = sO + (g + 8 * (e >> 1)) * ST + ch;
            const float x = o[n][e] * f[e >> 1];
            *d = w == 0 ? x : *d + x;
          }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < kRwRows * kD / 4; e += kRwThreads) {
      const int r = e >> 5, c4 = e & 31;
      if (a.r0 + r < a.r1)
        reinterpret_cast<float4*>(p.part_O + (((int64_t)a.slot * p.H + a.ks.h) * R + a.r0 + r) * kD)[c4] =
            *reinterpret_cast<const float4*>(sO + r * ST + 4 * c4);
    }
  }
}

// log2 of a row's sum of 2^(sl s) over every range, from the partial results
// (a row that sees nothing: +inf, so that every weight 2^(x - inf) is 0).
__device__ __forceinline__ float row_lse(const BatchParams& p, int h, int64_t r) {
  const int S = p.slots;
  float M = kNoMax, L = 0.0f;
  for (int s = 0; s < S; ++s) M = fmaxf(M, __ldg(p.part_ml + ((int64_t)s * p.H + h) * p.R + r).x);
  for (int s = 0; s < S; ++s) {
    const float2 ml = __ldg(p.part_ml + ((int64_t)s * p.H + h) * p.R + r);
    L += ml.y * ex2(ml.x - M);
  }
  return L == 0.0f ? INFINITY : M + log2f(L);
}

// out[h][j] = received[h][j] + sum over the rows of 2^(sl s_rj - lse_r): the
// keys stay in registers while up to 64 rows at a time pass by, so a column's
// sum is taken by one warp in one order.
template <int TT>
__global__ void __launch_bounds__(kRwThreads) qvg_weights_rows(const BatchParams p, const float* received, float* out) {
  __shared__ float2 nlut[16];
  __shared__ __align__(16) __nv_bfloat16 sq[2][kRwChunk * kRwQStride];
  __shared__ float s_lse[kRwChunk];
  __shared__ int s_limit[kRwChunk];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t per = (p.Nk + kRwStep - 1) / kRwStep;
  Keys ks{(int)(blockIdx.x / per), 0, false, p.Nk};
  const int64_t k = (int64_t)(blockIdx.x % per) * kRwStep + warp * kRwKeys;
  fill_nlut(p, nlut);
  for (int64_t r0 = 0; r0 < p.R; r0 += kRwChunk) {
    __syncthreads();
    const int64_t rows = p.R - r0 < kRwChunk ? p.R - r0 : kRwChunk;
    const int tiles = (int)((rows + kRwRows - 1) / kRwRows);
    for (int t = 0; t < tiles; ++t)
      rotate_queries<true>(p, ks.h, r0 + t * kRwRows, p.R, sq[0] + t * kRwRows * kRwQStride, sq[1] + t * kRwRows * kRwQStride);
    if (threadIdx.x < tiles * kRwRows) {
      const bool in = threadIdx.x < rows;
      s_lse[threadIdx.x] = in ? row_lse(p, ks.h, r0 + threadIdx.x) : INFINITY;
      s_limit[threadIdx.x] = in ? row_limit(p, query_pos(p, r0 + threadIdx.x)) : kLimitNone;
    }
    __syncthreads();
    if (k >= p.Nk) continue;
#pragma unroll 1
    for (int nt = 0; nt < 2; ++nt) {
      uint32_t kh[16], kl[16];
      rotated_key<TT, true>(p, nlut, ks, k + 8 * nt + g, c, [&](int i, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) { kh[4 * i + e] = hi[e]; kl[4 * i + e] = lo[e]; }
      });
      const int64_t j = k + 8 * nt + 2 * c;
      const int pos[2] = {mask_pos(p, false, ks.h, 0, j, p.Nk), mask_pos(p, false, ks.h, 0, j + 1, p.Nk)};
      float sum[2] = {0.0f, 0.0f};
#pragma unroll 1
      for (int t = 0; t < tiles; ++t) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t qh[4], ql[4];
          query_frag(sq[0] + t * kRwRows * kRwQStride, g, c, kk, qh);
          query_frag(sq[1] + t * kRwRows * kRwQStride, g, c, kk, ql);
          mma16816(s, qh, kh[2 * kk], kh[2 * kk + 1]);
          mma16816(s, ql, kh[2 * kk], kh[2 * kk + 1]);
          mma16816(s, qh, kl[2 * kk], kl[2 * kk + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = t * kRwRows + g + 8 * (e >> 1);
          if (pos[e & 1] <= s_limit[r]) sum[e & 1] += ex2(fmaf(s[e], p.sl, -s_lse[r]));
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 4);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 8);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 16);
        if (g == 0 && j + e < p.Nk) {
          const int64_t at = (int64_t)ks.h * p.Nk + j + e;
          const float base = r0 > 0 ? out[at] : received != nullptr ? __ldg(received + at) : 0.0f;
          out[at] = base + sum[e];
        }
      }
    }
  }
}

// The ranges of every row joined: O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// with M = max_s m_s, rounded to bf16; zeros for a row that sees nothing.  A
// warp per row, a lane per four channels.
__global__ void __launch_bounds__(128) qvg_batch_merge(const BatchParams p) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.R * p.H) return;
  const int h = (int)(row / p.R);
  const int64_t r = row - (int64_t)h * p.R;
  const int S = p.slots;
  float M = kNoMax;
  for (int s = 0; s < S; ++s) M = fmaxf(M, __ldg(p.part_ml + s * p.R * p.H + row).x);
  float L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < S; ++s) {
    const float2 ml = __ldg(p.part_ml + s * p.R * p.H + row);
    if (!(ml.y > 0.0f) && ml.y == ml.y) continue;      // an empty range; a NaN sum goes on
    const float w = ex2(ml.x - M);
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.part_O + (s * p.R * p.H + row) * kD) + lane);
    acc.x += w * x.x; acc.y += w * x.y; acc.z += w * x.z; acc.w += w * x.w;
    L += w * ml.y;
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  reinterpret_cast<uint2*>(p.O + query_row(p, h, r) * kD)[lane] =
      make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
}

template <bool VALUES>
cudaError_t launch_rows(const BatchParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.S1 * p.tiles1 * p.H + p.S2 * p.tiles2 * p.H * p.B);
  switch (p.T) {
    case 0: qvg_attention_rows<0, VALUES><<<grid, kRwThreads, 0, s>>>(p); break;
    case 1: qvg_attention_rows<1, VALUES><<<grid, kRwThreads, 0, s>>>(p); break;
    case 2: qvg_attention_rows<2, VALUES><<<grid, kRwThreads, 0, s>>>(p); break;
    case 3: qvg_attention_rows<3, VALUES><<<grid, kRwThreads, 0, s>>>(p); break;
    case 4: qvg_attention_rows<4, VALUES><<<grid, kRwThreads, 0, s>>>(p); break;
    default: qvg_attention_rows<-1, VALUES><<<grid, kRwThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_partial(const BatchParams& p, bool values, cudaStream_t s) {
  return values ? launch_rows<true>(p, s) : launch_rows<false>(p, s);
}

cudaError_t launch_rows_weights(const BatchParams& p, const float* received, float* out, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.Nk + kRwStep - 1) / kRwStep * p.H);
  switch (p.T) {
    case 0: qvg_weights_rows<0><<<grid, kRwThreads, 0, s>>>(p, received, out); break;
    case 1: qvg_weights_rows<1><<<grid, kRwThreads, 0, s>>>(p, received, out); break;
    case 2: qvg_weights_rows<2><<<grid, kRwThreads, 0, s>>>(p, received, out); break;
    case 3: qvg_weights_rows<3><<<grid, kRwThreads, 0, s>>>(p, received, out); break;
    case 4: qvg_weights_rows<4><<<grid, kRwThreads, 0, s>>>(p, received, out); break;
    default: qvg_weights_rows<-1><<<grid, kRwThreads, 0, s>>>(p, received, out);
  }
  return cudaGetLastError();
}

cudaError_t launch_batch_merge(const BatchParams& p, cudaStream_t s) {
  qvg_batch_merge<<<(unsigned)((p.R * p.H + 3) / 4), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qvg
