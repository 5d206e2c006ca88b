// kernel_attention_rows.cu -- the kernels of qvg_attention_batch and
// qvg_attention_weights for few rows, and the merge of partial results.
//
// For a row r with query q (rotated to its position) and the keys k_j it sees
// (rotated to theirs; the reconstructed prefix and its own tail),
//   s_j = q.k_j / sqrt(d),  O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m).
// All rows of a K/V head (every sequence, every query head of the group) read
// the same prefix: a CTA takes up to 64 of them and a range of the keys, 64 at a
// time.  Its four or eight warps rebuild the 64 keys and values into shared
// memory (rebuild.cuh), then multiply: mma.sync m16n8k16, fp16 operands for the
// scores and bf16 for O, fp32 sums.  For the scores a warp has 16 rows and as many
// of the 64 keys as leave no warp idle; the weights go through shared memory, and
// for O a warp has 32 channels of all rows, so that its sums take few registers.
// The weights are taken against a reference that the warps share and that rises
// only when a row's maximum exceeds it by more than 8 (base 2).  With few rows
// the rebuilding is the bound, and with it the latency of the centroid rows and
// the rotary table: small CTAs, three or four to an SM, overlap one's products
// with another's loads.  8 heads, 32 rows, 38,000 tokens (K = 256, T = 2): 83 us,
// the L1 data path 65 % busy.
#include <algorithm>

#include "batch.cuh"
#include "rebuild.cuh"

namespace qvg {
namespace {

__host__ __device__ constexpr int rw_warps(int mt, bool values) { return values || mt == 1 ? 4 : 8; }
constexpr int kRwKeys = 64;                       // keys per CTA and step
constexpr int kRwPPitch = kRwKeys + 8;            // the same for the weights
constexpr int kRwPitch = kD + 8;                  // padded row in shared memory (bf16): ldmatrix meets no bank twice

// D += A B, m16n8k16: fp16 operands for the scores, bf16 for O
__device__ __forceinline__ void mma_scores(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_values(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t shared_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Which keys and rows a CTA has: the prefix's CTAs first (range fastest, then
// row tile, then head), then the tails' (range, row tile, head, sequence).
struct Place {
  bool tail;
  int h, b, slot;
  int n;                          // keys of the prefix or tail (below 2^23)
  int k0, k1;                     // this CTA's keys
  int r0, r1;                     // its rows from r0, the unit's end r1 (below 2^23)
};
__device__ __forceinline__ Place place_of(const BatchParams& p, int rows_per_cta) {
  Place a;
  const int64_t first_tail = (int64_t)p.S1 * p.tiles1 * p.Hn;
  a.tail = blockIdx.x >= first_tail;
  const uint32_t e = (uint32_t)(a.tail ? blockIdx.x - first_tail : blockIdx.x);
  const uint32_t S = (uint32_t)(a.tail ? p.S2 : p.S1), tiles = (uint32_t)(a.tail ? p.tiles2 : p.tiles1);
  const uint32_t range = e % S, tile = e / S % tiles, unit = e / S / tiles;
  a.h = p.h0 + (int)(unit % (uint32_t)p.Hn);
  a.b = (int)(unit / (uint32_t)p.Hn);
  a.n = (int)(a.tail ? tail_length(p, a.b) : p.Nk);
  a.slot = (int)(a.tail ? p.slot2 + range : range);
  a.r0 = (int)((a.tail ? a.b * p.RB : 0) + (int64_t)tile * rows_per_cta);
  a.r1 = (int)(a.tail ? (a.b + 1) * p.RB : p.R);
  const int64_t steps = (a.n + kRwKeys - 1) / kRwKeys;
  a.k0 = (int)(steps * range / S) * kRwKeys;
  a.k1 = min((int)(steps * (range + 1) / S) * kRwKeys, a.n);
  return a;
}

// CTAs to an SM that the registers are cut for: 16 warps (of 64 rows 12) with the
// sums of O, 24 without, where eight warps to a CTA leave a thread half as many
// scores.  The weights of 64 rows over 16 heads of 11,011 tokens took 101 us with
// four warps and take 86; but 3 rows over 32 heads of 16,000 take 89 with four and would
// 100, attention of 32 rows over 8 heads of 38,000 takes 85 and would 95.
__host__ __device__ constexpr int rw_per_sm(int mt, bool values) { return rw_warps(mt, values) == 8 || mt == 4 ? 3 : 4; }

// Partial attention of 16 MT rows over a range of keys.  With VALUES the rows'
// unnormalised O, maximum and sum.  Without, the maximum and sum alone, and
// the prefix's scores themselves (base 2, -inf where masked) to p.scores: each
// from operands of two fp16 halves (three products: high x high, low x high,
// high x low), good to 2^-22, below 2^-3 to 2^-25 absolute.
template <int TT, int MT, bool VALUES>
__global__ void __launch_bounds__(32 * rw_warps(MT, VALUES), rw_per_sm(MT, VALUES)) qvg_attention_rows(const BatchParams p) {
  constexpr int W = rw_warps(MT, VALUES), kThreads = 32 * W;
  constexpr int kRows = 16 * MT;
  constexpr int kGroups = W / MT;                 // warps with the same rows
  constexpr int kWarpKeys = kRwKeys / kGroups;    // of a step's 64
  constexpr int kTiles = kWarpKeys / 8;           // tiles of 8 keys of a warp
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16* sK = reinterpret_cast<__nv_bfloat16*>(smem);        // keys (high halves)
  __nv_bfloat16* sV = sK + kRwKeys * kRwPitch;                       // values, or the keys' low halves
  __nv_bfloat16* sQ = sV + kRwKeys * kRwPitch;                       // rows (high halves, then low)
  float2* nlut = reinterpret_cast<float2*>(sQ + (VALUES ? 1 : 2) * kRows * kRwPitch);
  float2* sml = nlut + 16;                                           // [W][16]: a warp's rows: maxima, at the end sums
  float* sref = reinterpret_cast<float*>(sml + 16 * W);                // [64]: 2^(old - new) of a raised reference, by row
  int* sflag = reinterpret_cast<int*>(sref + 64);                    // [W]: a warp has a row that asks for it
  int* spos = sflag + W;                                                  // [2][64]: positions for the masks, by step
  uint32_t* turn = reinterpret_cast<uint32_t*>(spos + 2 * kRwKeys);  // rows of the rotary table
  using Block = Tokens<TT, kRwKeys>;
  Block& tk = *reinterpret_cast<Block*>(turn + kRwKeys);
  Block& tv = *reinterpret_cast<Block*>(reinterpret_cast<uint8_t*>(&tk) + Block::bytes(kD >> p.lgG));
  __nv_bfloat16* sP = reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<uint8_t*>(&tv) + Block::bytes(kD >> p.lgG));   // weights
  const Place a = place_of(p, kRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int mt = warp % MT, kg = warp / MT;       // the warp's rows and keys
  fill_nlut(p, nlut);
  // the rows, rotated
#pragma unroll (MT < 4 ? 2 * MT : 4)
  for (int i = 0; i < kRows * 16 / kThreads; ++i) {
    const int r = (int)(threadIdx.x >> 4) + i * (kThreads / 16), cb = threadIdx.x & 15;
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (a.r0 + r < a.r1) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.Q + query_row(p, a.h, a.r0 + r) * kD + 8 * cb));
      turn_chunk<!VALUES>(p.rope + rope_row(p, query_pos(p, a.r0 + r)) * (kD / 2) + 4 * cb, x, hi, lo);
    }
    *reinterpret_cast<uint4*>(sQ + r * kRwPitch + 8 * cb) = hi;
    if (!VALUES) *reinterpret_cast<uint4*>(sQ + (kRows + r) * kRwPitch + 8 * cb) = lo;
  }
  int limit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = a.r0 + 16 * mt + g + 8 * i;
    limit[i] = r < a.r1 ? row_limit(p, query_pos(p, r)) : kLimitNone;
  }
  float m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
  constexpr int kNt = 16 / W;                     // tiles of 8 channels of a warp
  float o[VALUES ? MT : 1][kNt][4];               // O of all rows and channels 8 kNt warp ..
  if (VALUES) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][n][e] = 0.0f;
  }
  // rebuilding: the lane's key of a pass and its chunks rc and rc + 8
  const int rc = threadIdx.x & 7, rkey = threadIdx.x >> 3;
  const Rebuild<TT, kRwKeys> keys(p, 0, a.h, rc);
  const Rebuild<TT, kRwKeys> vals(p, VALUES ? 1 : 0, a.h, rc);
  const __nv_bfloat16* tail_k = a.tail ? p.tail[0] + ((int64_t)a.b * p.H + a.h) * p.Nt * kD + 8 * rc : nullptr;
  const __nv_bfloat16* tail_v = a.tail && VALUES ? p.tail[1] + ((int64_t)a.b * p.H + a.h) * p.Nt * kD + 8 * rc : nullptr;
  // The bytes of a step's tokens, a step ahead in registers: threads 0 .. 63 have
  // a key each, 64 .. 127 a value, and the last 128 a half of both's codes.
  const int own = threadIdx.x & (kRwKeys - 1), w = threadIdx.x >> 6, part = (int)threadIdx.x - (kThreads - 2 * kRwKeys);
  TokenBytes<TT> held;
  uint4 held_codes[2];
  int64_t held_pos = 0;
  auto fetch = [&](int k0) {
    const int key = min(k0 + own, a.n - 1);
    if (w == 0) held_pos = raw_key_pos(p, a.tail, a.h, a.b, key);
    if (a.tail) return;
    if (w < (VALUES ? 2 : 1)) load_token<TT>(p, w, a.h, key, held);
    if (part >= 0) {
      const int64_t half = ((int64_t)a.h * p.Nk + min(k0 + (part >> 1), a.n - 1)) * 2 + (part & 1);
      held_codes[0] = __ldg(reinterpret_cast<const uint4*>(p.codes[0]) + half);
      if (VALUES) held_codes[1] = __ldg(reinterpret_cast<const uint4*>(p.codes[1]) + half);
    }
  };
  auto stash = [&](int k0, int parity) {
    const int key = k0 + own;
    if (w == 0) {
      spos[parity * kRwKeys + own] = key < a.n ? clamp_pos(held_pos) : kPosNever;
      turn[own] = (uint32_t)rope_row(p, held_pos);
    }
    if (a.tail) return;
    if (w < (VALUES ? 2 : 1)) store_token<TT, kRwKeys>(p, w, a.h, min(key, a.n - 1), held, w == 0 ? tk : tv, own);
    if (part >= 0) {
      tk.codes[part] = held_codes[0];
      if (VALUES) tv.codes[part] = held_codes[1];
    }
  };
  // ldmatrix: a warp's rows of Q, 8 keys of K (four 8 x 8 tiles along the channels), 16 keys of V
  const uint32_t aQ = shared_addr(sQ + (16 * mt + (lane & 15)) * kRwPitch + 8 * (lane >> 4));
  const uint32_t aK = shared_addr(sK + (kWarpKeys * kg + (lane & 7)) * kRwPitch + 8 * (lane >> 3));
  const uint32_t aV = shared_addr(sV + (lane & 15) * kRwPitch + 8 * kNt * warp + 8 * (lane >> 4));
  const uint32_t aP = shared_addr(sP + (lane & 15) * kRwPPitch + 8 * (lane >> 4));
  constexpr uint32_t kLow = kRwKeys * kRwPitch * 2;          // from the keys' high halves to the low ones
  if (a.k0 < a.k1) fetch(a.k0);
  int parity = 0;
#pragma unroll 1
  for (int k0 = a.k0; k0 < a.k1; k0 += kRwKeys, parity ^= 1) {
    stash(k0, parity);
    __syncthreads();                               // and the last step's products have read sK and sV
    if (k0 + kRwKeys < a.k1) fetch(k0 + kRwKeys);
#pragma unroll 2
    for (int pass = 0; pass < kRwKeys / (kThreads / 8); ++pass) {
      const int at = pass * (kThreads / 8) + rkey;
      uint4 x[2], y[2];
      if (!a.tail) {
        keys(nlut, tk, at, x);
        if (VALUES) vals(nlut, tv, at, y);
      } else {
        // a tail's tokens are bf16 rows already; behind its length zeros
        x[0] = x[1] = y[0] = y[1] = make_uint4(0, 0, 0, 0);
        if (k0 + at < a.n) {
          const uint4* row = reinterpret_cast<const uint4*>(tail_k + (int64_t)(k0 + at) * kD);
          x[0] = __ldg(row);
          x[1] = __ldg(row + 8);
          if (VALUES) {
            row = reinterpret_cast<const uint4*>(tail_v + (int64_t)(k0 + at) * kD);
            y[0] = __ldg(row);
            y[1] = __ldg(row + 8);
          }
        }
      }
      const float2* cs = p.rope + (int64_t)turn[at] * (kD / 2) + 4 * rc;
      uint4 hi[2], lo[2];
      turn_chunk<!VALUES>(cs, x[0], hi[0], lo[0]);
      turn_chunk<!VALUES>(cs + 32, x[1], hi[1], lo[1]);
      __nv_bfloat16* dk = sK + at * kRwPitch + 8 * rc;
      *reinterpret_cast<uint4*>(dk) = hi[0];
      *reinterpret_cast<uint4*>(dk + 64) = hi[1];
      __nv_bfloat16* dv = sV + at * kRwPitch + 8 * rc;
      *reinterpret_cast<uint4*>(dv) = VALUES ? y[0] : lo[0];
      *reinterpret_cast<uint4*>(dv + 64) = VALUES ? y[1] : lo[1];
    }
    __syncthreads();
    // scores of 16 rows x kWarpKeys keys
    float s[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {              // 32 channels at a time
      uint32_t q0[4], q1[4], u0[4], u1[4];
      ldm4(aQ + k4 * 64, q0);
      ldm4(aQ + k4 * 64 + 32, q1);
      if (!VALUES) {
        ldm4(aQ + kRows * kRwPitch * 2 + k4 * 64, u0);
        ldm4(aQ + kRows * kRwPitch * 2 + k4 * 64 + 32, u1);
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        uint32_t b[4];
        ldm4(aK + t * 8 * kRwPitch * 2 + k4 * 64, b);
        mma_scores(s[t], q0, b[0], b[1]);
        mma_scores(s[t], q1, b[2], b[3]);
        if (!VALUES) {
          uint32_t w[4];
          ldm4(aK + kLow + t * 8 * kRwPitch * 2 + k4 * 64, w);
          mma_scores(s[t], u0, b[0], b[1]);
          mma_scores(s[t], u1, b[2], b[3]);
          mma_scores(s[t], q0, w[0], w[1]);
          mma_scores(s[t], q1, w[2], w[3]);
        }
      }
    }
    float top[2] = {kNoMax, kNoMax};
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int2 pos = *reinterpret_cast<const int2*>(spos + parity * kRwKeys + kWarpKeys * kg + 8 * t + 2 * c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[t][2 * i] = pos.x <= limit[i] ? s[t][2 * i] * p.sl : -INFINITY;
        s[t][2 * i + 1] = pos.y <= limit[i] ? s[t][2 * i + 1] * p.sl : -INFINITY;
        top[i] = fmaxf(top[i], fmaxf(s[t][2 * i], s[t][2 * i + 1]));
      }
      if (!VALUES && !a.tail) {                    // the scores, for the sums by key
        const int key = k0 + kWarpKeys * kg + 8 * t + 2 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = a.r0 + 16 * mt + g + 8 * i;
          float* dst = p.scores + ((int64_t)(a.h - p.h0) * p.R + r) * p.Nkp + key;
          if (r < a.r1) *reinterpret_cast<float2*>(dst) = make_float2(s[t][2 * i], s[t][2 * i + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    if (VALUES) {
      // weights against the reference, of 16 rows x kWarpKeys keys
      float add[2];
      auto weigh = [&] {
        add[0] = add[1] = 0.0f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = pack2(ex2(s[t][2 * i] - m[i]), ex2(s[t][2 * i + 1] - m[i]));
            add[i] += lo_f(x) + hi_f(x);           // of the rounded weights, the ones the product uses
            *reinterpret_cast<uint32_t*>(sP + (16 * mt + g + 8 * i) * kRwPPitch + kWarpKeys * kg + 8 * t + 2 * c) = x;
          }
      };
      weigh();
      const bool raise = __any_sync(0xffffffffu, top[0] > m[0] + 8.0f || top[1] > m[1] + 8.0f);
      if (lane == 0) sflag[warp] = raise;
      __syncthreads();
      const int4 flags = *reinterpret_cast<const int4*>(sflag);        // of the four warps
      if (flags.x | flags.y | flags.z | flags.w) {
        // the reference rises to the rows' maxima: weights again, sums and O rescaled
        if (c == 0) { sml[warp * 16 + g].x = top[0]; sml[warp * 16 + g + 8].x = top[1]; }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mn = m[i];
#pragma unroll
          for (int w2 = 0; w2 < kGroups; ++w2) mn = fmaxf(mn, sml[(mt + w2 * MT) * 16 + g + 8 * i].x);
          const float f = ex2(m[i] - mn);
          if (kg == 0 && c == 0) sref[16 * mt + g + 8 * i] = f;
          l[i] *= f;
          m[i] = mn;
        }
        weigh();
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const float f0 = sref[16 * t + g], f1 = sref[16 * t + g + 8];
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            o[t][n][0] *= f0; o[t][n][1] *= f0;
            o[t][n][2] *= f1; o[t][n][3] *= f1;
          }
        }
      }
      l[0] += add[0];
      l[1] += add[1];
      // O of all rows and the warp's channels
#pragma unroll
      for (int k = 0; k < kRwKeys / 16; ++k) {
        uint32_t b[kNt / 2][4];
#pragma unroll
        for (int n = 0; n < kNt / 2; ++n) ldm4t(aV + k * 16 * kRwPitch * 2 + 32 * n, b[n]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t pa[4];
          ldm4(aP + (t * 16 * kRwPPitch + k * 16) * 2, pa);
#pragma unroll
          for (int n = 0; n < kNt; ++n) mma_values(o[t][n], pa, b[n / 2][2 * (n & 1)], b[n / 2][2 * (n & 1) + 1]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[i], top[i]);
        l[i] *= ex2(m[i] - mn);
        m[i] = mn;
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] += ex2(s[t][2 * i] - m[i]) + ex2(s[t][2 * i + 1] - m[i]);
    }
  }
  // the sums of the warps with the same rows joined (with VALUES their
  // references are equal), and O
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c == 0) sml[warp * 16 + g + 8 * i] = make_float2(m[i], l[i]);
  }
  __syncthreads();
  if (kg == 0 && c == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float M = kNoMax, L = 0.0f;
#pragma unroll
      for (int w2 = 0; w2 < kGroups; ++w2) M = fmaxf(M, sml[(mt + w2 * MT) * 16 + g + 8 * i].x);
#pragma unroll
      for (int w2 = 0; w2 < kGroups; ++w2) {
        const float2 x = sml[(mt + w2 * MT) * 16 + g + 8 * i];
        L += x.y * ex2(x.x - M);
      }
      const int r = a.r0 + 16 * mt + g + 8 * i;
      if (r < a.r1 && !(VALUES && p.slots == 1)) p.part_ml[((int64_t)a.slot * p.Hn + a.h - p.h0) * p.R + r] = make_float2(M, L);
    }
  }
  if (VALUES) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = a.r0 + 16 * t + g + 8 * i;
        if (r >= a.r1) continue;
        if (p.slots == 1) {                        // nothing to join: O itself
          float L = 0.0f;
#pragma unroll
          for (int w2 = 0; w2 < kGroups; ++w2) L += sml[(t + w2 * MT) * 16 + g + 8 * i].y;
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          uint32_t* row = reinterpret_cast<uint32_t*>(p.O + query_row(p, a.h, r) * kD + 8 * kNt * warp + 2 * c);
#pragma unroll
          for (int n = 0; n < kNt; ++n) row[4 * n] = pack2(o[t][n][2 * i] * inv, o[t][n][2 * i + 1] * inv);
          continue;
        }
        float* row = p.part_O + (((int64_t)a.slot * p.Hn + a.h - p.h0) * p.R + r) * kD + 8 * kNt * warp + 2 * c;
#pragma unroll
        for (int n = 0; n < kNt; ++n) *reinterpret_cast<float2*>(row + 8 * n) = make_float2(o[t][n][2 * i], o[t][n][2 * i + 1]);
      }
  }
}

// out[h][j] = received[h][j] + sum over the rows of 2^(x_rj - lse_r) from the
// scores x: a thread per four keys, the rows in order.  lse_r is log2 of row
// r's sum over every range (+inf for a row that sees nothing: weights 0).
__global__ void __launch_bounds__(128) qvg_weights_rows(const BatchParams p, const float* received, float* out) {
  extern __shared__ float lse[];
  const int per = (int)((p.Nk + 511) / 512), hl = (int)(blockIdx.x / per), h = p.h0 + hl;
  const int64_t stride = (int64_t)p.Hn * p.R;
  // as many lanes to a row (a power of two) as let all rows go at once, or two
  int per_row = 32;
  while (per_row > 2 && per_row * p.R > 128) per_row >>= 1;
  for (int r0 = 0; r0 < (int)p.R; r0 += 128 / per_row) {
    const int r = r0 + (int)threadIdx.x / per_row;
    float M = kNoMax, L = 0.0f;
    const float2* ml = p.part_ml + (int64_t)hl * p.R + min(r, (int)p.R - 1);
#pragma unroll 1
    for (int s0 = (int)threadIdx.x % per_row; s0 < p.slots; s0 += 8 * per_row) {
      float2 x[8];
      float mn = M, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int s = s0 + i * per_row;
        x[i] = s < p.slots ? __ldg(ml + s * stride) : make_float2(kNoMax, 0.0f);
        mn = fmaxf(mn, x[i].x);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i].y * ex2(x[i].x - mn);
      L = L * ex2(M - mn) + sum;
      M = mn;
    }
    for (int o = per_row >> 1; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o), mn = fmaxf(M, m2);
      L = L * ex2(M - mn) + l2 * ex2(m2 - mn);
      M = mn;
    }
    if (r < (int)p.R && threadIdx.x % per_row == 0) lse[r] = L == 0.0f ? INFINITY : M + log2f(L);
  }
  __syncthreads();
  const int64_t j = (int64_t)(blockIdx.x % per) * 512 + 4 * threadIdx.x;
  if (j >= p.Nk) return;
  const float* x = p.scores + (int64_t)hl * p.R * p.Nkp + j;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int64_t r = 0; r < p.R; ++r) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(x + r * p.Nkp));
    const float z = lse[r];
    sum.x += ex2(v.x - z); sum.y += ex2(v.y - z); sum.z += ex2(v.z - z); sum.w += ex2(v.w - z);
  }
  const float add[4] = {sum.x, sum.y, sum.z, sum.w};
  const int64_t at = (int64_t)h * p.Nk + j;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < p.Nk) out[at + e] = (received != nullptr ? received[at + e] : 0.0f) + add[e];
}

// The ranges of every row joined: O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// with M = max_s m_s, rounded to bf16; zeros for a row that sees nothing.  A
// lane per four channels.
__device__ __forceinline__ void store_joined(const BatchParams& p, int64_t row, const float4& acc, float L) {
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int hl = (int)(row / p.R);
  reinterpret_cast<uint2*>(p.O + query_row(p, p.h0 + hl, row - (int64_t)hl * p.R) * kD)[threadIdx.x & 31] =
      make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
}

// Few ranges: a warp per row, with a running maximum.
__global__ void __launch_bounds__(128) qvg_batch_merge(const BatchParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), stride = p.R * p.Hn;
  if (row >= stride) return;
  float M = kNoMax, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < p.slots; ++s) {
    const float2 ml = __ldg(p.part_ml + s * stride + row);
    if (ml.y == 0.0f) continue;                    // an empty range
    const float4 x = __ldg(reinterpret_cast<const float4*>(p.part_O + (s * stride + row) * kD) + lane);
    const float mn = fmaxf(M, ml.x), f = ex2(M - mn), w = ex2(ml.x - mn);
    acc.x = acc.x * f + w * x.x; acc.y = acc.y * f + w * x.y; acc.z = acc.z * f + w * x.z; acc.w = acc.w * f + w * x.w;
    L = L * f + w * ml.y;
    M = mn;
  }
  store_joined(p, row, acc, L);
}

// Many: four warps per row.  The factors first, a lane to a range, then every
// warp adds up every fourth range: with a running maximum the loads waited for
// one another (16 us for 64 ranges of 256 rows, now 11).
__global__ void __launch_bounds__(128) qvg_batch_merge_wide(const BatchParams p) {
  __shared__ float4 acc_s[4][32];
  __shared__ float factor[kMaxSlots];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x, stride = p.R * p.Hn;
  constexpr int kPer = kMaxSlots / 32;
  float2 ml[kPer];
  float M = kNoMax, L = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = 32 * i + lane;
    ml[i] = s < p.slots ? __ldg(p.part_ml + s * stride + row) : make_float2(kNoMax, 0.0f);
    M = fmaxf(M, ml[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float f = ml[i].y == 0.0f ? 0.0f : ex2(ml[i].x - M);         // an empty range has no O
    L += f * ml[i].y;
    if (warp == 0) factor[32 * i + lane] = f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  __syncthreads();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4* src = reinterpret_cast<const float4*>(p.part_O + row * kD) + lane;
#pragma unroll 8
  for (int s = warp; s < p.slots; s += 4) {
    const float f = factor[s];
    if (f == 0.0f) continue;
    const float4 x = __ldg(src + s * stride * (kD / 4));
    acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
  }
  acc_s[warp][lane] = acc;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 x = acc_s[w][lane];
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
  }
  store_joined(p, row, acc, L);
}

size_t rows_smem(int T, int G, int mt, bool values) {
  const size_t tiles = (size_t)(2 * kRwKeys + (values ? 1 : 2) * 16 * mt) * kRwPitch * 2;
  const size_t block = kRwKeys * (32 + sizeof(uint32_t) * (T >= 0 && T <= 4 ? (T > 0 ? T : 1) : kMaxT) + kD / G * sizeof(float2));
  return tiles + (16 + 16 * rw_warps(mt, values)) * sizeof(float2) + (64 + rw_warps(mt, values) + 3 * kRwKeys) * sizeof(int) + (values ? 2 : 1) * block +
         (values ? (size_t)16 * mt * kRwPPitch * 2 : 0);
}

template <int TT, int MT, bool VALUES>
cudaError_t launch_rows_mt(const BatchParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.S1 * p.tiles1 * p.Hn + p.S2 * p.tiles2 * p.Hn * p.B);
  const size_t smem = rows_smem(p.T, p.G, MT, VALUES);
  static_assert(Tokens<TT, kRwKeys>::bytes(1) == kRwKeys * (32 + sizeof(uint32_t) * Tokens<TT, kRwKeys>::TR + sizeof(float2)), "block size");
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_attention_rows<TT, MT, VALUES>), smem);
  if (e != cudaSuccess) return e;
  qvg_attention_rows<TT, MT, VALUES><<<grid, 32 * rw_warps(MT, VALUES), smem, s>>>(p);
  return cudaGetLastError();
}
template <int TT, bool VALUES>
cudaError_t launch_rows_t(const BatchParams& p, cudaStream_t s) {
  switch (p.row_tiles) {
    case 1: return launch_rows_mt<TT, 1, VALUES>(p, s);
    case 2: return launch_rows_mt<TT, 2, VALUES>(p, s);
    default: return launch_rows_mt<TT, 4, VALUES>(p, s);
  }
}
template <bool VALUES>
cudaError_t launch_rows(const BatchParams& p, cudaStream_t s) {
  switch (p.T) {
    case 0: return launch_rows_t<0, VALUES>(p, s);
    case 1: return launch_rows_t<1, VALUES>(p, s);
    case 2: return launch_rows_t<2, VALUES>(p, s);
    case 3: return launch_rows_t<3, VALUES>(p, s);
    case 4: return launch_rows_t<4, VALUES>(p, s);
    default: return launch_rows_t<-1, VALUES>(p, s);
  }
}

}  // namespace

// CTAs to an SM: fewer than their registers allow where the rows or small groups
// need more shared memory.
int rows_per_sm(const BatchParams& p, bool values) {
  const size_t smem = rows_smem(p.T, p.G, p.row_tiles, values) + 1024;
  const int n = (int)(size_t(228 * 1024) / smem);
  return std::min(n, rw_per_sm(p.row_tiles, values));
}

cudaError_t launch_rows_partial(const BatchParams& p, bool values, cudaStream_t s) {
  return values ? launch_rows<true>(p, s) : launch_rows<false>(p, s);
}

cudaError_t launch_rows_weights(const BatchParams& p, const float* received, float* out, cudaStream_t s) {
  qvg_weights_rows<<<(unsigned)((p.Nk + 511) / 512 * p.Hn), 128, p.R * sizeof(float), s>>>(p, received, out);
  return cudaGetLastError();
}

cudaError_t launch_batch_merge(const BatchParams& p, cudaStream_t s) {
  const int64_t rows = p.R * p.Hn;
  if (p.slots > 8) qvg_batch_merge_wide<<<(unsigned)rows, 128, 0, s>>>(p);
  else qvg_batch_merge<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qvg
