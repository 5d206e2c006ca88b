// rebuild.cuh -- cached tokens rebuilt and rotated in registers, eight lanes to
// a token, for the kernels of qvg_attention_batch and qvg_attention_weights.
//
// What belongs to a token as a whole (its codes, scales, centroid indices, its
// row of the rotary table) is brought into shared memory by one thread each,
// in the form in which the lanes use it; the eight lanes then take two 8-channel
// chunks each (c and c + 8), so that a warp reads 128 contiguous bytes of a
// centroid row and writes 128 of its result.  The arithmetic is that of
// qvg_dequant_fused, about 75 instructions for 16 channels with one stage and
// 105 with two; loading and decoding the token's bytes in every lane took a
// third more.
#pragma once

#include <cuda_fp16.h>

#include "batch.cuh"

namespace qvg {
namespace {

// Operands of the scores are fp16: their rounding (2^-11) disturbs a score an
// eighth as much as bf16's, at the same rate of products.  Magnitudes beyond
// 65504 saturate; below 2^-14 the rounding is 2^-25 absolute.
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// (a + ib) e^(i phi) of a pair of channels as fp16: high halves, and (PRECISE)
// what their rounding left
template <bool PRECISE>
__device__ __forceinline__ void turn_pair(uint32_t x, float c, float s, uint32_t& hi, uint32_t& lo) {
  const float a = lo_f(x), b = hi_f(x);
  const float u = fmaf(a, c, -(b * s)), w = fmaf(a, s, b * c);
  hi = pack_half(u, w);
  if (PRECISE) {
    const float2 h = unpack_half(hi);
    lo = pack_half(u - h.x, w - h.y);
  }
}
// (cos, sin) of a chunk's four pairs in one 32-byte load: eight lanes read 256
// contiguous bytes (two 16-byte loads would touch each cache line twice)
__device__ __forceinline__ void load_turn(const float2* at, float (&t)[8]) {
  asm("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=f"(t[0]), "=f"(t[1]), "=f"(t[2]), "=f"(t[3]), "=f"(t[4]), "=f"(t[5]), "=f"(t[6]), "=f"(t[7])
      : "l"(at));
}
template <bool PRECISE>
__device__ __forceinline__ void turn_chunk(const float2* cs, uint4 x, uint4& hi, uint4& lo) {
  float t[8];
  load_turn(cs, t);
  turn_pair<PRECISE>(x.x, t[0], t[1], hi.x, lo.x);
  turn_pair<PRECISE>(x.y, t[2], t[3], hi.y, lo.y);
  turn_pair<PRECISE>(x.z, t[4], t[5], hi.z, lo.z);
  turn_pair<PRECISE>(x.w, t[6], t[7], hi.w, lo.w);
}

// nibble -> two codes (q, or u - 2 in the symmetric mode)
__device__ __forceinline__ void fill_nlut(const BatchParams& p, float2* nlut) {
  if (threadIdx.x < 16) {
    const float off = p.sym ? 2.0f : 0.0f;
    nlut[threadIdx.x] = make_float2((float)(threadIdx.x & 3u) - off, (float)(threadIdx.x >> 2) - off);
  }
}

// The bytes of NK tokens of one cache, in shared memory.  `sm` has room for
// NK * d/G pairs (scale, zero point).
template <int TT, int NK>
struct Tokens {
  static constexpr int TR = TT >= 0 ? (TT > 0 ? TT : 1) : kMaxT;
  uint4 codes[NK * 2];
  uint32_t row[TR][NK];           // byte offsets of the centroid rows in a head's stage table
  static __host__ __device__ constexpr size_t bytes(int ng) { return sizeof(Tokens) + (size_t)NK * ng * sizeof(float2); }
  __device__ __forceinline__ float2* sm() { return reinterpret_cast<float2*>(this + 1); }
  __device__ __forceinline__ const float2* sm() const { return reinterpret_cast<const float2*>(this + 1); }
};

// What one thread holds of a token between loading and storing it (so that the
// next block's bytes can be on their way while this one's are used).
template <int TT>
struct TokenBytes {
  static constexpr int TR = TT > 0 ? TT : 1;
  uint4 scale, zero;
  uint32_t k[TR];
};
__device__ __forceinline__ uint4 load_bytes(const uint8_t* base, int64_t tok, int ng) {
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
template <int TT>
__device__ __forceinline__ void load_token(const BatchParams& p, int w, int h, int tok, TokenBytes<TT>& x) {
  const int64_t at = (int64_t)h * p.Nk + tok;
  const int ng = kD >> p.lgG;
  x.scale = load_bytes(p.scale[w], at, ng);
  if (!p.sym) x.zero = load_bytes(p.zero[w], at, ng);
  if (TT > 0) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
      x.k[t] = min((uint32_t)__ldg(p.assign[w] + ((int64_t)t * p.H + h) * p.Nk + tok), (uint32_t)p.K - 1);
  }
}
template <int TT, int NK>
__device__ __forceinline__ void store_token(const BatchParams& p, int w, int h, int tok, const TokenBytes<TT>& x, Tokens<TT, NK>& to, int at) {
  const int ng = kD >> p.lgG;
  const uint32_t s[4] = {x.scale.x, x.scale.y, x.scale.z, x.scale.w}, z[4] = {x.zero.x, x.zero.y, x.zero.z, x.zero.w};
  float2* sm = to.sm() + at * ng;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * i >= ng) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (4 * i + e >= ng) break;
      const uint32_t sb = (s[i] >> (8 * e)) & 0xFFu, zb = p.sym ? 0u : (z[i] >> (8 * e)) & 0xFFu;
      sm[4 * i + e] = e4m3_pair(sb | (zb << 8));
    }
  }
  if (TT > 0) {
#pragma unroll
    for (int t = 0; t < TT; ++t) to.row[t][at] = x.k[t] * (kD * 2);
  } else if (TT < 0) {
    for (int t = 0; t < p.T; ++t)
      to.row[t][at] = min((uint32_t)__ldg(p.assign[w] + ((int64_t)t * p.H + h) * p.Nk + tok), (uint32_t)p.K - 1) * (kD * 2);
  }
}

// The lane's two chunks of a token as packed bf16 pairs.
template <int TT, int NK>
struct Rebuild {
  const uint8_t* tab;             // the head's first stage table, at the lane's chunk
  int64_t tab_stage;
  int ng, g0, g1, sym, T, c;

  __device__ __forceinline__ Rebuild(const BatchParams& p, int w, int h, int lane_c) {
    c = lane_c;
    ng = kD >> p.lgG;
    tab = reinterpret_cast<const uint8_t*>(p.tab[w] + (int64_t)h * p.K * kD + 8 * c);
    tab_stage = (int64_t)p.H * p.K * kD * 2;
    g0 = (8 * c) >> p.lgG;
    g1 = (64 + 8 * c) >> p.lgG;
    sym = p.sym;
    T = TT >= 0 ? TT : p.T;
  }
  __device__ __forceinline__ void operator()(const float2* nlut, const Tokens<TT, NK>& from, int at, uint4 (&out)[2]) const {
    constexpr int TR = TT > 0 ? TT : 1;
    uint4 rows[TR][2];
    if (TT > 0) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint4* row = reinterpret_cast<const uint4*>(tab + t * tab_stage + from.row[t][at]);
        rows[t][0] = __ldg(row);
        rows[t][1] = __ldg(row + 8);
      }
    }
    const uint16_t* code = reinterpret_cast<const uint16_t*>(from.codes + 2 * at) + c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 sm = from.sm()[at * ng + (i == 0 ? g0 : g1)];
      const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
      const uint32_t q8 = (uint32_t)code[8 * i] << 3;             // nibbles as byte offsets into the table
      float2 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 q = *reinterpret_cast<const float2*>(reinterpret_cast<const char*>(nlut) + ((q8 >> (4 * e)) & 0x78u));
        y[e] = sym ? __fmul2_rn(s2, q) : __ffma2_rn(s2, q, m2);
      }
      auto add = [&](const uint4& v) {
        y[0] = __fadd2_rn(y[0], make_float2(lo_f(v.x), hi_f(v.x)));
        y[1] = __fadd2_rn(y[1], make_float2(lo_f(v.y), hi_f(v.y)));
        y[2] = __fadd2_rn(y[2], make_float2(lo_f(v.z), hi_f(v.z)));
        y[3] = __fadd2_rn(y[3], make_float2(lo_f(v.w), hi_f(v.w)));
      };
      if (TT > 0) {
#pragma unroll
        for (int t = TT - 1; t >= 0; --t) add(rows[t][i]);
      } else if (TT < 0) {
        for (int t = T - 1; t >= 0; --t)
          add(__ldg(reinterpret_cast<const uint4*>(tab + t * tab_stage + from.row[t][at]) + 8 * i));
      }
      out[i] = make_uint4(pack2(y[0].x, y[0].y), pack2(y[1].x, y[1].y), pack2(y[2].x, y[2].y), pack2(y[3].x, y[3].y));
    }
  }
};

}  // namespace
}  // namespace qvg
