// rebuild.cuh -- cached tokens rebuilt and rotated in registers, eight lanes to
// a token, for the kernels of qvg_attention_batch and qvg_attention_weights.
#pragma once

#include "batch.cuh"

namespace qvg {
namespace {

// (a + ib) e^(i phi) of a pair of channels: high halves, and (PRECISE) what
// their rounding left
template <bool PRECISE>
__device__ __forceinline__ void turn_pair(uint32_t x, float c, float s, uint32_t& hi, uint32_t& lo) {
  const float a = lo_f(x), b = hi_f(x);
  const float u = fmaf(a, c, -(b * s)), w = fmaf(a, s, b * c);
  hi = pack2(u, w);
  if (PRECISE) lo = pack2(u - lo_f(hi), w - hi_f(hi));
}
template <bool PRECISE>
__device__ __forceinline__ void turn_chunk(const float4* cs, uint4 x, uint4& hi, uint4& lo) {
  const float4 t0 = __ldg(cs), t1 = __ldg(cs + 1);
  turn_pair<PRECISE>(x.x, t0.x, t0.y, hi.x, lo.x);
  turn_pair<PRECISE>(x.y, t0.z, t0.w, hi.y, lo.y);
  turn_pair<PRECISE>(x.z, t1.x, t1.y, hi.z, lo.z);
  turn_pair<PRECISE>(x.w, t1.z, t1.w, hi.w, lo.w);
}

// The reconstructed chunks c and c + 8 of a prefix token as packed bf16 pairs
// (the arithmetic of qvg_dequant_fused).  The pointers are the head's; offsets
// within a head fit in 32 bits.
template <int TT>
struct Rebuild {
  const uint8_t *codes, *scale, *zero, *assign;
  const __nv_bfloat16* tab;
  int64_t assign_stage, tab_stage;
  uint32_t top;                   // K - 1
  int lgng, g0, g1, sym, T;       // log2(d/G), the chunks' groups

  __device__ __forceinline__ Rebuild(const BatchParams& p, int w, int h, int c) {
    lgng = 7 - p.lgG;
    const int64_t row = (int64_t)h * p.Nk;
    codes = p.codes[w] + row * (kD / 4) + 2 * c;
    scale = p.scale[w] + (row << lgng);
    zero = p.zero[w] + (p.sym ? 0 : (row << lgng));
    assign = p.assign[w] + row;
    tab = p.tab[w] + (int64_t)h * p.K * kD + 8 * c;
    assign_stage = (int64_t)p.H * p.Nk;
    tab_stage = (int64_t)p.H * p.K * kD;
    top = (uint32_t)p.K - 1;
    g0 = (8 * c) >> p.lgG;
    g1 = (64 + 8 * c) >> p.lgG;
    sym = p.sym;
    T = TT >= 0 ? TT : p.T;
  }
  __device__ __forceinline__ void operator()(const float2* nlut, uint32_t tok, uint4 (&out)[2]) const {
    const uint32_t code[2] = {__ldg(reinterpret_cast<const uint16_t*>(codes + tok * 32u)),
                              __ldg(reinterpret_cast<const uint16_t*>(codes + tok * 32u + 16u))};
    const uint32_t at = tok << lgng;
    uint32_t sz[2] = {__ldg(scale + at + g0), __ldg(scale + at + g1)};
    if (!sym) {
      sz[0] |= (uint32_t)__ldg(zero + at + g0) << 8;
      sz[1] |= (uint32_t)__ldg(zero + at + g1) << 8;
    }
    constexpr int TR = TT > 0 ? TT : 1;
    uint4 rows[TR][2];
    if (TT > 0) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t k = min((uint32_t)__ldg(assign + t * assign_stage + tok), top);
        const uint4* row = reinterpret_cast<const uint4*>(tab + t * tab_stage + k * (uint32_t)kD);
        rows[t][0] = __ldg(row);
        rows[t][1] = __ldg(row + 8);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 sm = e4m3_pair(sz[i]);
      const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
      float2 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 q = nlut[(code[i] >> (4 * e)) & 0xFu];
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
        for (int t = T - 1; t >= 0; --t) {
          const uint32_t k = min((uint32_t)__ldg(assign + t * assign_stage + tok), top);
          add(__ldg(reinterpret_cast<const uint4*>(tab + t * tab_stage + k * (uint32_t)kD) + 8 * i));
        }
      }
      out[i] = make_uint4(pack2(y[0].x, y[0].y), pack2(y[1].x, y[1].y), pack2(y[2].x, y[2].y), pack2(y[3].x, y[3].y));
    }
  }
};

}  // namespace
}  // namespace qvg
