// batch.cuh -- the parameter block and the device helpers shared by the
// kernels of qvg_attention_batch and qvg_attention_weights.
//
// Rows.  The queries of K/V head h are the rows r = 0 .. R-1 of all B
// sequences, R = B * RB, RB = group * Nq; row r belongs to sequence r / RB,
// and its query vector is row (b * H + h) * RB + r % RB of Q (the queries of
// the heads that share a K/V head are contiguous in Q).
//
// Masks.  A row with a limit sees the keys at positions <= limit: its own
// position when causal, every key otherwise, none when its position is
// negative (padding).  Positions are compared as 32-bit integers.
#pragma once

#include "qvg_common.cuh"
#include "qvg_launch.h"

namespace qvg {

struct BatchParams {
  const uint8_t* codes[2];        // K, V: [H][Nk][d/4]
  const uint8_t* scale[2];        // [H][Nk][d/G]
  const uint8_t* zero[2];         // [H][Nk][d/G] (asymmetric mode)
  const uint8_t* assign[2];       // [T][H][Nk]
  const __nv_bfloat16* tab[2];    // [T][H][K][d]
  const __nv_bfloat16* Q;         // [B][H * group][Nq][d], before the rotary embedding
  const int64_t* q_pos;           // [B][Nq]
  const int64_t* k_pos;           // [H][Nk] or nullptr: token i at position i
  const __nv_bfloat16* tail[2];   // K, V: [B][H][Nt][d], keys before the rotary embedding
  const int64_t* tail_pos;        // [B][Nt] or nullptr: tail token i at position Nk + i
  const int32_t* tail_len;        // [B] or nullptr: Nt
  const float2* rope;             // [max_pos + 1][d/2]: (cos, sin) of p theta_i
  int64_t max_pos;
  int64_t Nk, Nq, Nt;
  int64_t R, RB;                  // rows per K/V head, and of one sequence
  int B, H, K, T, G, lgG, sym, causal;
  float sl;                       // log2(e) / sqrt(d)
  int S1, S2;                     // ranges of the prefix and of each tail
  int64_t tiles1, tiles2;         // row tiles of a head, and of one sequence's rows
  float* part_O;                  // [S1 + S2][H][R][d]: unnormalised O of each range
  float2* part_ml;                // [S1 + S2][H][R]: (row maximum, row sum) of each range, base 2
};

// The tensor-core kernels' plans (into tiles1, tiles2, S1 and S2) and launches.
int plan_batch_tc(BatchParams& p);                 // returns the CTAs per cluster
cudaError_t launch_batch_tc(const BatchParams& p, int pair, void* tables, cudaStream_t s);

namespace {

constexpr int kPosNever = 0x7FFFFFFF;             // a key that no row sees (past the end)
constexpr int kLimitAll = 0x7FFFFFFE;             // a row that sees every key
constexpr int kLimitNone = -0x7FFFFFFF - 1;       // a row that sees none
constexpr float kNoMax = -3.0e38f;                // row maximum before any key


__device__ __forceinline__ int clamp_pos(int64_t pos) {
  return (int)(pos < -0x7FFFFFFFll ? -0x7FFFFFFFll : pos > 0x7FFFFFFDll ? 0x7FFFFFFDll : pos);
}
__device__ __forceinline__ int64_t rope_row(const BatchParams& p, int64_t pos) {
  return pos < 0 ? 0 : pos > p.max_pos ? p.max_pos : pos;
}
__device__ __forceinline__ int64_t query_row(const BatchParams& p, int h, int64_t r) {
  const int64_t b = r / p.RB;
  return (b * p.H + h) * p.RB + (r - b * p.RB);
}
__device__ __forceinline__ int64_t query_pos(const BatchParams& p, int64_t r) {
  const int64_t b = r / p.RB;
  return __ldg(p.q_pos + b * p.Nq + (r - b * p.RB) % p.Nq);
}
__device__ __forceinline__ int row_limit(const BatchParams& p, int64_t pos) {
  return pos < 0 ? kLimitNone : p.causal ? clamp_pos(pos) : kLimitAll;
}
__device__ __forceinline__ int64_t tail_length(const BatchParams& p, int b) {
  const int64_t n = p.tail_len != nullptr ? (int64_t)__ldg(p.tail_len + b) : p.Nt;
  return n < 0 ? 0 : n < p.Nt ? n : p.Nt;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two E4M3 bytes (low byte first) as fp32 values (exact).
__device__ __forceinline__ float2 e4m3_pair(uint32_t pair16) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(pair16));
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}

}  // namespace
}  // namespace qvg
