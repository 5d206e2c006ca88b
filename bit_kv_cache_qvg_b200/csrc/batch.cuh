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
  // The keys are cut into ranges, each with a slot of partial results: the
  // prefix's from slot 0, the tails' from slot2.  A launch handles S1 ranges of
  // the prefix and S2 of every tail (0: another launch does).
  int S1, S2, slot2, slots;
  int64_t tiles1, tiles2;         // this launch's row tiles of a head, and of one sequence's rows
  float* part_O;                  // [slots][Hn][R][d]: unnormalised O of each range
  float2* part_ml;                // [slots][Hn][R]: (row maximum, row sum) of each range, base 2
  __nv_bfloat16* O;               // where a single slot needs no merge
  int row_tiles;                  // tiles of 16 rows to a CTA of the kernels for few rows
  int row_cuts;                   // cuts of the rows for the sums by key (weights of many rows)
  float* part_w;                  // [row_cuts][Hn][Nkp]: their sums, when there are several
  float* scores;                  // [Hn][R][Nkp]: the prefix's scores, base 2 (weights of few rows)
  int64_t Nkp;                    // Nk padded to 64
  int h0, Hn;                     // the launch's heads h0 .. h0 + Hn - 1: the workspace is theirs alone
  // Tensor-core operands, laid out as the kernels' shared memory wants them
  // (kernel_batch_expand.cu).
  int64_t nt1, nt2;               // tiles of 128 keys of the prefix and of a tail
  int64_t Rp, RBp;                // rows of a head, and of one sequence, padded to 256
  uint8_t* key_img[2];            // prefix, tails: [Hn][nt1], [B][Hn][nt2] tiles of 32 KB
  uint8_t* val_img[2];            // the same of V (or of the keys' low halves)
  uint8_t* row_img[2];            // rows by head [Hn][2][Rp][128 B], and by sequence [B][Hn][2][RBp][128 B]
  uint8_t* row_lo[2];             // the rows' low halves
  float* lse;                     // [Hn][Rp]: log2 of the rows' sums (weights)
  int* limits;                    // [Hn][Rp]
  uint32_t* status;
};

constexpr int kMaxSlots = 256;                    // ranges of the prefix and a tail together, at most
constexpr int64_t kImageBytes = 128 * kD * 2;     // one 128 x 128 bf16 operand tile

cudaError_t launch_rows_partial(const BatchParams& p, bool values, cudaStream_t s);      // kernel_attention_rows.cu
int rows_per_sm(const BatchParams& p, bool values);
cudaError_t launch_single_partial(const BatchParams& p, bool values, cudaStream_t s);    // kernel_attention_single.cu
int single_per_sm(const BatchParams& p, bool values);
cudaError_t launch_rows_weights(const BatchParams& p, const float* received, float* out, cudaStream_t s);
cudaError_t launch_batch_merge(const BatchParams& p, cudaStream_t s);
cudaError_t launch_batch_expand(const BatchParams& p, bool precise, cudaStream_t s);     // kernel_batch_expand.cu
cudaError_t launch_batch_attend(const BatchParams& p, cudaStream_t s);                   // kernel_batch_attend.cu
cudaError_t launch_batch_stats(const BatchParams& p, cudaStream_t s);                    // kernel_batch_weights.cu
cudaError_t launch_batch_weights(const BatchParams& p, float* lse, int* limits, const float* received, float* out, cudaStream_t s);

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
// Rows are below 2^23: 32-bit divisions (a 64-bit one takes about a hundred
// instructions).
__device__ __forceinline__ int64_t query_row(const BatchParams& p, int h, int64_t r) {
  const uint32_t b = (uint32_t)r / (uint32_t)p.RB;
  return ((int64_t)b * p.H + h) * p.RB + ((uint32_t)r - b * (uint32_t)p.RB);
}
__device__ __forceinline__ int64_t query_pos(const BatchParams& p, int64_t r) {
  const uint32_t b = (uint32_t)r / (uint32_t)p.RB;
  return __ldg(p.q_pos + b * p.Nq + ((uint32_t)r - b * (uint32_t)p.RB) % (uint32_t)p.Nq);
}
__device__ __forceinline__ int row_limit(const BatchParams& p, int64_t pos) {
  return pos < 0 ? kLimitNone : p.causal ? clamp_pos(pos) : kLimitAll;
}
// The limit of a row that sees no key, for the sums by key: its logarithm of +inf
// takes every finite score to a weight of 0, without a mask, and the operands of
// padding rows and behind the last row are zeros.  The queries of a causal row
// before every key may be anything: that one is masked.
__device__ __forceinline__ int unseen_limit(const BatchParams& p, int64_t pos) {
  return p.causal && pos >= 0 ? kLimitNone : kLimitAll;
}
__device__ __forceinline__ int64_t tail_length(const BatchParams& p, int b) {
  const int64_t n = p.tail_len != nullptr ? (int64_t)__ldg(p.tail_len + b) : p.Nt;
  return n < 0 ? 0 : n < p.Nt ? n : p.Nt;
}

// Row of the rotary table and position for the masks of key `key` (below the
// count n) of head h's prefix, or of sequence b's tail.
__device__ __forceinline__ int64_t raw_key_pos(const BatchParams& p, bool tail, int h, int b, int64_t key) {
  if (tail) return p.tail_pos != nullptr ? __ldg(p.tail_pos + (int64_t)b * p.Nt + key) : p.Nk + key;
  return p.k_pos != nullptr ? __ldg(p.k_pos + (int64_t)h * p.Nk + key) : key;
}
__device__ __forceinline__ int mask_pos(const BatchParams& p, bool tail, int h, int b, int64_t key, int64_t n) {
  return key < n ? clamp_pos(raw_key_pos(p, tail, h, b, key)) : kPosNever;
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
