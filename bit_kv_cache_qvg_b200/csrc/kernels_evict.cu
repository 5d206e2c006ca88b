// kernels_evict.cu -- qvg_evict: the tokens of a compressed cache that
// received the most attention weight are kept, and the packed streams close up
// over the others.
//
// A token's codes, scales and centroid indices do not depend on its
// neighbours, and the centroid tables stay as they are, so eviction moves
// bytes and quantises nothing again: the reconstruction of a kept token is
// the same, bit for bit.
//
// Two launches:
//   qvg_evict_select  one CTA per head: a radix select finds the weight of the
//                     last token that is kept, then one pass in token order
//                     writes the indices of the kept ones;
//   qvg_evict_gather  every kept token's bytes, position and weight.
#include "qvg_common.cuh"
#include "qvg_launch.h"

namespace qvg {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;                     // 11 + 11 + 10 bits of a weight's order
constexpr int kEvKeysSmem = 48 * 1024;            // weights of a head held in shared memory, at most
constexpr int kEvTile = 128;                      // kept tokens per gather CTA

// The order of the weights as unsigned integers: larger weight, larger
// integer; NaN below everything, the two zeros equal.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0u;
  if (w == 0.0f) w = 0.0f;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictParams {
  const float* weights;           // [H][Nk]
  const int64_t* k_pos;           // [H][Nk] or nullptr (token i at position i)
  int32_t* kept;                  // [H][keep]
  int64_t* pos_out;               // [H][keep] or nullptr
  float* weights_out;             // [H][keep] or nullptr
  const uint8_t* codes[2];        // K, V streams
  const uint8_t* scale[2];
  const uint8_t* zero[2];         // nullptr when symmetric
  const uint8_t* assign[2];
  uint8_t* codes_out[2];
  uint8_t* scale_out[2];
  uint8_t* zero_out[2];
  uint8_t* assign_out[2];
  int64_t Nk, keep, first, recent;
  int H, T, ng;
  int in_smem;
};

// Exclusive prefix sum over the CTA of two counts packed in 64 bits; *total
// gets the sum.
__device__ __forceinline__ unsigned long long block_exclusive(unsigned long long v, unsigned long long* warp_sums,
                                                              unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const unsigned long long base = warp > 0 ? warp_sums[warp - 1] : 0ull;
  *total = warp_sums[31];
  __syncthreads();
  return base + x - v;
}

// One CTA per head.  need = keep - first - recent tokens are chosen from the
// middle [first, Nk - recent): all whose order lies above a threshold tau,
// and of those equal to it the first ones.  tau comes from three histograms,
// from the highest bits down, each over the tokens that agree with the bits
// found so far.
__global__ void __launch_bounds__(kEvThreads, 1) qvg_evict_select(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kEvBins];
  __shared__ unsigned long long warp_sums[32];
  __shared__ uint32_t s_bin, s_above;
  const int h = blockIdx.x;
  const float* w = p.weights + (int64_t)h * p.Nk;
  const int64_t lo = p.first, hi = p.Nk - p.recent;
  const int64_t need = p.keep - p.first - p.recent;
  auto order_at = [&](int64_t i) { return p.in_smem ? keys[i] : weight_order(__ldg(w + i)); };
  if (p.in_smem)
    for (int64_t i = lo + threadIdx.x; i < hi; i += kEvThreads) keys[i] = weight_order(__ldg(w + i));
  uint32_t tau = 0;
  int64_t left = need;                  // tokens still to be taken among those that agree with tau so far
  if (need > 0) {
    uint32_t mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
      const uint32_t field = (1u << bits) - 1u;
      for (int b = threadIdx.x; b < kEvBins; b += kEvThreads) hist[b] = 0;
      __syncthreads();
      for (int64_t i0 = lo; i0 < hi; i0 += kEvThreads) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t o = i < hi ? order_at(i) : 0u;
        const bool in = i < hi && (o & mask) == tau;
        const uint32_t bin = in ? (o >> shift) & field : 0xFFFFFFFFu;
        // equal weights (zeros above all) meet in one bin: one add for the lanes that agree
        const uint32_t same = __match_any_sync(0xffffffffu, bin);
        if (in && (int)(threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&hist[bin], (uint32_t)__popc(same));
      }
      __syncthreads();
      // bins from the highest down: the first whose running count reaches `left`
      const int b1 = kEvBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
      const unsigned long long c1 = hist[b1], c0 = hist[b0];
      unsigned long long total;
      const unsigned long long above = block_exclusive(c1 + c0, warp_sums, &total);
      if (above < (unsigned long long)left && above + c1 + c0 >= (unsigned long long)left) {
        const bool upper = above + c1 >= (unsigned long long)left;
        s_bin = (uint32_t)(upper ? b1 : b0);
        s_above = (uint32_t)(upper ? above : above + c1);
      }
      __syncthreads();
      tau |= s_bin << shift;
      mask |= field << shift;
      left -= s_above;
      __syncthreads();
    }
  }
  // `left` of the tokens equal to tau are kept, the first ones.  Every thread
  // takes a run of consecutive tokens; an odd length keeps a warp's reads of
  // shared memory in distinct banks.
  const int64_t run = ((p.Nk + kEvThreads - 1) / kEvThreads) | 1;
  const int64_t a = (int64_t)threadIdx.x * run < p.Nk ? (int64_t)threadIdx.x * run : p.Nk;
  const int64_t z = a + run < p.Nk ? a + run : p.Nk;
  uint32_t sure = 0, equal = 0;
  for (int64_t i = a; i < z; ++i) {
    if (i < lo || i >= hi) { ++sure; continue; }
    if (need > 0) {
      const uint32_t o = order_at(i);
      sure += o > tau;
      equal += o == tau;
    }
  }
  unsigned long long total;
  const unsigned long long before = block_exclusive(((unsigned long long)sure << 32) | equal, warp_sums, &total);
  int64_t eq = (int64_t)(before & 0xFFFFFFFFull);
  int64_t at = (int64_t)(before >> 32) + (eq < left ? eq : left);
  int32_t* out = p.kept + (int64_t)h * p.keep;
  for (int64_t i = a; i < z; ++i) {
    bool take = i < lo || i >= hi;
    if (!take && need > 0) {
      const uint32_t o = order_at(i);
      take = o > tau;
      if (o == tau) take = eq++ < left;
    }
    if (take) out[at++] = (int32_t)i;
  }
}

__device__ __forceinline__ void copy_row(const uint8_t* src, uint8_t* dst, int n) {
  switch (n) {
    case 16: *reinterpret_cast<uint4*>(dst) = __ldg(reinterpret_cast<const uint4*>(src)); break;
    case 8: *reinterpret_cast<uint2*>(dst) = __ldg(reinterpret_cast<const uint2*>(src)); break;
    case 4: *reinterpret_cast<uint32_t*>(dst) = __ldg(reinterpret_cast<const uint32_t*>(src)); break;
    case 2: *reinterpret_cast<uint16_t*>(dst) = __ldg(reinterpret_cast<const uint16_t*>(src)); break;
    default: *dst = __ldg(src);
  }
}

// kEvTile kept tokens of one head: their codes (two 16-byte halves), scale
// and zero rows (d/G bytes), centroid indices, positions and weights.
__global__ void __launch_bounds__(256) qvg_evict_gather(const EvictParams p) {
  __shared__ int32_t from[kEvTile];
  const int h = blockIdx.y;
  const int64_t i0 = (int64_t)blockIdx.x * kEvTile;
  const int n = (int)(p.keep - i0 < kEvTile ? p.keep - i0 : kEvTile);
  const int64_t in0 = (int64_t)h * p.Nk, out0 = (int64_t)h * p.keep + i0;
  if (threadIdx.x < n) {
    const int32_t f = __ldg(p.kept + out0 + threadIdx.x);
    from[threadIdx.x] = f;
    if (p.pos_out != nullptr) p.pos_out[out0 + threadIdx.x] = p.k_pos != nullptr ? __ldg(p.k_pos + in0 + f) : (int64_t)f;
    if (p.weights_out != nullptr) p.weights_out[out0 + threadIdx.x] = __ldg(p.weights + in0 + f);
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    for (int e = threadIdx.x; e < 2 * n; e += 256) {
      const int i = e >> 1, half = e & 1;
      reinterpret_cast<uint4*>(p.codes_out[c])[2 * (out0 + i) + half] =
          __ldg(reinterpret_cast<const uint4*>(p.codes[c]) + 2 * (in0 + from[i]) + half);
    }
    for (int i = threadIdx.x; i < n; i += 256) {
      copy_row(p.scale[c] + (in0 + from[i]) * p.ng, p.scale_out[c] + (out0 + i) * p.ng, p.ng);
      if (p.zero[c] != nullptr) copy_row(p.zero[c] + (in0 + from[i]) * p.ng, p.zero_out[c] + (out0 + i) * p.ng, p.ng);
    }
    for (int e = threadIdx.x; e < p.T * n; e += 256) {
      const int t = e / n, i = e - t * n;
      p.assign_out[c][(int64_t)t * p.H * p.keep + out0 + i] = __ldg(p.assign[c] + (int64_t)t * p.H * p.Nk + in0 + from[i]);
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  EvictParams p{};
  p.weights = a.weights; p.k_pos = a.k_pos; p.kept = a.kept; p.pos_out = a.pos_out; p.weights_out = a.weights_out;
  const qvg_packed* in[2] = {a.k, a.v};
  const qvg_packed* out[2] = {a.k_out, a.v_out};
  for (int c = 0; c < 2; ++c) {
    p.codes[c] = in[c]->codes; p.scale[c] = in[c]->scale; p.assign[c] = in[c]->assign;
    p.zero[c] = a.sym ? nullptr : in[c]->zero;
    p.codes_out[c] = out[c]->codes; p.scale_out[c] = out[c]->scale; p.zero_out[c] = out[c]->zero;
    p.assign_out[c] = out[c]->assign;
  }
  p.Nk = a.Nk; p.keep = a.keep; p.first = a.first; p.recent = a.recent;
  p.H = a.H; p.T = a.T; p.ng = kD / a.G;
  p.in_smem = a.Nk <= kEvKeysSmem ? 1 : 0;
  const size_t smem = p.in_smem ? (size_t)a.Nk * sizeof(uint32_t) : 0;
  // the histogram's static shared memory counts towards the 48 KB that need no attribute
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_evict_select),
                                      smem > 32 * 1024 ? kEvKeysSmem * sizeof(uint32_t) : 0);
  if (e != cudaSuccess) return e;
  qvg_evict_select<<<(unsigned)a.H, kEvThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.keep + kEvTile - 1) / kEvTile), (unsigned)a.H);
  qvg_evict_gather<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qvg
