// kernels_evict.cu -- qvg_evict: the tokens of a compressed cache that
// received the most attention weight are kept, and the packed streams close up
// over the others.
//
// A token's codes, scales and centroid indices do not depend on its
// neighbours, and the centroid tables stay as they are, so eviction moves
// bytes and quantises nothing again: the reconstruction of a kept token is
// the same, bit for bit.
//
// Two launches, or for few tokens the first alone:
//   qvg_evict_select  a cluster of CTAs per head: a radix select finds the
//                     weight of the last token that is kept, then one pass in
//                     token order writes the indices of the kept ones;
//   qvg_evict_gather  every kept token's bytes, position and weight.
// Half of 32 heads of 38,000 tokens (T = 4, G = 16): 25 and 27 us, the gather at
// 70 % of a copy's bandwidth.
#include "qvg_common.cuh"
#include "qvg_launch.h"

namespace qvg {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;                     // 11 + 11 + 10 bits of a weight's order
constexpr int kEvKeysSmem = 48 * 1024;            // weights of a CTA held in shared memory, at most
constexpr int kEvCluster = 8;                     // CTAs per head, at most
constexpr int kEvTile = 128;                      // kept tokens per gather CTA
// Kept tokens up to which a head's one CTA gathers them, too, two threads to each:
// 376 of 501 for 2 heads take 9 us on the device, and a call 2.4 us less than with
// two launches; with a thousand the gather alone in its CTAs is faster (11.8 us
// against 13.1).
constexpr int kEvFused = 512;

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
  int cluster;                    // CTAs per head
  int fused;                      // the select's CTAs gather, too
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

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// two words of another CTA of the cluster, at the place of `p` in this one's
// shared memory (8-byte aligned)
__device__ __forceinline__ uint2 cluster_words(const uint32_t* p, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// A token's d/G scale (or zero) bytes.
__device__ __forceinline__ uint4 load_row(const uint8_t* src, int n) {
  uint4 v = make_uint4(0, 0, 0, 0);
  switch (n) {
    case 16: v = __ldg(reinterpret_cast<const uint4*>(src)); break;
    case 8: { const uint2 x = __ldg(reinterpret_cast<const uint2*>(src)); v.x = x.x; v.y = x.y; break; }
    case 4: v.x = __ldg(reinterpret_cast<const uint32_t*>(src)); break;
    case 2: v.x = __ldg(reinterpret_cast<const uint16_t*>(src)); break;
    default: v.x = __ldg(src);
  }
  return v;
}
__device__ __forceinline__ void store_row(uint8_t* dst, const uint4& v, int n) {
  switch (n) {
    case 16: *reinterpret_cast<uint4*>(dst) = v; break;
    case 8: *reinterpret_cast<uint2*>(dst) = make_uint2(v.x, v.y); break;
    case 4: *reinterpret_cast<uint32_t*>(dst) = v.x; break;
    case 2: *reinterpret_cast<uint16_t*>(dst) = (uint16_t)v.x; break;
    default: *dst = (uint8_t)v.x;
  }
}

// Kept token i of head h, token f of the cache, by two threads (side 0 and 1):
// each moves a half of both caches' codes and one cache's scales, zero points and
// centroid indices, and one of them the position, the other the weight.  Everything
// a thread reads is on its way before it writes: stores between the loads made a
// chain of a dozen memory latencies of it.
__device__ __forceinline__ void gather_token(const EvictParams& p, int h, int64_t i, int32_t f, int side) {
  const int64_t out = (int64_t)h * p.keep + i, in = (int64_t)h * p.Nk + f;
  uint4 codes[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) codes[c] = __ldg(reinterpret_cast<const uint4*>(p.codes[c]) + 2 * in + side);
  const uint4 scale = load_row(p.scale[side] + in * p.ng, p.ng);
  uint4 zero = make_uint4(0, 0, 0, 0);
  if (p.zero[side] != nullptr) zero = load_row(p.zero[side] + in * p.ng, p.ng);
  uint8_t assign[kMaxT];
#pragma unroll
  for (int t = 0; t < kMaxT; ++t)
    if (t < p.T) assign[t] = __ldg(p.assign[side] + (int64_t)t * p.H * p.Nk + in);
  int64_t pos = f;
  float weight = 0.0f;
  if (side == 0 && p.pos_out != nullptr && p.k_pos != nullptr) pos = __ldg(p.k_pos + in);
  if (side == 1 && p.weights_out != nullptr) weight = __ldg(p.weights + in);
#pragma unroll
  for (int c = 0; c < 2; ++c) reinterpret_cast<uint4*>(p.codes_out[c])[2 * out + side] = codes[c];
  store_row(p.scale_out[side] + out * p.ng, scale, p.ng);
  if (p.zero[side] != nullptr) store_row(p.zero_out[side] + out * p.ng, zero, p.ng);
#pragma unroll
  for (int t = 0; t < kMaxT; ++t)
    if (t < p.T) p.assign_out[side][(int64_t)t * p.H * p.keep + out] = assign[t];
  if (side == 0 && p.pos_out != nullptr) p.pos_out[out] = pos;
  if (side == 1 && p.weights_out != nullptr) p.weights_out[out] = weight;
}

// A cluster of C CTAs per head, each with a run of its tokens.  need = keep -
// first - recent tokens are chosen from the middle [first, Nk - recent): all
// whose order lies above a threshold tau, and of those equal to it the first
// ones.  tau comes from three histograms, from the highest bits down, each over
// the tokens that agree with the bits found so far; every CTA adds up the
// cluster's through distributed shared memory and finds the same tau.
// Latency-bound (a pass over a CTA's weights in shared memory, a barrier and a
// scan, three times): one CTA a head took 64 us for 32 heads of 38,000 tokens.
__global__ void __launch_bounds__(kEvThreads, 1) qvg_evict_select(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(8) uint32_t hist[3][kEvBins];
  __shared__ unsigned long long warp_sums[32];
  __shared__ uint32_t s_bin, s_above;
  __shared__ __align__(8) uint32_t s_counts[2];
  const int C = p.cluster, rank = (int)(blockIdx.x % (unsigned)C), h = (int)(blockIdx.x / (unsigned)C);
  const float* w = p.weights + (int64_t)h * p.Nk;
  const int64_t slice = (p.Nk + C - 1) / C;
  const int64_t from = min(rank * slice, p.Nk), to = min(from + slice, p.Nk);
  const int64_t lo = max(p.first, from), hi = min(p.Nk - p.recent, to);      // of the middle, this CTA's
  const int64_t need = p.keep - p.first - p.recent;
  auto order_at = [&](int64_t i) { return p.in_smem ? keys[i - from] : weight_order(__ldg(w + i)); };
  for (int b = threadIdx.x; b < 3 * kEvBins; b += kEvThreads) (&hist[0][0])[b] = 0;
  if (p.in_smem)
    for (int64_t i = lo + threadIdx.x; i < hi; i += kEvThreads) keys[i - from] = weight_order(__ldg(w + i));
  __syncthreads();
  uint32_t tau = 0;
  int64_t left = need;                  // tokens still to be taken among those that agree with tau so far
  if (need > 0) {
    uint32_t mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
      const uint32_t field = (1u << bits) - 1u;
      for (int64_t i0 = lo; i0 < hi; i0 += kEvThreads) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t o = i < hi ? order_at(i) : 0u;
        const bool in = i < hi && (o & mask) == tau;
        const uint32_t bin = in ? (o >> shift) & field : 0xFFFFFFFFu;
        // a run of equal weights (zeros above all) meets in one bin: one add for the warp
        if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
          if (in && (threadIdx.x & 31) == 0) atomicAdd(&hist[pass][bin], 32u);
        } else if (in) {
          atomicAdd(&hist[pass][bin], 1u);
        }
      }
      if (C > 1) cluster_barrier(); else __syncthreads();
      // bins from the highest down: the first whose running count reaches `left`
      const int b1 = kEvBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
      unsigned long long c1 = 0, c0 = 0;
      if (C > 1) {
        uint2 v[kEvCluster];
#pragma unroll
        for (int r = 0; r < kEvCluster; ++r) v[r] = r < C ? cluster_words(&hist[pass][b0], (uint32_t)r) : make_uint2(0u, 0u);
#pragma unroll
        for (int r = 0; r < kEvCluster; ++r) { c0 += v[r].x; c1 += v[r].y; }
      } else {
        c1 = hist[pass][b1];
        c0 = hist[pass][b0];
      }
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
  const int64_t run = ((slice + kEvThreads - 1) / kEvThreads) | 1;
  const int64_t a = min(from + (int64_t)threadIdx.x * run, to), z = min(a + run, to);
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
  unsigned long long before = block_exclusive(((unsigned long long)sure << 32) | equal, warp_sums, &total);
  if (C > 1) {                          // and what the CTAs before this one hold
    if (threadIdx.x == 0) { s_counts[0] = (uint32_t)(total >> 32); s_counts[1] = (uint32_t)total; }
    cluster_barrier();
    uint2 v[kEvCluster];
#pragma unroll
    for (int r = 0; r < kEvCluster; ++r) v[r] = r < rank ? cluster_words(s_counts, (uint32_t)r) : make_uint2(0u, 0u);
#pragma unroll
    for (int r = 0; r < kEvCluster; ++r) before += ((unsigned long long)v[r].x << 32) + v[r].y;
  }
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
  if (C > 1) cluster_barrier();         // no CTA leaves while another reads its counts
  if (p.fused) {                        // one CTA to the head, few tokens: the gather, too
    __syncthreads();
    for (int64_t i = threadIdx.x >> 1; i < p.keep; i += kEvThreads / 2) gather_token(p, h, i, out[i], threadIdx.x & 1);
  }
}

// kEvTile kept tokens of one head, two threads to a token.
__global__ void __launch_bounds__(2 * kEvTile) qvg_evict_gather(const EvictParams p) {
  const unsigned tiles = (unsigned)((p.keep + kEvTile - 1) / kEvTile);
  const int h = (int)(blockIdx.x / tiles);
  const int64_t i = (int64_t)(blockIdx.x % tiles) * kEvTile + (threadIdx.x >> 1);
  if (i < p.keep) gather_token(p, h, i, __ldg(p.kept + (int64_t)h * p.keep + i), threadIdx.x & 1);
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
  // CTAs for a head: a power of two up to the portable cluster size, as long as
  // the heads leave SMs idle and a CTA has a few thousand tokens
  p.cluster = 1;
  while (p.cluster < kEvCluster && 2 * p.cluster * p.H <= device_sm_count() && p.Nk >= 2 * p.cluster * 2048) p.cluster *= 2;
  p.fused = p.cluster == 1 && a.keep <= kEvFused ? 1 : 0;
  const int64_t slice = (a.Nk + p.cluster - 1) / p.cluster;
  p.in_smem = slice <= kEvKeysSmem ? 1 : 0;
  const size_t smem = p.in_smem ? (size_t)slice * sizeof(uint32_t) : 0;
  // the histograms' static shared memory counts towards the 48 KB that need no attribute
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_evict_select),
                                      smem > 16 * 1024 ? kEvKeysSmem * sizeof(uint32_t) : 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.H * p.cluster));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  if ((e = cudaLaunchKernelEx(&cfg, qvg_evict_select, p)) != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess || p.fused) return e;
  qvg_evict_gather<<<(unsigned)((a.keep + kEvTile - 1) / kEvTile * a.H), 2 * kEvTile, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qvg
