// kernel_attention_single.cu -- the kernel of qvg_attention_batch for one row a
// head, a token of one sequence, and of qvg_attention_weights for one or two.
//
// With so few rows a tensor-core tile would be mostly padding, and the way there
// (keys rounded to bf16, stored, read back as operands) costs more than the
// products.  Here a key has no operand tile: eight lanes take it (two
// 8-channel chunks each), rebuild and rotate it, multiply with the rotated
// query and add up over the lanes; then they rebuild the value and add it,
// weighted, to sums over the same 16 channels, all in fp32.  A warp works on four
// keys at a time with a maximum and sum for each of its four groups of lanes, and meets
// the others only at the end.  The tokens' bytes come 32 at a time through
// shared memory (rebuild.cuh); loading them a block ahead cost registers, and
// with them warps, worth more (six CTAs to an SM); at their 80
// registers what a lane holds of a block's bytes between its loads and its stores
// spills (192 bytes a thread with one stage, 256 with two, 544 with four).  Bound by the instructions of
// the rebuilding and the latency of the centroid rows: 32 heads of 28,011 tokens
// (K = 256, T = 1) take 142 us, 59 % of the issue slots and of the L1 data path;
// one CTA of 24 warps, whose head's tables stay in the SM's L1, made it 158.
#include <algorithm>

#include "batch.cuh"
#include "rebuild.cuh"

namespace qvg {
namespace {

constexpr int kSgThreads = 128;                   // 4 warps
constexpr int kSgKeys = 32;                       // keys per block of a warp
constexpr int kSgPerSm = 6;                       // CTAs to an SM (four for two rows)

// The keys and rows of a CTA: the prefix's CTAs first (range fastest, then
// head), then the tails' (range, head, sequence).
struct SgPlace {
  bool tail;
  int h, b, slot;
  int n;                          // keys of the prefix or tail (below 2^23)
  int k0, k1;                     // this CTA's
  int r0, rows;
};
__device__ __forceinline__ SgPlace sg_place(const BatchParams& p) {
  SgPlace a;
  const uint32_t first_tail = (uint32_t)(p.S1 * p.Hn);
  a.tail = blockIdx.x >= first_tail;
  const uint32_t e = a.tail ? blockIdx.x - first_tail : blockIdx.x;
  const uint32_t S = (uint32_t)(a.tail ? p.S2 : p.S1), range = e % S, unit = e / S;
  a.h = p.h0 + (int)(unit % (uint32_t)p.Hn);
  a.b = (int)(unit / (uint32_t)p.Hn);
  a.n = (int)(a.tail ? tail_length(p, a.b) : p.Nk);
  a.slot = (int)(a.tail ? p.slot2 + range : range);
  a.r0 = a.tail ? a.b * (int)p.RB : 0;
  a.rows = (int)(a.tail ? p.RB : p.R);
  const int64_t blocks = (a.n + kSgKeys - 1) / kSgKeys;
  a.k0 = (int)(blocks * range / S) * kSgKeys;
  a.k1 = min((int)(blocks * (range + 1) / S) * kSgKeys, a.n);
  return a;
}

// NR rows over a range of keys.  With VALUES their unnormalised O, maximum and
// sum; without, the maximum and sum, and the prefix's scores (base 2, -inf where
// masked) to p.scores.
template <int TT, int NR, bool VALUES>
__global__ void __launch_bounds__(kSgThreads, NR == 1 ? kSgPerSm : 4) qvg_attention_single(const BatchParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7, group = lane >> 3;
  using Block = Tokens<TT, kSgKeys>;
  const size_t block_bytes = Block::bytes(kD >> p.lgG);
  float2* nlut = reinterpret_cast<float2*>(smem);
  float* joined = reinterpret_cast<float*>(nlut + 16);               // [4 warps][NR][d + 2] at the end
  int* spos = reinterpret_cast<int*>(joined + 4 * NR * (kD + 4)) + warp * 2 * kSgKeys;
  uint32_t* turn = reinterpret_cast<uint32_t*>(spos + kSgKeys);
  uint8_t* blocks = reinterpret_cast<uint8_t*>(joined + 4 * NR * (kD + 4)) + 4 * 2 * kSgKeys * sizeof(int);
  Block& tk = *reinterpret_cast<Block*>(blocks + warp * (VALUES ? 2 : 1) * block_bytes);
  Block& tv = *reinterpret_cast<Block*>(blocks + (warp * 2 + 1) * block_bytes);     // VALUES only
  const SgPlace a = sg_place(p);
  fill_nlut(p, nlut);
  // the rotated queries' 16 channels of this lane
  float q[NR][16];
  int limit[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    limit[r] = kLimitNone;
#pragma unroll
    for (int e = 0; e < 16; ++e) q[r][e] = 0.0f;
    if (r < a.rows) {
      const int64_t pos = query_pos(p, a.r0 + r);
      limit[r] = row_limit(p, pos);
      const __nv_bfloat16* row = p.Q + query_row(p, a.h, a.r0 + r) * kD + 8 * c;
      const float2* cs = p.rope + rope_row(p, pos) * (kD / 2) + 4 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + 64 * i));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        float t[8];
        load_turn(cs + 32 * i, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {              // scaled once here: scores come in base 2
          const float u = lo_f(w[e]) * p.sl, v = hi_f(w[e]) * p.sl;
          q[r][8 * i + 2 * e] = fmaf(u, t[2 * e], -(v * t[2 * e + 1]));
          q[r][8 * i + 2 * e + 1] = fmaf(u, t[2 * e + 1], v * t[2 * e]);
        }
      }
    }
  }
  float m[NR], l[NR];
  float2 o[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m[r] = kNoMax;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[r][e] = make_float2(0.0f, 0.0f);
  }
  const Rebuild<TT, kSgKeys> keys(p, 0, a.h, c);
  const Rebuild<TT, kSgKeys> vals(p, VALUES ? 1 : 0, a.h, c);
  const int64_t tail0 = ((int64_t)a.b * p.H + a.h) * p.Nt;
  // a lane's token of a block: a key and a value, and half the codes of two of each
  TokenBytes<TT> hk, hv;
  uint4 ck[2], cv[2];
  int64_t pos = 0;
  auto fetch = [&](int k0) {
    const int key = min(k0 + lane, a.n - 1);
    pos = raw_key_pos(p, a.tail, a.h, a.b, key);
    if (a.tail) return;
    load_token<TT>(p, 0, a.h, key, hk);
    if (VALUES) load_token<TT>(p, 1, a.h, key, hv);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t half = ((int64_t)a.h * p.Nk + min(k0 + 16 * i + (lane >> 1), a.n - 1)) * 2 + (lane & 1);
      ck[i] = __ldg(reinterpret_cast<const uint4*>(p.codes[0]) + half);
      if (VALUES) cv[i] = __ldg(reinterpret_cast<const uint4*>(p.codes[1]) + half);
    }
  };
  __syncthreads();
  // blocks of 32 keys, or a quarter of a short range
  const int per = min(kSgKeys, (a.k1 - a.k0 + 31) / 32 * 8), first = a.k0 + warp * per;
#pragma unroll 1
  for (int k0 = first; k0 < a.k1; k0 += 4 * per) {
    fetch(k0);
    __syncwarp();
    spos[lane] = k0 + lane < a.n ? clamp_pos(pos) : kPosNever;
    turn[lane] = (uint32_t)rope_row(p, pos);
    if (!a.tail) {
      const int key = min(k0 + lane, a.n - 1);
      store_token<TT, kSgKeys>(p, 0, a.h, key, hk, tk, lane);
      if (VALUES) store_token<TT, kSgKeys>(p, 1, a.h, key, hv, tv, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tk.codes[32 * i + lane] = ck[i];
        if (VALUES) tv.codes[32 * i + lane] = cv[i];
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int it = 0; it < per; it += 8)
#pragma unroll
    for (int u = 0; u < 2; ++u) {                  // two keys of a group at a time
      const int at = it + 4 * u + group;
      uint4 x[2], y[2];
      if (!a.tail) {
        keys(nlut, tk, at, x);
        if (VALUES) vals(nlut, tv, at, y);
      } else {
        x[0] = x[1] = y[0] = y[1] = make_uint4(0, 0, 0, 0);
        if (k0 + at < a.n) {
          const uint4* row = reinterpret_cast<const uint4*>(p.tail[0] + (tail0 + k0 + at) * kD + 8 * c);
          x[0] = __ldg(row);
          x[1] = __ldg(row + 8);
          if (VALUES) {
            row = reinterpret_cast<const uint4*>(p.tail[1] + (tail0 + k0 + at) * kD + 8 * c);
            y[0] = __ldg(row);
            y[1] = __ldg(row + 8);
          }
        }
      }
      const float2* cs = p.rope + (int64_t)turn[at] * (kD / 2) + 4 * c;
      float s[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) s[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t[8];
        load_turn(cs + 32 * i, t);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float xa = lo_f(w[e]), xb = hi_f(w[e]);
          const float ku = fmaf(xa, t[2 * e], -(xb * t[2 * e + 1])), kw = fmaf(xa, t[2 * e + 1], xb * t[2 * e]);
#pragma unroll
          for (int r = 0; r < NR; ++r) s[r] = fmaf(q[r][8 * i + 2 * e + 1], kw, fmaf(q[r][8 * i + 2 * e], ku, s[r]));
        }
      }
      const int at_pos = spos[at];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], 4);
        s[r] = at_pos <= limit[r] ? s[r] : -INFINITY;
        if (!VALUES && !a.tail && c == 0 && r < a.rows)
          p.scores[((int64_t)(a.h - p.h0) * p.R + r) * p.Nkp + k0 + at] = s[r];
        if (s[r] > m[r] + 8.0f) {                  // the reference rises: rarely
          const float f = ex2(m[r] - s[r]);
          m[r] = s[r];
          l[r] *= f;
          if (VALUES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[r][e] = __fmul2_rn(o[r][e], make_float2(f, f));
          }
        }
        const float w = ex2(s[r] - m[r]);
        l[r] += w;
        if (VALUES) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[r][4 * i + e] = __ffma2_rn(make_float2(w, w), make_float2(lo_f(v[e]), hi_f(v[e])), o[r][4 * i + e]);
          }
        }
      }
    }
  }
  // the four groups of a warp joined, then the four warps
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], d), l2 = __shfl_xor_sync(0xffffffffu, l[r], d), M = fmaxf(m[r], m2);
      const float f = ex2(m[r] - M), g = ex2(m2 - M);
      l[r] = l[r] * f + l2 * g;
      m[r] = M;
      if (VALUES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __shfl_xor_sync(0xffffffffu, o[r][e].x, d), y = __shfl_xor_sync(0xffffffffu, o[r][e].y, d);
          o[r][e] = make_float2(o[r][e].x * f + x * g, o[r][e].y * f + y * g);
        }
      }
    }
    float* j = joined + (warp * NR + r) * (kD + 4);
    if (VALUES && group == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(j + 64 * i + 8 * c + 2 * e) = o[r][4 * i + e];
    }
    if (lane == 0) { j[kD] = m[r]; j[kD + 1] = l[r]; }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (r >= a.rows) break;
    float M = kNoMax, L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, joined[(w * NR + r) * (kD + 4) + kD]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float* j = joined + (w * NR + r) * (kD + 4);
      const float f = ex2(j[kD] - M);
      L += f * j[kD + 1];
      if (VALUES) O += f * j[threadIdx.x];
    }
    if (VALUES && p.slots == 1) {                  // nothing to join: O itself
      p.O[query_row(p, a.h, a.r0 + r) * kD + threadIdx.x] = __float2bfloat16_rn(L == 0.0f ? 0.0f : O / L);
      continue;
    }
    const int64_t out = ((int64_t)a.slot * p.Hn + a.h - p.h0) * p.R + a.r0 + r;
    if (threadIdx.x == 0) p.part_ml[out] = make_float2(M, L);
    if (VALUES) p.part_O[out * kD + threadIdx.x] = O;
  }
}

size_t sg_smem(int T, int G, int nr, bool values) {
  const size_t block = kSgKeys * (32 + sizeof(uint32_t) * (T >= 0 && T <= 4 ? (T > 0 ? T : 1) : kMaxT) + kD / G * sizeof(float2));
  return 16 * sizeof(float2) + 4 * nr * (kD + 4) * sizeof(float) + 4 * 2 * kSgKeys * sizeof(int) + (values ? 8 : 4) * block;
}

template <int TT, int NR, bool VALUES>
cudaError_t launch_single_t(const BatchParams& p, cudaStream_t s) {
  const size_t smem = sg_smem(p.T, p.G, NR, VALUES);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_attention_single<TT, NR, VALUES>), smem);
  if (e != cudaSuccess) return e;
  qvg_attention_single<TT, NR, VALUES><<<(unsigned)(p.S1 * p.Hn + p.S2 * p.Hn * p.B), kSgThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <int NR, bool VALUES>
cudaError_t launch_single_r(const BatchParams& p, cudaStream_t s) {
  switch (p.T) {
    case 0: return launch_single_t<0, NR, VALUES>(p, s);
    case 1: return launch_single_t<1, NR, VALUES>(p, s);
    case 2: return launch_single_t<2, NR, VALUES>(p, s);
    case 3: return launch_single_t<3, NR, VALUES>(p, s);
    case 4: return launch_single_t<4, NR, VALUES>(p, s);
    default: return launch_single_t<-1, NR, VALUES>(p, s);
  }
}

}  // namespace

int single_per_sm(const BatchParams& p, bool values) {
  const size_t smem = sg_smem(p.T, p.G, p.R > 1 ? 2 : 1, values) + 1024;
  return std::min((int)(size_t(228 * 1024) / smem), p.R > 1 ? 4 : kSgPerSm);
}

cudaError_t launch_single_partial(const BatchParams& p, bool values, cudaStream_t s) {
  if (values) return launch_single_r<1, true>(p, s);
  return p.R > 1 ? launch_single_r<2, false>(p, s) : launch_single_r<1, false>(p, s);
}

}  // namespace qvg
