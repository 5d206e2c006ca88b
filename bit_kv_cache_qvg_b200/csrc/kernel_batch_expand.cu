// kernel_batch_expand.cu -- the tensor-core operands of qvg_attention_batch and
// qvg_attention_weights for many rows, written once for all of them.
//
// The attention kernels read a key tile once for every 256 rows.  With more
// rows than that, rebuilding it each time costs more than the products: the
// rebuilding kernel of qvg_attention, over the rows of a batch, took 2.58 ms
// for 1,520 rows over 38,000 tokens of 32 heads.  So a tile is rebuilt once,
// into the workspace, as the 32 KB image that a bulk copy brings into shared
// memory as it is: bf16, K-major, 128-byte swizzle (attention_tc.cuh), keys by
// channels for K and channels by keys for V.  The rows are rotated once, too.
//
// One CTA builds one tile (128 keys of K and V, or the high and low halves of
// K) in shared memory and stores it with bulk copies; bound by the 512 bytes
// written a token.
#include "attention_tc.cuh"
#include "batch.cuh"

namespace qvg {
namespace {

constexpr int kExThreads = 256;

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// u + iw = (a + ib) e^(i phi): high halves, and (precise) what their rounding left
__device__ __forceinline__ void turn_pair(uint32_t x, float c, float s, bool precise, uint32_t& hi, uint32_t& lo) {
  const float a = lo_f(x), b = hi_f(x);
  const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), w = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  hi = pack2(u, w);
  lo = precise ? pack2(u - lo_f(hi), w - hi_f(hi)) : 0u;
}
__device__ __forceinline__ void turn_chunk(const BatchParams& p, uint4 x, int64_t pos, int c0, bool precise, uint4& hi, uint4& lo) {
  const float4* cs4 = reinterpret_cast<const float4*>(p.rope + rope_row(p, pos) * (kD / 2) + c0 / 2);
  const float4 t0 = __ldg(cs4), t1 = __ldg(cs4 + 1);
  turn_pair(x.x, t0.x, t0.y, precise, hi.x, lo.x);
  turn_pair(x.y, t0.z, t0.w, precise, hi.y, lo.y);
  turn_pair(x.z, t1.x, t1.y, precise, hi.z, lo.z);
  turn_pair(x.w, t1.z, t1.w, precise, hi.w, lo.w);
}
__device__ __forceinline__ uint4 pack_row(const float (&y)[8]) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// 128 rows of a head (r0 in the head's rows) or of one sequence, rotated at
// their positions; zeros behind the last one.
__device__ __forceinline__ void expand_rows(const BatchParams& p, bool by_sequence, int hl, int b, int64_t tile, bool precise) {
  const int which = by_sequence ? 1 : 0;
  const int64_t rows = by_sequence ? p.RB : p.R, pad = by_sequence ? p.RBp : p.Rp;
  const int64_t base = ((by_sequence ? (int64_t)b * p.Hn : 0) + hl) * 2 * pad;
  for (int e = threadIdx.x; e < 128 * 16; e += kExThreads) {
    const int cb = e & 15;
    const int64_t r = tile * 128 + (e >> 4);
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (r < rows) {
      const int64_t row = by_sequence ? b * p.RB + r : r;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.Q + query_row(p, p.h0 + hl, row) * kD + 8 * cb));
      turn_chunk(p, x, query_pos(p, row), 8 * cb, precise, hi, lo);
    }
    const int64_t at = (base + (cb >> 3) * pad + r) * 128 + (((cb & 7) ^ (int)(r & 7)) << 4);
    *reinterpret_cast<uint4*>(p.row_img[which] + at) = hi;
    if (precise) *reinterpret_cast<uint4*>(p.row_lo[which] + at) = lo;
  }
}

// CTAs: the prefix's key tiles, the tails', the rows by head, the rows by
// sequence.  PRECISE: the second image of a tile holds the keys' low halves
// instead of the values.
template <int TT, bool PRECISE>
__global__ void __launch_bounds__(kExThreads, 3) qvg_batch_expand(const BatchParams p, const int64_t tiles_p, const int64_t tiles_t,
                                                                 const int64_t row_tiles) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sK = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sV = sK + kImageBytes;
  __shared__ float2 nlut[16];
  int64_t id = blockIdx.x;
  if (id >= tiles_p + tiles_t) {
    id -= tiles_p + tiles_t;
    const bool by_sequence = id >= row_tiles;
    if (by_sequence) id -= row_tiles;
    const int64_t per = (by_sequence ? p.RBp : p.Rp) / 128;
    const int64_t unit = id / per;
    expand_rows(p, by_sequence, (int)(unit % p.Hn), (int)(unit / p.Hn), id % per, PRECISE);
    return;
  }
  const bool tail = id >= tiles_p;
  if (tail) id -= tiles_p;
  const int64_t nt = tail ? p.nt2 : p.nt1, unit = id / nt;
  const int j = (int)(id % nt), hl = (int)(unit % p.Hn), b = (int)(unit / p.Hn), h = p.h0 + hl;
  const int64_t n = tail ? tail_length(p, b) : p.Nk;
  const int tile0 = j * kAtTile;
  if (tile0 >= n) return;                          // a tail's tile that nobody reads
  if (threadIdx.x < 16) {
    const float off = p.sym ? 2.0f : 0.0f;
    nlut[threadIdx.x] = make_float2((float)(threadIdx.x & 3u) - off, (float)(threadIdx.x >> 2) - off);
  }
  __syncthreads();
  const int r = threadIdx.x;
  const int rb = r >> 4, cb = r & 15;              // K: rows 32 s + 2 rb, + 1, channels 8 cb ..
  const int rbv = r & 31, cbv = r >> 5;            // V: keys 64 (s & 1) + 2 rbv, + 1, channels 8 (cbv + 8 (s >> 1)) ..
  auto put_k = [&](int row, uint4 x, int64_t pos) {
    uint4 hi, lo;
    turn_chunk(p, x, pos, 8 * cb, PRECISE, hi, lo);
    *reinterpret_cast<uint4*>(sK + op_off(row, 8 * cb)) = hi;
    if (PRECISE) *reinterpret_cast<uint4*>(sV + op_off(row, 8 * cb)) = lo;
  };
  if (!tail) {
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      ReconBlock<TT, 2, BatchParams> bk, bv;
      const int rk = 32 * s + 2 * rb, rv = 64 * (s & 1) + 2 * rbv, cv = 8 * (cbv + 8 * (s >> 1));
      bk.load_tokens(p, 0, h, tile0 + rk, 8 * cb);
      if (!PRECISE) bv.load_tokens(p, 1, h, tile0 + rv, cv);
      bk.load_rows(p, h);
      if (!PRECISE) bv.load_rows(p, h);
      float y[2][8];
      bk.finish(p, nlut, h, y);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int64_t key = tile0 + rk + rr < n ? tile0 + rk + rr : n - 1;
        put_k(rk + rr, pack_row(y[rr]), raw_key_pos(p, false, h, 0, key));
      }
      if (!PRECISE) {
        bv.finish(p, nlut, h, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint32_t*>(sV + op_off(cv + e, rv)) = pack2(y[0][e], y[1][e]);
      }
    }
  } else {
    // a tail's tokens are bf16 rows already; behind its length zeros
    const int64_t base = ((int64_t)b * p.H + h) * p.Nt;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int rk = 32 * s + 2 * rb, rv = 64 * (s & 1) + 2 * rbv, cv = 8 * (cbv + 8 * (s >> 1));
      uint4 v[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int64_t key = tile0 + rk + rr, val = tile0 + rv + rr;
        uint4 x = make_uint4(0, 0, 0, 0);
        v[rr] = x;
        if (key < n) x = __ldg(reinterpret_cast<const uint4*>(p.tail[0] + (base + key) * kD + 8 * cb));
        put_k(rk + rr, x, key < n ? raw_key_pos(p, true, h, b, key) : 0);
        if (!PRECISE && val < n) v[rr] = __ldg(reinterpret_cast<const uint4*>(p.tail[1] + (base + val) * kD + cv));
      }
      if (!PRECISE) {
        const uint32_t x0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, x1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          *reinterpret_cast<uint32_t*>(sV + op_off(cv + 2 * e, rv)) = __byte_perm(x0[e], x1[e], 0x5410);
          *reinterpret_cast<uint32_t*>(sV + op_off(cv + 2 * e + 1, rv)) = __byte_perm(x0[e], x1[e], 0x7632);
        }
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const int64_t at = (((tail ? (int64_t)b * p.Hn : 0) + hl) * nt + j) * kImageBytes;
    bulk_store(p.key_img[tail] + at, smem_addr(sK), (uint32_t)kImageBytes);
    bulk_store(p.val_img[tail] + at, smem_addr(sV), (uint32_t)kImageBytes);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

template <int TT>
cudaError_t expand_t(const BatchParams& p, bool precise, cudaStream_t s) {
  // the launch's key tiles and rows: none of a part that another kernel handles
  const int64_t tiles_p = p.S1 > 0 ? p.Hn * p.nt1 : 0, tiles_t = p.S2 > 0 ? p.B * p.Hn * p.nt2 : 0;
  const int64_t rows_h = p.S1 > 0 ? p.Hn * (p.Rp / 128) : 0, rows_s = p.S2 > 0 ? p.B * p.Hn * (p.RBp / 128) : 0;
  const unsigned grid = (unsigned)(tiles_p + tiles_t + rows_h + rows_s);
  const size_t smem = 1024 + 2 * (size_t)kImageBytes;
  const void* k = precise ? reinterpret_cast<const void*>(qvg_batch_expand<TT, true>)
                          : reinterpret_cast<const void*>(qvg_batch_expand<TT, false>);
  const cudaError_t e = ensure_dynamic_smem(k, smem);
  if (e != cudaSuccess) return e;
  if (precise) qvg_batch_expand<TT, true><<<grid, kExThreads, smem, s>>>(p, tiles_p, tiles_t, rows_h);
  else qvg_batch_expand<TT, false><<<grid, kExThreads, smem, s>>>(p, tiles_p, tiles_t, rows_h);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_batch_expand(const BatchParams& p, bool precise, cudaStream_t s) {
  switch (p.T) {
    case 0: return expand_t<0>(p, precise, s);
    case 1: return expand_t<1>(p, precise, s);
    case 2: return expand_t<2>(p, precise, s);
    case 3: return expand_t<3>(p, precise, s);
    case 4: return expand_t<4>(p, precise, s);
    default: return expand_t<-1>(p, precise, s);
  }
}

}  // namespace qvg
