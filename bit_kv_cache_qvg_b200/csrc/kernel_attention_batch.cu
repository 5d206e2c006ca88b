// kernel_attention_batch.cu -- qvg_attention_batch for many rows: the
// warp-specialised tcgen05 attention of qvg_attention_fused over the rows of a
// whole batch.
//
// A unit is a block of 256 rows of one K/V head (two row tiles of 128) and a
// range of the keys: of the prefix, which the rows of every sequence and query
// head share, or of one sequence's tail, with that sequence's rows.  All
// units are one launch; each leaves its unnormalised O with the rows' maxima
// and sums in the workspace, and qvg_batch_merge joins the ranges.  With few
// long sequences a prefix tile is reconstructed once for every 512 rows, a pair
// of CTAs sharing it through distributed shared memory.
//
// The roles, the ring of operands and the online softmax are those of
// qvg_attention_fused (kernel_attention.cu).  What differs: rows are found
// through the batch's layout, a cached token may have a position of its own,
// tail tiles are copied from bf16 rows instead of reconstructed, and tiles that
// some row must not see entirely (the ragged end, a causal border) take a
// masked path; the others have no masks to evaluate.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attention_tc.cuh"
#include "batch.cuh"

namespace qvg {
namespace {

constexpr int kBtRows = kAtQTiles * kAtTile;      // rows per CTA
constexpr int kBtMaxRanges = 16;                  // of the prefix
constexpr int kBtMaxDevices = 64;

struct BtShared {
  AtBars bars;
  float2 nlut[16];                // nibble -> two codes (q, or u - 2)
  int min_limit[2];               // least limit of a row tile's live rows
  int kpos[2][kAtTile];           // key positions of a masked tile, per row tile
};

struct BtPlace {
  bool tail;
  int h, b, slot;
  int n;                          // keys of the prefix or tail (below 2^23)
  int j0, ntiles;                 // tiles of 128 keys
  int r0, r1;                     // rows (below 2^23)
};

// Cluster ids: the prefix's (range fastest, then row blocks, then head), then
// the tails' (the same, then sequence).
__device__ __forceinline__ BtPlace bt_place(const BatchParams& p, int pair, unsigned id, int pr) {
  BtPlace a;
  const int64_t n1 = (p.tiles1 + pair - 1) / pair, n2 = (p.tiles2 + pair - 1) / pair;
  const int64_t first_tail = (int64_t)p.S1 * n1 * p.H;
  a.tail = id >= first_tail;
  const int64_t e = a.tail ? id - first_tail : id;
  const int S = a.tail ? p.S2 : p.S1;
  const int64_t nb = a.tail ? n2 : n1;
  const int range = (int)(e % S);
  const int64_t block = e / S % nb, unit = e / S / nb;
  a.h = (int)(unit % p.H);
  a.b = (int)(unit / p.H);
  a.n = (int)(a.tail ? tail_length(p, a.b) : p.Nk);
  a.slot = a.tail ? p.S1 + range : range;
  a.r0 = (int)((a.tail ? a.b * p.RB : 0) + (block * pair + pr) * kBtRows);
  a.r1 = (int)(a.tail ? (a.b + 1) * p.RB : p.R);
  const int64_t nt = (a.n + kAtTile - 1) / kAtTile;
  a.j0 = (int)(nt * range / S);
  a.ntiles = (int)(nt * (range + 1) / S) - a.j0;
  return a;
}

// Position of key `key` of the unit for the masks.
__device__ __forceinline__ int bt_key_pos(const BatchParams& p, const BtPlace& a, int key) {
  if (key >= a.n) return kPosNever;
  if (a.tail) return clamp_pos(p.tail_pos != nullptr ? __ldg(p.tail_pos + (int64_t)a.b * p.Nt + key) : p.Nk + key);
  return clamp_pos(p.k_pos != nullptr ? __ldg(p.k_pos + (int64_t)a.h * p.Nk + key) : key);
}
// Row of the rotary table for key `key` (past the end: the last key's).
__device__ __forceinline__ int bt_rope_row(const BatchParams& p, const BtPlace& a, int key) {
  key = key < a.n ? key : a.n - 1;
  int64_t pos = key;
  if (a.tail) pos = p.tail_pos != nullptr ? __ldg(p.tail_pos + (int64_t)a.b * p.Nt + key) : p.Nk + key;
  else if (p.k_pos != nullptr) pos = __ldg(p.k_pos + (int64_t)a.h * p.Nk + key);
  return (int)rope_row(p, pos);
}

template <int TT>
__global__ void __launch_bounds__(kAtThreads, 1) qvg_attention_batch_tc(const BatchParams p, const int pair, uint32_t* status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                               // A of S: two row tiles x channels
  uint8_t* sK0 = sQ + kAtQTiles * kAtOpBytes;       // ring stage s: K at sK0 + 2s tiles, V after it
  BtShared* sh = reinterpret_cast<BtShared*>(sK0 + 4 * kAtOpBytes);
  AtBars* bars = &sh->bars;
  const float2* nlut = sh->nlut;
  volatile int* abort_flag = &bars->abort_flag;
  auto stage_k = [&](int st) { return sK0 + (2 * st) * kAtOpBytes; };
  auto stage_v = [&](int st) { return sK0 + (2 * st + 1) * kAtOpBytes; };

  const int pr = (int)(blockIdx.x % (unsigned)pair);            // rank in the cluster
  const BtPlace a = bt_place(p, pair, blockIdx.x / (unsigned)pair, pr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = a.h, ntiles = a.ntiles, j_begin = a.j0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&bars->s_done[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&bars->o_done[i])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&bars->kv_full[i])),
                   "r"(kAtReconThreads / 32 * pair));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&bars->kv_empty[i])), "r"(2 * pair));
    }
    bars->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&bars->tmem_base)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x < 16) {
    const float off = p.sym ? 2.0f : 0.0f;
    sh->nlut[threadIdx.x] = make_float2((float)(threadIdx.x & 3u) - off, (float)(threadIdx.x >> 2) - off);
  }
  if (threadIdx.x < 2) sh->min_limit[threadIdx.x] = kPosNever;
  __syncthreads();
  // rows: rotary embedding at their positions, bf16, into the A layout (512
  // threads: rows 4*rb .. 4*rb+3 of each tile, channels 8*cb ..)
  if (threadIdx.x < 512) {
    const int rb = threadIdx.x >> 4, cb = threadIdx.x & 15;
    for (int qt = 0; qt < kAtQTiles; ++qt) {
      for (int r = 0; r < 4; ++r) {
        const int qi = 4 * rb + r;
        const int row = a.r0 + qt * kAtTile + qi;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (row < a.r1) {
          const uint4 v = *reinterpret_cast<const uint4*>(p.Q + query_row(p, h, row) * kD + 8 * cb);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
          const int64_t pos = query_pos(p, row);
          if (cb == 0 && pos >= 0) atomicMin(&sh->min_limit[qt], row_limit(p, pos));
          const float2* turn = p.rope + rope_row(p, pos) * (kD / 2) + 4 * cb;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float xa = lo_f(x[e]), xb = hi_f(x[e]);
            const float2 cs = __ldg(turn + e);
            w[e] = pack2(xa * cs.x - xb * cs.y, xa * cs.y + xb * cs.x);
          }
        }
        *reinterpret_cast<uint4*>(sQ + qt * kAtOpBytes + op_off(qi, 8 * cb)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  if (pair > 1) cluster_sync();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t tS = tmem, tO = tmem + 256;        // S of row tile t at column 128 t, O at 256 + 128 t
  int s_issued = 0, o_issued = 0;

  if (warp >= 8) {
    // ---------------------------------------------------------------- reconstruction warps (see qvg_attention_fused)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    const int r = threadIdx.x - kAtSoftmaxThreads;
    const int rb = r >> 4, cb = r & 15;             // K: two rows from 2*rb (4*rb alone), channels 8*cb ..
    const int rbv = r & 31, cbv = r >> 5;           // V: the same blocks, transposed
    const bool paired = pair > 1;
    const uint32_t own_base = smem_addr(smem);
    const uint32_t peer_base = paired ? cluster_addr(own_base, (uint32_t)(pr ^ 1)) : 0u;
    constexpr bool kAhead = TT >= 0 && TT <= 2;
    const int nh = 2 / pair;
    const int nsteps = ntiles * nh;
    auto row_k = [&](int half) { return paired ? 64 * pr + 2 * rb : 4 * rb + 2 * half; };
    auto row_v = [&](int half) { return paired ? 64 * pr + 2 * rbv : 4 * rbv + 2 * half; };
    auto tile_of = [&](int s) { return nh == 1 ? s : s >> 1; };
    // stage st is free again once the O products of tile j - 2 have completed
    auto wait_empty = [&](int j) {
      const bool w = j < 2 || bar_wait_cluster(&bars->kv_empty[j & 1], (uint32_t)(((j >> 1) - 1) & 1), abort_flag);
      if (__any_sync(0xffffffffu, !w || *abort_flag)) {
        *abort_flag = 1;
        return false;
      }
      fence_after();
      return true;
    };
    auto put_k = [&](int st, int row, uint4 v) {
      uint8_t* dst = stage_k(st) + op_off(row, 8 * cb);
      *reinterpret_cast<uint4*>(dst) = v;
      if (paired) st_cluster_v4(peer_base + (smem_addr(dst) - own_base), v);
    };
    auto put_v = [&](int st, int ch, int row, uint32_t v2) {
      uint8_t* dst = stage_v(st) + op_off(ch, row);
      *reinterpret_cast<uint32_t*>(dst) = v2;
      if (paired) st_cluster_b32(peer_base + (smem_addr(dst) - own_base), v2);
    };
    auto turned = [&](float xa, float xb, float c, float s) {
      return pack2(__fsub_rn(__fmul_rn(xa, c), __fmul_rn(xb, s)), __fadd_rn(__fmul_rn(xa, s), __fmul_rn(xb, c)));
    };
    auto arrive_full = [&](int st) {
      if (paired) asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
      else asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->kv_full[st]);
        if (paired) mbar_arrive_remote(cluster_addr(smem_addr(&bars->kv_full[st]), (uint32_t)(pr ^ 1)));
      }
    };
    if (!a.tail) {
      ReconBlock<TT, 2, BatchParams> bk, bv;
      int at[2] = {0, 0};                           // rows of the rotary table
      auto positions = [&](int tok0, int (&to)[2]) {
        to[0] = bt_rope_row(p, a, tok0);
        to[1] = bt_rope_row(p, a, tok0 + 1);
      };
      if (kAhead && nsteps > 0) {
        bk.load_tokens(p, 0, h, j_begin * kAtTile + row_k(0), 8 * cb);
        bv.load_tokens(p, 1, h, j_begin * kAtTile + row_v(0), 8 * cbv);
        positions(bk.tok0, at);
      }
#pragma unroll 1
      for (int s = 0; s < nsteps; ++s) {
        const int j = tile_of(s), half = s - j * nh, st = j & 1;
        if (half == 0 && !wait_empty(j)) break;
        float vk[2][8];
        const int r0 = row_k(half), rv = row_v(half);
        if (!kAhead) {
          bk.load_tokens(p, 0, h, (j_begin + j) * kAtTile + r0, 8 * cb);
          bv.load_tokens(p, 1, h, (j_begin + j) * kAtTile + rv, 8 * cbv);
          positions(bk.tok0, at);
        }
        bk.load_rows(p, h);
        bv.load_rows(p, h);
        ReconBlock<TT, 2, BatchParams> nk, nv;
        int nat[2] = {0, 0};
        if (kAhead && s + 1 < nsteps) {
          const int j1 = tile_of(s + 1), half1 = s + 1 - j1 * nh;
          nk.load_tokens(p, 0, h, (j_begin + j1) * kAtTile + row_k(half1), 8 * cb);
          nv.load_tokens(p, 1, h, (j_begin + j1) * kAtTile + row_v(half1), 8 * cbv);
          positions(nk.tok0, nat);
        }
        bk.finish(p, nlut, h, vk);
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const float4* cs4 = reinterpret_cast<const float4*>(p.rope + (int64_t)at[rr] * (kD / 2) + 4 * cb);
          const float4 t0 = __ldg(cs4), t1 = __ldg(cs4 + 1);
          put_k(st, r0 + rr, make_uint4(turned(vk[rr][0], vk[rr][1], t0.x, t0.y), turned(vk[rr][2], vk[rr][3], t0.z, t0.w),
                                        turned(vk[rr][4], vk[rr][5], t1.x, t1.y), turned(vk[rr][6], vk[rr][7], t1.z, t1.w)));
        }
        bv.finish(p, nlut, h, vk);
#pragma unroll
        for (int e = 0; e < 8; ++e) put_v(st, 8 * cbv + e, rv, pack2(vk[0][e], vk[1][e]));
        if (kAhead) {
          bk.take_tokens(nk);
          bv.take_tokens(nv);
          at[0] = nat[0];
          at[1] = nat[1];
        }
        if (half == nh - 1) arrive_full(st);
      }
    } else {
      // a tail's tokens are bf16 rows already; behind its length zeros
      const int64_t base = ((int64_t)a.b * p.H + h) * p.Nt;
#pragma unroll 1
      for (int s = 0; s < nsteps; ++s) {
        const int j = tile_of(s), half = s - j * nh, st = j & 1;
        if (half == 0 && !wait_empty(j)) break;
        const int r0 = row_k(half), rv = row_v(half);
        const int tk = (j_begin + j) * kAtTile + r0, tv = (j_begin + j) * kAtTile + rv;
        uint4 xk[2], xv[2];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          xk[rr] = xv[rr] = make_uint4(0, 0, 0, 0);
          if (tk + rr < a.n) xk[rr] = __ldg(reinterpret_cast<const uint4*>(p.tail[0] + (base + tk + rr) * kD + 8 * cb));
          if (tv + rr < a.n) xv[rr] = __ldg(reinterpret_cast<const uint4*>(p.tail[1] + (base + tv + rr) * kD + 8 * cbv));
        }
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const float4* cs4 = reinterpret_cast<const float4*>(p.rope + (int64_t)bt_rope_row(p, a, tk + rr) * (kD / 2) + 4 * cb);
          const float4 t0 = __ldg(cs4), t1 = __ldg(cs4 + 1);
          const uint4 x = xk[rr];
          put_k(st, r0 + rr, make_uint4(turned(lo_f(x.x), hi_f(x.x), t0.x, t0.y), turned(lo_f(x.y), hi_f(x.y), t0.z, t0.w),
                                        turned(lo_f(x.z), hi_f(x.z), t1.x, t1.y), turned(lo_f(x.w), hi_f(x.w), t1.z, t1.w)));
        }
        const uint32_t x0[4] = {xv[0].x, xv[0].y, xv[0].z, xv[0].w}, x1[4] = {xv[1].x, xv[1].y, xv[1].z, xv[1].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          put_v(st, 8 * cbv + 2 * e, rv, __byte_perm(x0[e], x1[e], 0x5410));
          put_v(st, 8 * cbv + 2 * e + 1, rv, __byte_perm(x0[e], x1[e], 0x7632));
        }
        if (half == nh - 1) arrive_full(st);
      }
    }
    // Paired, the other CTA's commits arrive here too: the last use of each
    // stage must have completed before this CTA may leave (bounded; skipped
    // once a role has aborted).
    if (paired && r == 0 && !*abort_flag)
      for (int j = ntiles - 2 > 0 ? ntiles - 2 : 0; j < ntiles; ++j)
        if (!bar_wait_cluster(&bars->kv_empty[j & 1], (uint32_t)((j >> 1) & 1), abort_flag)) *abort_flag = 1;
  } else {
    // ---------------------------------------------------------------- softmax warps, two independent groups
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    const int g = warp >> 2;
    const bool issuer = threadIdx.x == 128 * g;
    const int qi = 32 * (warp & 3) + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tSt = tS + 128 * g, tOt = tO + 128 * g;
    const int limit = a.r0 + g * kAtTile + qi < a.r1 ? row_limit(p, query_pos(p, a.r0 + g * kAtTile + qi)) : kLimitNone;
    const volatile int& least = sh->min_limit[g];   // of the tile's live rows; kPosNever when there are none
    const bool in_order = !a.tail && p.k_pos == nullptr;
    int* kpos = sh->kpos[g];
    float m_run = kNoMax, l_run = 0.0f;
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      const int st = j & 1;
      const int k0 = (j_begin + j) * kAtTile;
      // 1. S_g once the stage is full and the previous O_g has completed
      if (issuer) {
        bool w = bar_wait_cluster(&bars->kv_full[st], (uint32_t)((j >> 1) & 1), abort_flag);
        if (w && j > 0) w = bar_wait_or_abort(&bars->o_done[g], (uint32_t)((j - 1) & 1), abort_flag);
        if (w) {
          fence_after();
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          const uint32_t a0 = smem_addr(sQ + g * kAtOpBytes), b0 = smem_addr(stage_k(st));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma(tSt, op_desc_k(a0, kk), op_desc_k(b0, kk), kk > 0 ? 1u : 0u);
          mma_commit(&bars->s_done[g]);
          ++s_issued;
        } else {
          *abort_flag = 1;
        }
      }
      // Meanwhile: does any live row miss a key of this tile?  Where positions
      // are in order the last one tells; otherwise every thread looks at a key.
      const int valid = min(a.n - k0, kAtTile);
      bool masked = valid < kAtTile;
      if (p.causal) {
        if (in_order) {
          masked |= k0 + valid - 1 > least;
          if (masked) kpos[qi] = bt_key_pos(p, a, k0 + qi);
        } else {
          const int kp = bt_key_pos(p, a, k0 + qi);
          kpos[qi] = kp;
          masked = named_bar_or(1 + g, 128, kp > least);
        }
      } else if (masked) {
        kpos[qi] = qi < valid ? 0 : kPosNever;
      }
      // 2. the scores (the previous O_g is complete too: the issuer waited for it)
      bool w_ok = bar_wait_or_abort(&bars->s_done[g], (uint32_t)(j & 1), abort_flag);
      if (named_bar_or(1 + g, 128, !w_ok)) { ok = false; break; }
      fence_after();
      // 3. online softmax of the thread's row; P_g into tensor memory
      {
        float mt = kNoMax;
        auto pass1 = [&](auto full) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t rg[16];
            tld16(tSt + lane_base + (uint32_t)(16 * c), rg);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (decltype(full)::value || kpos[16 * c + e] <= limit) mt = fmaxf(mt, __uint_as_float(rg[e]));
          }
        };
        if (!masked) pass1(std::true_type{}); else pass1(std::false_type{});
        // the reference maximum rises only when the row's exceeds it by more than 8
        const float m_row = mt > kNoMax ? fmaxf(m_run, mt * p.sl) : m_run;
        const float m_new = m_row > m_run + 8.0f ? m_row : m_run;
        const float alpha = exp2_approx(m_run - m_new);
        const float2 sl2 = make_float2(p.sl, p.sl), nm2 = make_float2(-m_new, -m_new);
        float2 sum2 = make_float2(0.0f, 0.0f);
        auto pass2 = [&](auto full) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t rg[16];
            tld16(tSt + lane_base + (uint32_t)(16 * c), rg);
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(rg[2 * e]), __uint_as_float(rg[2 * e + 1])), sl2, nm2);
              float pa = exp2_approx(x.x), pb = exp2_approx(x.y);
              if (!decltype(full)::value) {
                if (kpos[16 * c + 2 * e] > limit) pa = 0.0f;
                if (kpos[16 * c + 2 * e + 1] > limit) pb = 0.0f;
              }
              w[e] = pack_bf16(pa, pb);
              sum2 = __fadd2_rn(sum2, make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)));
            }
            tst8(tSt + lane_base + (uint32_t)(8 * c), w);
          }
        };
        if (!masked) pass2(std::true_type{}); else pass2(std::false_type{});
        l_run = l_run * alpha + (sum2.x + sum2.y);
        m_run = m_new;
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {   // rescale O_g
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t rg[16];
            tld16(tOt + lane_base + (uint32_t)(16 * c), rg);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(rg[e]), __uint_as_float(rg[e + 1])),
                                          make_float2(alpha, alpha));
              rg[e] = __float_as_uint(v.x);
              rg[e + 1] = __float_as_uint(v.y);
            }
            tst16(tOt + lane_base + (uint32_t)(16 * c), rg);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      fence_before();
      named_bar_or(1 + g, 128, false);                 // P_g written, O_g rescaled, kpos read
      // 4. O_g += P_g V; the stage is free once both row tiles' products complete
      if (issuer) {
        fence_after();
        const uint32_t b0 = smem_addr(stage_v(st));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ta(tOt, tSt + (uint32_t)(8 * kk), op_desc_k(b0, kk), (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&bars->o_done[g]);
        if (pair > 1) mma_commit_mc(&bars->kv_empty[st], (uint16_t)3);
        else mma_commit(&bars->kv_empty[st]);
        ++o_issued;
      }
    }
    // the last product, then the unnormalised O with the row's maximum and sum
    if (ok && ntiles > 0) {
      const bool w_ok = bar_wait_or_abort(&bars->o_done[g], (uint32_t)((ntiles - 1) & 1), abort_flag);
      ok = !named_bar_or(1 + g, 128, !w_ok);
      fence_after();
    }
    if (!ok) *abort_flag = 1;
    if (ok) {
      const int row = a.r0 + g * kAtTile + qi;
      const int64_t out = ((int64_t)a.slot * p.H + h) * p.R + row;
      if (limit == kLimitNone) l_run = 0.0f;           // a padding row: the merge skips the range
      if (row < a.r1) p.part_ml[out] = make_float2(m_run, l_run);
      if (ntiles > 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t rg[32];
          tld32(tOt + lane_base + (uint32_t)(32 * c), rg);
          if (row < a.r1) {
            float4* dst = reinterpret_cast<float4*>(p.part_O + out * kD + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(rg[4 * e]), __uint_as_float(rg[4 * e + 1]),
                                   __uint_as_float(rg[4 * e + 2]), __uint_as_float(rg[4 * e + 3]));
          }
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (*abort_flag && (threadIdx.x == 0 || threadIdx.x == 128)) {
    const int g = threadIdx.x >> 7;
    if (g == 0) atomicOr(status, 1u);
    // let the products this thread issued finish (bounded) before the tensor memory is freed
    if (s_issued > 0) bar_wait(&bars->s_done[g], (uint32_t)((s_issued - 1) & 1));
    if (o_issued > 0) bar_wait(&bars->o_done[g], (uint32_t)((o_issued - 1) & 1));
  }
  __syncthreads();
  // no CTA leaves while the other still writes its shared memory
  if (pair > 1) cluster_sync();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

size_t bt_smem_bytes() { return 1024 + (size_t)(kAtQTiles + 4) * kAtOpBytes + sizeof(BtShared); }

const void* bt_kernel(int T) {
  switch (T) {
    case 0: return reinterpret_cast<const void*>(qvg_attention_batch_tc<0>);
    case 1: return reinterpret_cast<const void*>(qvg_attention_batch_tc<1>);
    case 2: return reinterpret_cast<const void*>(qvg_attention_batch_tc<2>);
    case 3: return reinterpret_cast<const void*>(qvg_attention_batch_tc<3>);
    case 4: return reinterpret_cast<const void*>(qvg_attention_batch_tc<4>);
    default: return reinterpret_cast<const void*>(qvg_attention_batch_tc<-1>);
  }
}

cudaLaunchConfig_t bt_config(int pair, unsigned clusters, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clusters * (unsigned)pair);
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = bt_smem_bytes();
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)pair;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of `pair` CTAs on the device at once (cached per device, stages and pair).
int bt_resident(int T, int pair) {
  static std::atomic<int> cache[kBtMaxDevices][7][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kBtMaxDevices) return 0;
  std::atomic<int>& known = cache[dev][T >= 0 && T <= 4 ? T : 5][pair];
  if (const int n = known.load(std::memory_order_relaxed)) return n;
  if (ensure_dynamic_smem(bt_kernel(T), bt_smem_bytes()) != cudaSuccess) return 0;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = bt_config(pair, 1, nullptr, attr);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, bt_kernel(T), &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  known.store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

// The cut: ranges of the prefix (and of the tails, of about the same length)
// such that the clusters of all units finish together.  The cost of a plan is
// the time of its waves, in tiles: a unit of t tiles takes t + 2, the tails'
// units fill the gaps of the prefix's last wave first, and every range's
// partial results cost their way through memory (about 0.4 of a tile per wave).
int plan_batch_tc(BatchParams& p) {
  p.tiles1 = (p.R + kBtRows - 1) / kBtRows;
  p.tiles2 = (p.RB + kBtRows - 1) / kBtRows;
  const int pair = p.tiles1 >= 2 ? 2 : 1;
  const int64_t nt1 = (p.Nk + kAtTile - 1) / kAtTile, nt2 = (p.Nt + kAtTile - 1) / kAtTile;
  const int64_t u1 = (p.tiles1 + pair - 1) / pair * p.H, u2 = p.Nt > 0 ? (p.tiles2 + pair - 1) / pair * p.H * p.B : 0;
  const double n = std::max(1, bt_resident(p.T, pair));
  double best = -1.0;
  for (int64_t s1 = 1; s1 <= std::min<int64_t>(nt1, kBtMaxRanges); ++s1) {
    const double t1 = (double)((nt1 + s1 - 1) / s1);
    const int64_t s2 = u2 > 0 ? std::max<int64_t>(1, std::min<int64_t>(nt2, (int64_t)((double)nt2 / t1 + 0.5))) : 0;
    const double t2 = s2 > 0 ? (double)((nt2 + s2 - 1) / s2) + 2.0 : 0.0;
    const double waves = (double)((u1 * s1 + (int64_t)n - 1) / (int64_t)n);
    double cost = waves * (t1 + 2.0);
    const double gaps = (waves * n - (double)(u1 * s1)) * (t1 + 2.0), rest = (double)(u2 * s2) * t2 - 0.8 * gaps;
    if (rest > 0.0) cost += std::max(t2, rest / n + 0.5 * t2);
    cost += 0.4 * (double)(s1 + s2) * (double)u1 / n;
    if (best < 0.0 || cost < best) { best = cost; p.S1 = (int)s1; p.S2 = (int)s2; }
  }
  return pair;
}

cudaError_t launch_batch_tc(const BatchParams& p, int pair, void* tables, cudaStream_t s) {
  const void* k = bt_kernel(p.T);
  cudaError_t e = ensure_dynamic_smem(k, bt_smem_bytes());
  if (e != cudaSuccess) return e;
  const int64_t clusters = (int64_t)p.S1 * ((p.tiles1 + pair - 1) / pair) * p.H +
                           (int64_t)p.S2 * ((p.tiles2 + pair - 1) / pair) * p.H * p.B;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = bt_config(pair, (unsigned)clusters, s, attr);
  uint32_t* status = static_cast<uint32_t*>(tables);
  void* args[] = {const_cast<BatchParams*>(&p), &pair, &status};
  return cudaLaunchKernelExC(&cfg, k, args);
}

}  // namespace qvg
