// kernel_batch_attend.cu -- qvg_attention_batch for many rows: softmax
// attention over the operand tiles that kernel_batch_expand.cu wrote, on
// tcgen05; and the plans and launches of qvg_attention_batch and
// qvg_attention_weights.
//
// One CTA = 256 rows of one K/V head (two row tiles of 128) x a range of key
// tiles, of the prefix (the rows of every sequence and query head share it)
// or of one sequence's tail.  Eighteen warps:
//   * one thread streams K and V tiles (32 KB bulk copies) through a ring of
//     five slots, K0 V0 K1 V1 ...;
//   * one thread issues the products, S_g = Q_g K'^T and O_g += P_g V for the
//     two row tiles g = 0, 1 in turn (kind::f16, M = N = K = 128, fp16 operands
//     for S and bf16 for O, fp32 accumulators in tensor memory; P read from
//     tensor memory).  P_g lies over
//     S_g's columns: the products run in the order they are issued, so S_g of
//     the next tile follows O_g of this one without a wait;
//   * eight warps per row tile run its softmax, two threads to a row with 64 of
//     its scores in registers each.  While one tile's softmax runs, the other's
//     products do.  The reference maximum rises only when a row's maximum exceeds
//     it by more than 8 (base 2), so O is rescaled rarely.
// A pair of tiles takes 2,048 cycles of products and as many of exponentials: the
// two have to run all the time, and the clock falls to about 1.5 GHz under the
// power limit.  32 heads, 1,520 rows, 38,380 keys: 838 us, 1,140 TFLOP/s (69 %
// of cuBLAS's burst rate); without the softmax it would be 600 us.
// Every wait is bounded and gives up when another role has; the kernel then
// records QVG_ERR_DEVICE_TIMEOUT in the tables' status word.
#include <algorithm>
#include <type_traits>

#include "attention_tc.cuh"
#include "batch.cuh"

namespace qvg {
namespace {

constexpr int kAdThreads = 576;                   // 16 softmax warps, the issuer's, the loader's
constexpr int kAdRows = 256;                      // rows per CTA
constexpr int kAdSlots = 5;                       // ring of operand tiles
constexpr int kAdMaxRanges = 64;                  // of the prefix, and of a tail

struct __align__(8) AdShared {
  uint64_t full[kAdSlots], empty[kAdSlots];
  uint64_t q_full;
  uint64_t s_done[2];             // S_g complete (and every product issued before it)
  uint64_t p_full[2];             // P_g written, O_g rescaled: an arrival of each of 8 warps
  uint64_t drained;               // after a failed wait: every product issued is complete
  uint32_t tmem_base;
  int abort_flag;
  float top[2][2][kAtTile];       // the maxima of a row's two halves, scaled
};

constexpr int kAdSharedBytes = 3 * 1024;
static_assert(sizeof(AdShared) <= kAdSharedBytes, "the barriers' part of shared memory");

// B operand of O += P V: V's image holds a key's 64 channels of a half in 128
// bytes, so B is N-major: 64 channels to the swizzled row, the other half
// LBO = 16 KB on, 8 keys to the 1,024-byte group (SBO).
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(kAtHalfBytes >> 4) << 16;     // LBO
  d |= (uint64_t)(1024 >> 4) << 32;             // SBO
  d |= (uint64_t)1 << 46;                       // version
  d |= (uint64_t)2 << 61;                       // SWIZZLE_128B
  return d;
}
constexpr uint32_t kIdescValues = kIdesc | (1u << 16);      // B N-major

// What a CTA has to do.
struct AdPlace {
  bool tail;
  int hl, h, b;
  uint32_t part;                  // place among the partial results: slot * Hn + hl
  int n;                          // keys of the prefix or tail (below 2^23)
  int j0, ntiles;                 // tiles of 128 keys
  int r0, r1;                     // rows of the head (below 2^23)
  int groups;                     // row tiles with rows: 1 or 2
};
__device__ __forceinline__ AdPlace ad_place(const BatchParams& p) {
  AdPlace a;
  const int64_t first_tail = (int64_t)p.S1 * p.tiles1 * p.Hn;
  a.tail = blockIdx.x >= first_tail;
  const uint32_t e = (uint32_t)(a.tail ? blockIdx.x - first_tail : blockIdx.x);
  const uint32_t S = (uint32_t)(a.tail ? p.S2 : p.S1), nb = (uint32_t)(a.tail ? p.tiles2 : p.tiles1);
  const uint32_t range = e % S, block = e / S % nb, unit = e / S / nb;
  a.hl = (int)(unit % (uint32_t)p.Hn);
  a.h = p.h0 + a.hl;
  a.b = (int)(unit / (uint32_t)p.Hn);
  a.n = (int)(a.tail ? tail_length(p, a.b) : p.Nk);
  a.part = (a.tail ? (uint32_t)p.slot2 + range : range) * (uint32_t)p.Hn + (uint32_t)a.hl;
  a.r0 = (int)((a.tail ? a.b * p.RB : 0) + block * kAdRows);
  a.r1 = (int)(a.tail ? (a.b + 1) * p.RB : p.R);
  a.groups = a.r1 - a.r0 > kAtTile ? 2 : 1;
  const uint32_t nt = (uint32_t)(a.n + kAtTile - 1) / kAtTile;       // below 2^16, S at most 64
  a.j0 = (int)(nt * range / S);
  a.ntiles = (int)(nt * (range + 1) / S) - a.j0;
  return a;
}

__global__ void __launch_bounds__(kAdThreads, 1) qvg_batch_attend(const BatchParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the barriers first, then the tiles, to the last byte there is: the start has
  // to be a 1,024-byte boundary
  AdShared* sh = reinterpret_cast<AdShared*>(smem_raw);
  uint8_t* sQ = smem_raw + kAdSharedBytes;
  uint8_t* ring = sQ + 2 * kAtOpBytes;
  if ((smem_addr(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.status, 1u);
    return;
  }
  volatile int* abort_flag = &sh->abort_flag;
  const AdPlace a = ad_place(p);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int ntiles = uniform(a.ntiles), groups = uniform(a.groups);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kAdSlots; ++i) { bar_init(&sh->full[i], 1); bar_init(&sh->empty[i], 1); }
    bar_init(&sh->q_full, 1);
    for (int g = 0; g < 2; ++g) { bar_init(&sh->s_done[g], 1); bar_init(&sh->p_full[g], 8); }
    bar_init(&sh->drained, 1);
    sh->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh->tmem_base)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(sh->tmem_base);
  const uint32_t tS = tmem, tO = tmem + 256;        // S of row tile g at column 128 g, O at 256 + 128 g

  if (warp == 17) {
    // ---------------------------------------------------------------- loader
    if (lane == 0 && ntiles > 0) {
      const int64_t pad = a.tail ? p.RBp : p.Rp, first = a.tail ? a.r0 - a.b * p.RB : a.r0;
      const uint8_t* rows = p.row_img[a.tail] + (((a.tail ? (int64_t)a.b * p.Hn : 0) + a.hl) * 2 * pad + first) * 128;
      expect_bytes(&sh->q_full, (uint32_t)(a.groups * kAtOpBytes));
      for (int g = 0; g < a.groups; ++g)
        for (int half = 0; half < 2; ++half)
          bulk_load(smem_addr(sQ) + g * kAtOpBytes + half * kAtHalfBytes, rows + (half * pad + g * kAtTile) * 128, kAtHalfBytes,
                    &sh->q_full);
      const int64_t nt = a.tail ? p.nt2 : p.nt1;
      const int64_t at = (((a.tail ? (int64_t)a.b * p.Hn : 0) + a.hl) * nt + a.j0) * kImageBytes;
      const uint8_t* src[2] = {p.key_img[a.tail] + at, p.val_img[a.tail] + at};
      int issued = 0;
      for (int i = 0; i < 2 * ntiles; ++i) {
        const int slot = i % kAdSlots, turn = i / kAdSlots;
        if (turn > 0 && !bar_wait_or_abort(&sh->empty[slot], (uint32_t)((turn - 1) & 1), abort_flag)) { *abort_flag = 1; break; }
        expect_bytes(&sh->full[slot], (uint32_t)kImageBytes);
        bulk_load(smem_addr(ring) + slot * kAtOpBytes, src[i & 1] + (int64_t)(i >> 1) * kImageBytes, (uint32_t)kImageBytes,
                  &sh->full[slot]);
        ++issued;
      }
      // no copy may be in flight when the CTA leaves
      bar_wait(&sh->q_full, 0);
      for (int i = issued > kAdSlots ? issued - kAdSlots : 0; i < issued; ++i)
        bar_wait(&sh->full[i % kAdSlots], (uint32_t)((i / kAdSlots) & 1));
    }
  } else if (warp == 16) {
    // ---------------------------------------------------------------- issuer
    // After a failed wait the loop runs on without waiting or issuing.
    if (ntiles > 0) {
      bool dead = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !bar_wait_or_abort(bar, parity, abort_flag);
        dead = __any_sync(0xffffffffu, dead);
        fence_after();
      };
      const uint64_t rows0 = op_desc(smem_addr(sQ)), keys0 = op_desc(smem_addr(ring)), vals0 = value_desc(smem_addr(ring));
      constexpr uint32_t kTile = kAtOpBytes >> 4;
      auto scores = [&](int g, uint32_t slot) {
        const uint64_t a0 = rows0 + g * kTile, b0 = keys0 + slot * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_as(tS + 128 * g, a0 + desc_step(kk), b0 + desc_step(kk), kIdescScores, kk > 0 ? 1u : 0u);
      };
      wait(&sh->q_full, 0);
      wait(&sh->full[0], 0);
      if (!dead && elect_one()) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (g < groups) {
            scores(g, 0);
            mma_commit(&sh->s_done[g]);
          }
        mma_commit(&sh->empty[0]);
      }
      __syncwarp();
      uint32_t slot = 1, turn = 0;                   // V's place in the ring, and which pass over it; K's next tile follows
#pragma unroll 1
      for (int j = 0; j < ntiles; ++j) {
        const uint32_t next = slot + 1 == kAdSlots ? 0 : slot + 1;
        const uint32_t next_turn = turn ^ (next == 0 ? 1u : 0u);
        const bool more = j + 1 < ntiles;
        wait(&sh->full[slot], turn);
        if (more) wait(&sh->full[next], next_turn);
        const uint64_t b0 = vals0 + slot * kTile;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g >= groups) continue;
          wait(&sh->p_full[g], (uint32_t)(j & 1));
          if (!dead && elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)           // K-step kk: 16 keys, 2 KB on
              mma_ta_as(tO + 128 * g, tS + 128 * g + (uint32_t)(8 * kk), b0 + (uint64_t)(kk * 128), kIdescValues,
                        (j > 0 || kk > 0) ? 1u : 0u);
            if (more) scores(g, next);
            mma_commit(&sh->s_done[g]);                // without more: O_g is complete
            if (g == groups - 1) {
              mma_commit(&sh->empty[slot]);
              if (more) mma_commit(&sh->empty[next]);
            }
          }
          __syncwarp();
        }
        slot = next + 1 == kAdSlots ? 0 : next + 1;
        turn = next_turn ^ (slot == 0 ? 1u : 0u);
      }
      if (dead) {
        *abort_flag = 1;
        // let the products that were issued finish (bounded) before the tensor memory is freed
        if (elect_one()) mma_commit(&sh->drained);
        __syncwarp();
        bar_wait(&sh->drained, 0);
      }
    }
  } else if ((warp >> 3) < a.groups) {
    // ---------------------------------------------------------------- softmax of row tile g
    // two threads of warps four apart take columns 0 .. 63 and 64 .. 127 of a row
    const int g = warp >> 3, side = (warp >> 2) & 1, qi = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tSt = tS + 128 * g + 64 * side + lane_base, tPt = tS + 128 * g + 32 * side + lane_base;
    const uint32_t tOt = tO + 128 * g + 64 * side + lane_base;
    const int row = a.r0 + g * kAtTile + qi;
    const int limit = row < a.r1 ? row_limit(p, query_pos(p, row)) : kLimitNone;
    // the least limit of the warp's live rows
    const int least = __reduce_min_sync(0xffffffffu, limit != kLimitNone ? limit : kPosNever);
    const bool in_order = !a.tail && p.k_pos == nullptr;
    float m_run = kNoMax, l_run = 0.0f;
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      // Does any live row of the warp miss a key of this tile?  Where positions
      // are in order the last one tells; otherwise the lanes look at two each.
      const int k0 = (a.j0 + j) * kAtTile, valid = min(a.n - k0, kAtTile);
      bool masked = valid < kAtTile || (p.causal && in_order && k0 + valid - 1 > least);
      int kp[2];
      if (masked || (p.causal && !in_order)) {
        bool over = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          kp[c] = mask_pos(p, a.tail, a.h, a.b, k0 + 64 * side + 32 * c + lane, a.n);
          over |= kp[c] > least;
        }
        masked = __any_sync(0xffffffffu, over);
      }
      ok = bar_wait_or_abort(&sh->s_done[g], (uint32_t)(j & 1), abort_flag);
      ok = !__any_sync(0xffffffffu, !ok);
      fence_after();
      // The weights are taken against the reference at once; only if some row's
      // maximum turns out more than 8 above it, it rises and they are taken again.
      uint32_t w[2][16];
      float2 sum[2];
      bool gone = false;
      for (;;) {
        uint32_t s[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tld32_start(tSt + 32 * c, s[c]);
        tld_wait();
#pragma unroll
        for (int c = 0; c < 2; ++c) hold32(s[c]);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (__shfl_sync(0xffffffffu, kp[c], e) > limit) s[c][e] = 0xFF800000u;       // -inf
        }
        const float2 sl2 = make_float2(p.sl, p.sl), nm2 = make_float2(-m_run, -m_run);
        float mx[2] = {__uint_as_float(s[0][0]), __uint_as_float(s[1][0])};
        sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float u = __uint_as_float(s[c][2 * e]), v = __uint_as_float(s[c][2 * e + 1]);
            mx[c] = fmaxf(mx[c], fmaxf(u, v));
            const float2 x = __ffma2_rn(make_float2(u, v), sl2, nm2);
            w[c][e] = pack_bf16(exp2_approx(x.x), exp2_approx(x.y));
            // the sum of the rounded weights, the ones the product uses
            sum[c] = __fadd2_rn(sum[c], make_float2(__uint_as_float(w[c][e] << 16), __uint_as_float(w[c][e] & 0xFFFF0000u)));
          }
        const float mine = fmaxf(mx[0], mx[1]) * p.sl;
        sh->top[g][side][qi] = mine;
        // (all of S_g has been read, too: P_g may overwrite it)
        if (!named_bar_or(1 + g, 256, !ok || mine > m_run + 8.0f)) break;
        const float m_new = fmaxf(m_run, fmaxf(mine, sh->top[g][side ^ 1][qi]));
        gone = named_bar_or(1 + g, 256, !ok);
        if (gone) break;
        const float alpha = exp2_approx(m_run - m_new);
        l_run *= alpha;
        m_run = m_new;
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {           // rescale O_g
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t rg[16];
            tld16(tOt + 16 * c, rg);
#pragma unroll
            for (int e = 0; e < 16; ++e) rg[e] = __float_as_uint(__uint_as_float(rg[e]) * alpha);
            tst16(tOt + 16 * c, rg);
          }
        }
      }
      if (gone) { ok = false; break; }
#pragma unroll
      for (int c = 0; c < 2; ++c) tst16(tPt + 16 * c, w[c]);
      l_run += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      warp_arrive(&sh->p_full[g], lane);
    }
    if (ok) {
      if (ntiles > 0) ok = bar_wait_or_abort(&sh->s_done[g], (uint32_t)(ntiles & 1), abort_flag);
      __syncwarp();                                    // the lanes' waits end apart, the barrier below wants them together
      fence_after();
      // the two sums of a row joined, through the row tile, which no product reads any more
      float* sums = reinterpret_cast<float*>(sQ + g * kAtOpBytes);
      sums[128 * side + qi] = l_run;
      ok = !named_bar_or(1 + g, 256, !ok);
      l_run += sums[128 * (side ^ 1) + qi];
    }
    if (!ok) *abort_flag = 1;
    if (ok) {
      const bool whole = p.slots == 1;                 // nothing to join: O itself
      const bool dead = limit == kLimitNone || l_run == 0.0f;
      const int64_t out = (int64_t)a.part * p.R + row;
      if (row < a.r1 && side == 0 && !whole) p.part_ml[out] = make_float2(m_run, dead ? 0.0f : l_run);
      const float inv = dead ? 0.0f : 1.0f / l_run;
      if (ntiles > 0) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t rg[32];
          __syncwarp();                                // a load of the whole warp, which the stores' branches divide
          tld32(tOt + 32 * c, rg);
          if (row >= a.r1) {
            // behind the last row: nothing to store
          } else if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.O + query_row(p, a.h, row) * kD + 64 * side + 32 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = __uint_as_float(rg[8 * e + 2 * i]), y = __uint_as_float(rg[8 * e + 2 * i + 1]);
                w[i] = dead ? 0u : pack_bf16(x * inv, y * inv);
              }
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_O + out * kD + 64 * side + 32 * c);
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
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, 1u);
  if (warp == 0) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

size_t ad_smem_bytes() { return kAdSharedBytes + (size_t)(2 + kAdSlots) * kAtOpBytes; }

}  // namespace

cudaError_t launch_batch_attend(const BatchParams& p, cudaStream_t s) {
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_batch_attend), ad_smem_bytes());
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(p.S1 * p.tiles1 * p.Hn + p.S2 * p.tiles2 * p.Hn * p.B);
  qvg_batch_attend<<<grid, kAdThreads, ad_smem_bytes(), s>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- plans
namespace {

constexpr int kRowStep = 64;                      // keys of a step of the kernels for few rows
constexpr int kSingleStep = 32;                   // and in registers
// Rows beyond which tcgen05 takes over, and up to which registers do.  One
// pass over 16,000 tokens of 32 heads (K = 256, T = 2, G = 64):
//   attention   1 row 95 us in registers; 2 rows 115, and 104 by mma.sync; 64 rows
//               163 by mma.sync, 65 rows 163 by tcgen05 (where the time grows by 8 us
//               up to 128 rows, by mma.sync it doubles);
//   weights     2 rows 75 us in registers, 3 rows 87 by mma.sync; 64 rows 182 by
//               mma.sync, 65 rows 235 by tcgen05, and more by mma.sync.
constexpr int64_t kManyRows = 64;
// Attention of more rows stays with mma.sync while it is so little that the
// launches count: blocks of 64 rows x 64 keys in all.  256 rows: 2 heads of 2,000
// tokens (256 blocks) 25.5 us by mma.sync, 32.5 by tcgen05; 12 of 512 (384) 27.6
// and 32.5; 2 of 5,000 (632) 34.1 and 34.6; 12 of 2,000 (1,536) 50.3 and 36.7.
constexpr int64_t kFewBlocks = 400;
constexpr int64_t kFewMaxRanges = 128;             // ranges of few rows, of the prefix and of a tail
static_assert(2 * kFewMaxRanges <= kMaxSlots && 2 * kAdMaxRanges <= kMaxSlots && kAdMaxRanges + kFewMaxRanges <= kMaxSlots,
              "slots of partial results");
constexpr size_t kImageBudget = size_t(1) << 30;  // operand tiles in the workspace at a time, about

BatchParams params_of(const BatchArgs& a) {
  BatchParams p{};
  for (int w = 0; w < 2; ++w) {
    const qvg_packed* pk = w == 0 ? a.k : a.v;
    if (pk == nullptr) continue;
    p.codes[w] = pk->codes; p.scale[w] = pk->scale; p.zero[w] = pk->zero; p.assign[w] = pk->assign;
    p.tab[w] = static_cast<const __nv_bfloat16*>(pk->centroids);
  }
  const qvg_batch& q = *a.batch;
  p.Q = static_cast<const __nv_bfloat16*>(q.Q);
  p.q_pos = q.q_pos;
  p.k_pos = q.k_pos;
  p.tail[0] = static_cast<const __nv_bfloat16*>(q.tail_k);
  p.tail[1] = static_cast<const __nv_bfloat16*>(q.tail_v);
  p.tail_pos = q.tail_pos;
  p.tail_len = q.tail_len;
  p.rope = reinterpret_cast<const float2*>(static_cast<const char*>(a.tables) + kRopeHeaderBytes);
  p.status = static_cast<uint32_t*>(const_cast<void*>(a.tables));
  p.max_pos = a.max_pos;
  p.Nk = a.Nk; p.Nq = q.Nq; p.Nt = q.Nt;
  p.RB = q.group * q.Nq;
  p.R = q.B * p.RB;
  p.B = q.B; p.H = a.H; p.K = a.K; p.T = a.T; p.G = a.G; p.sym = a.sym; p.causal = q.causal;
  for (int g = a.G; g > 1; g >>= 1) ++p.lgG;
  p.sl = 1.4426950408889634f / sqrtf((float)kD);
  p.nt1 = (p.Nk + kAtTile - 1) / kAtTile;
  p.nt2 = (p.Nt + kAtTile - 1) / kAtTile;
  p.Rp = (p.R + kAdRows - 1) / kAdRows * kAdRows;
  p.RBp = (p.RB + kAdRows - 1) / kAdRows * kAdRows;
  p.Nkp = (p.Nk + kRowStep - 1) / kRowStep * kRowStep;
  p.Hn = p.H;
  return p;
}

// Which kernels run, over which ranges, and what they need of the workspace.
// The prefix goes to the tensor-core kernels when a head has many rows, a tail
// when a sequence has.
struct BatchPlan {
  bool tc1, tc2;                  // prefix, tails
  int S1, S2, Hn;                 // ranges; heads at a time
  int row_tiles;
  int row_cuts;                   // weights of many rows: cuts of the rows of the second pass
  bool single;                    // one row (weights: or two): kernel_attention_single.cu
  size_t bytes;
};

// Places everything in the workspace at `ws` (null: sizes only) and returns
// its length.
size_t place(BatchParams& p, const BatchPlan& plan, bool values, char* ws) {
  size_t at = 0;
  auto take = [&](size_t n) {
    char* r = ws != nullptr ? ws + at : nullptr;
    at += (n + 255) & ~size_t(255);
    return r;
  };
  p.slots = plan.S1 + plan.S2;
  p.slot2 = plan.S1;
  const size_t rows = (size_t)plan.Hn * p.R;
  if (values) p.part_O = reinterpret_cast<float*>(take(p.slots > 1 ? p.slots * rows * kD * sizeof(float) : 0));
  p.part_ml = reinterpret_cast<float2*>(take(p.slots * rows * sizeof(float2)));
  if (!values && !plan.tc1) p.scores = reinterpret_cast<float*>(take((size_t)plan.Hn * p.R * p.Nkp * sizeof(float)));
  if (plan.tc1) {
    p.key_img[0] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.nt1 * kImageBytes));
    p.val_img[0] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.nt1 * kImageBytes));
    p.row_img[0] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.Rp * kD * 2));
    if (!values) {
      p.row_lo[0] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.Rp * kD * 2));
      p.lse = reinterpret_cast<float*>(take((size_t)plan.Hn * p.Rp * sizeof(float)));
      p.limits = reinterpret_cast<int*>(take((size_t)plan.Hn * p.Rp * sizeof(int)));
      p.row_cuts = plan.row_cuts;
      if (p.row_cuts > 1) p.part_w = reinterpret_cast<float*>(take((size_t)plan.row_cuts * plan.Hn * p.Nkp * sizeof(float)));
    }
  }
  if (plan.tc2) {
    p.key_img[1] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.B * p.nt2 * kImageBytes));
    p.val_img[1] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.B * p.nt2 * kImageBytes));
    p.row_img[1] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.B * p.RBp * kD * 2));
    if (!values) p.row_lo[1] = reinterpret_cast<uint8_t*>(take((size_t)plan.Hn * p.B * p.RBp * kD * 2));
  }
  return at;
}

// Estimated time, in steps (or tiles) of keys, of u1 * s1 CTAs of the prefix and
// u2 * s2 of the tails, of which `room` run at a time: a CTA of t steps takes
// t + start, and the tails' CTAs fill the gaps of the prefix's last wave first.
double estimate(int64_t u1, int64_t s1, int64_t n1, int64_t u2, int64_t s2, int64_t n2, double room, double start) {
  const double t1 = s1 > 0 ? (double)((n1 + s1 - 1) / s1) + start : 0.0, t2 = s2 > 0 ? (double)((n2 + s2 - 1) / s2) + start : 0.0;
  const double waves = std::ceil((double)(u1 * s1) / room), free = waves * room - (double)(u1 * s1);
  if ((double)(u2 * s2) <= free && t2 <= t1) return waves * t1;
  const double gaps = free * t1, rest = (double)(u2 * s2) * t2 - 0.8 * gaps;
  return waves * t1 + (rest > 0.0 ? std::max(t2, rest / room + 0.5 * t2) : 0.0);
}

// Ranges for few rows, about as long in the prefix (n1 steps, u1 CTAs a range) as
// in the tails: either part's CTAs fill one to four waves, with or without the
// other's; the least estimated time.
void cut_few(int64_t u1, int64_t n1, int64_t u2, int64_t n2, int64_t room, double start, int* S1, int* S2) {
  double best = -1.0;
  auto consider = [&](int64_t n, int64_t ranges) {
    ranges = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(n, kFewMaxRanges), ranges));
    const int64_t len = (n + ranges - 1) / ranges;
    const int64_t s1 = std::min<int64_t>((n1 + len - 1) / len, kFewMaxRanges), s2 = std::min<int64_t>((n2 + len - 1) / len, kFewMaxRanges);
    const double cost = estimate(u1, s1, n1, u2, s2, n2, (double)room, start);
    if (best >= 0.0 && cost >= best) return;
    best = cost;
    *S1 = (int)s1;
    *S2 = (int)s2;
  };
  for (int64_t k = 1; k <= 4; ++k) {
    if (n1 > 0) consider(n1, k * room / u1);
    if (n1 > 0 && n2 > 0) consider(n1, (k * room - u2) / u1);
    if (n2 > 0) consider(n2, k * room / u2);
    if (n1 > 0 && n2 > 0) consider(n2, (k * room - u1) / u2);
  }
}

// The cut of the keys, by estimated times.  Many rows: a CTA holds an SM, its
// start and end take 3 tiles, and a range's partial results cost their way
// through memory (about a fifth of a tile per CTA's worth of rows and range).
//
// `most` heads at a time at most, in groups of about the same size (a last one of
// few heads would leave SMs idle); `images`
// false: no operand tiles (attention only, the kernels for few rows take any).
BatchPlan plan_heads(BatchParams& p, bool values, int64_t most, bool images) {
  BatchPlan plan{};
  auto heads = [&](int64_t n) {
    n = std::max<int64_t>(1, std::min<int64_t>(n, std::min<int64_t>(most, p.H)));
    const int64_t groups = (p.H + n - 1) / n;
    return (int)((p.H + groups - 1) / groups);
  };
  const double sms = (double)device_sm_count();
  const int64_t blocks = ((p.R + 63) / 64 * ((p.Nk + 63) / 64) + p.B * ((p.RB + 63) / 64) * ((p.Nt + 63) / 64)) * p.H;
  plan.tc1 = p.R > kManyRows && !(values && (blocks <= kFewBlocks || !images));
  plan.tc2 = plan.tc1 && p.Nt > 0 && p.RB > kManyRows;
  plan.Hn = heads(p.H);
  const int64_t few = plan.tc1 ? p.RB : p.R;       // rows of the CTAs of the kernels for few rows
  plan.row_tiles = few <= 16 ? 1 : few <= 32 ? 2 : 4;
  p.row_tiles = plan.row_tiles;
  plan.single = p.R <= (values ? 1 : 2);
  const int64_t tile = 16 * plan.row_tiles, step = plan.single ? kSingleStep : kRowStep;
  const int64_t room = (int64_t)sms * (plan.single ? single_per_sm(p, values) : rows_per_sm(p, values));
  const int64_t steps1 = plan.tc1 ? 0 : (p.Nk + step - 1) / step, steps2 = plan.tc2 ? 0 : (p.Nt + step - 1) / step;
  if (plan.tc1) {
    size_t per_head = (size_t)p.nt1 * 2 * kImageBytes;
    if (plan.tc2) per_head += (size_t)p.B * p.nt2 * 2 * kImageBytes;
    plan.Hn = heads((int64_t)(kImageBudget / per_head));
  } else if (!values) {
    plan.Hn = heads((int64_t)(kImageBudget / ((size_t)p.R * p.Nkp * sizeof(float))));
  }
  if (steps1 + steps2 > 0) {
    const int64_t units1 = (p.R + tile - 1) / tile * plan.Hn, units2 = (p.RB + tile - 1) / tile * plan.Hn * p.B;
    cut_few(units1, steps1, units2, steps2, room, plan.single ? 6.0 : 1.5, &plan.S1, &plan.S2);
  }
  if (plan.tc1) {
    const int64_t u1 = (p.Rp / kAdRows) * plan.Hn, u2 = plan.tc2 ? (p.RBp / kAdRows) * plan.Hn * p.B : 0;
    double best = -1.0;
    for (int64_t s1 = 1; s1 <= std::min<int64_t>(p.nt1, kAdMaxRanges); ++s1) {
      if (s1 > 16 && (double)(u1 * s1) > 2.0 * sms) break;            // beyond two waves more ranges gain nothing
      // a tail's ranges about as long as the prefix's, or the whole tail
      const int64_t len = (p.nt1 + s1 - 1) / s1 + 3;
      const int64_t cut = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(p.nt2, kAdMaxRanges), (p.nt2 + len / 2) / len));
      for (int64_t s2 : {u2 > 0 ? cut : 0, u2 > 0 ? int64_t(1) : 0}) {
        double cost = estimate(u1, s1, p.nt1, u2, s2, p.nt2, sms, 3.0);
        if (s1 + s2 + (plan.tc2 ? 0 : plan.S2) > 1) cost += 2.0 + 0.2 * ((double)s1 * (double)u1 + (double)s2 * (double)u2) / sms;
        if (best < 0.0 || cost < best) {
          best = cost;
          plan.S1 = (int)s1;
          if (plan.tc2) plan.S2 = (int)s2;
        }
      }
    }
  }
  plan.row_cuts = 1;
  if (plan.tc1 && !values) {
    // The sums by key of few keys leave SMs idle: cut the rows, too, where that
    // saves more than the joining launch takes (about 2.5 tiles' time): 2 heads
    // of 66 keys and 2,774 rows 49 us a call in one piece, 31 in cuts.
    const int64_t units = (p.nt1 + 1) / 2 * plan.Hn, tiles = (p.R + kAtTile - 1) / kAtTile;
    double least = estimate(units, 1, tiles, 0, 0, 0, sms, 3.0);
    for (int64_t s = 2; s <= std::min<int64_t>(tiles, 32) && units * s <= 2 * (int64_t)sms; ++s) {
      const int64_t per = (tiles + s - 1) / s;
      const double cost = std::ceil((double)(units * s) / sms) * ((double)per + 3.0) + 2.5;
      if (cost < least) { least = cost; plan.row_cuts = (int)s; }
    }
  }
  plan.bytes = place(p, plan, values, nullptr);
  return plan;
}

// The plan for a workspace of `room` bytes: where it does not hold what the
// call would like, fewer heads at a time, and where not even one head's tiles
// fit, attention without them.  One head's plan does not depend on how many there
// are, so that what the call asks for with H = 1 is always enough.
BatchPlan plan_within(BatchParams& p, bool values, size_t room) {
  BatchPlan plan{};
  for (const bool images : {true, false}) {
    plan = plan_heads(p, values, p.H, images);
    while (plan.bytes > room && plan.Hn > 1)
      plan = plan_heads(p, values, std::min<int64_t>(plan.Hn - 1, (int64_t)((double)plan.Hn * ((double)room / (double)plan.bytes))), images);
    if (plan.bytes <= room || !values || !plan.tc1) break;
  }
  return plan;
}
BatchPlan plan_batch(BatchParams& p, bool values) { return plan_heads(p, values, p.H, true); }

// Partial results of few rows.
cudaError_t launch_few(const BatchPlan& plan, const BatchParams& p, bool values, cudaStream_t s) {
  return plan.single ? launch_single_partial(p, values, s) : launch_rows_partial(p, values, s);
}

// The launch's share of the plan: what the kernels for few rows take, or the
// tensor-core kernels, of the heads from h0.
BatchParams share(const BatchParams& p, const BatchPlan& plan, bool tc, int h0) {
  BatchParams q = p;
  q.h0 = h0;
  q.Hn = std::min(plan.Hn, p.H - h0);
  q.S1 = plan.tc1 == tc ? plan.S1 : 0;
  q.S2 = plan.tc2 == tc ? plan.S2 : 0;
  q.row_tiles = plan.row_tiles;
  const int64_t tile = tc ? kAdRows : 16 * plan.row_tiles;
  q.tiles1 = (p.R + tile - 1) / tile;
  q.tiles2 = (p.RB + tile - 1) / tile;
  return q;
}

}  // namespace

size_t attention_batch_workspace_bytes(const BatchArgs& a) {
  BatchParams p = params_of(a);
  return plan_batch(p, true).bytes;
}

size_t attention_weights_workspace_bytes(const BatchArgs& a) {
  BatchParams p = params_of(a);
  return plan_batch(p, false).bytes;
}

// The tensor-core kernels record a timeout in the tables' status word; those
// for few rows wait for nothing.
static qvg_status ready(const BatchPlan& plan, const BatchArgs& a, size_t ws_bytes, cudaStream_t s) {
  if (ws_bytes < plan.bytes) return QVG_ERR_WORKSPACE_TOO_SMALL;
  return plan.tc1 || plan.tc2 ? peek_sticky(a.tables, s) : QVG_OK;
}

static cudaError_t queue_attention(const BatchPlan& plan, BatchParams& p, void* O, void* ws, cudaStream_t s) {
  place(p, plan, true, static_cast<char*>(ws));
  p.O = static_cast<__nv_bfloat16*>(O);
  cudaError_t e = cudaSuccess;
  for (int h0 = 0; h0 < p.H; h0 += plan.Hn) {
    const BatchParams few = share(p, plan, false, h0), tc = share(p, plan, true, h0);
    if (few.S1 + few.S2 > 0 && (e = launch_few(plan, few, true, s)) != cudaSuccess) return e;
    if (plan.tc1) {
      if ((e = launch_batch_expand(tc, false, s)) != cudaSuccess) return e;
      if ((e = launch_batch_attend(tc, s)) != cudaSuccess) return e;
    }
    if (p.slots > 1 && (e = launch_batch_merge(few, s)) != cudaSuccess) return e;
  }
  return e;
}

static cudaError_t queue_weights(const BatchPlan& plan, BatchParams& p, const float* received, float* out, void* ws, cudaStream_t s) {
  place(p, plan, false, static_cast<char*>(ws));
  cudaError_t e = cudaSuccess;
  for (int h0 = 0; h0 < p.H; h0 += plan.Hn) {
    const BatchParams few = share(p, plan, false, h0), tc = share(p, plan, true, h0);
    if (few.S1 + few.S2 > 0 && (e = launch_few(plan, few, false, s)) != cudaSuccess) return e;
    if (!plan.tc1) {
      if ((e = launch_rows_weights(few, received, out, s)) != cudaSuccess) return e;
      continue;
    }
    if ((e = launch_batch_expand(tc, true, s)) != cudaSuccess) return e;
    if ((e = launch_batch_stats(tc, s)) != cudaSuccess) return e;
    if ((e = launch_batch_weights(tc, tc.lse, tc.limits, received, out, s)) != cudaSuccess) return e;
  }
  return e;
}

qvg_status launch_attention_batch(const BatchArgs& a, void* O, void* ws, size_t ws_bytes, cudaStream_t s) {
  BatchParams p = params_of(a);
  const BatchPlan plan = plan_within(p, true, ws_bytes);
  const qvg_status st = ready(plan, a, ws_bytes, s);
  if (st != QVG_OK) return st;
  return queue_attention(plan, p, O, ws, s) == cudaSuccess ? QVG_OK : QVG_ERR_CUDA;
}

qvg_status launch_attention_weights(const BatchArgs& a, const float* received, float* out, void* ws, size_t ws_bytes, cudaStream_t s) {
  BatchParams p = params_of(a);
  const BatchPlan plan = plan_within(p, false, ws_bytes);
  const qvg_status st = ready(plan, a, ws_bytes, s);
  if (st != QVG_OK) return st;
  return queue_weights(plan, p, received, out, ws, s) == cudaSuccess ? QVG_OK : QVG_ERR_CUDA;
}

}  // namespace qvg
