// kernel_batch_weights.cu -- qvg_attention_weights for many rows, on tcgen05.
//
// The weight of key j is sum_r 2^(x_rj - lse_r), x_rj = sl q_r.k_j, lse_r the
// base-2 logarithm of row r's sum over all its keys: a pass over the rows'
// scores for lse, and a second one for the sums by key.  Both are one kernel:
// two tiles of 128 stay in shared memory (rows in the first pass, keys in the
// second) while the others stream by, and two threads reduce the scores of
// each resident row or key over the stream, 64 columns of a tile each.  In the second pass the keys are the
// M side of the product, so a key's sum stays in its threads and is taken
// in one order, without atomics.
//
// A score must be good to about fp32 (a sum of weights is an fp32 result), so each
// operand is two fp16 halves (2^-22 of itself, below 2^-3 2^-25 absolute) and a
// score three products, high x high, low x high and high x low: 24 tensor
// instructions a pair of tiles; the products are
// the bound (12 heads, 1,560 rows, 24,960 keys: 311 and 300 us a pass, 1,180
// TFLOP/s of products, 84 % of cuBLAS's sustained rate).
// Stream tiles come as a high and a low half of 32 KB through a ring of three
// slots; the scores are double-buffered in tensor memory, 128 columns for each
// of two resident tiles.  Eighteen warps as in kernel_batch_attend.cu, all waits
// bounded.
#include "attention_tc.cuh"
#include "batch.cuh"

namespace qvg {
namespace {

constexpr int kWtThreads = 576;                   // 16 reducing warps, the issuer's, the loader's
constexpr int kWtSlots = 3;                       // ring of half tiles

struct __align__(16) WtShared {
  float lse[2][kAtTile];          // of the streamed rows (second pass)
  uint64_t full[kWtSlots], empty[kWtSlots];
  uint64_t resident;
  uint64_t s_done[2][2];          // scores of resident tile g in buffer i complete
  uint64_t s_free[2][2];          // and read: an arrival of each of 8 warps
  uint64_t v_full[2], v_free[2];  // lse buffers: 8 warps' arrivals for each resident tile free them
  uint64_t drained;
  uint32_t tmem_base;
  int abort_flag;
  int failed;                     // second pass: a wait had run out before this launch
};

// What a CTA has to do.  First pass (STATS): rows r0 .. of head h over tiles
// j0 .. of the prefix's or a tail's keys.  Second: keys 256 tile .. over the
// tiles j0 .. of rows: all of them, or where there are few keys one of the
// plan's cuts, whose sums qvg_batch_sums joins.
struct WtPlace {
  bool tail;
  int hl, h, b, slot;
  int n;                          // keys of the prefix or tail
  int j0, steps;                  // stream tiles
  int first, end;                 // resident rows (of the head) or keys
  int groups;
};
template <bool STATS>
__device__ __forceinline__ WtPlace wt_place(const BatchParams& p) {
  WtPlace a;
  if (STATS) {
    const int64_t first_tail = (int64_t)p.S1 * p.tiles1 * p.Hn;
    a.tail = blockIdx.x >= first_tail;
    const uint32_t e = (uint32_t)(a.tail ? blockIdx.x - first_tail : blockIdx.x);
    const uint32_t S = (uint32_t)(a.tail ? p.S2 : p.S1), nb = (uint32_t)(a.tail ? p.tiles2 : p.tiles1);
    const uint32_t range = e % S, block = e / S % nb, unit = e / S / nb;
    a.hl = (int)(unit % (uint32_t)p.Hn);
    a.b = (int)(unit / (uint32_t)p.Hn);
    a.n = (int)(a.tail ? tail_length(p, a.b) : p.Nk);
    a.slot = (int)(a.tail ? p.slot2 + range : range);
    a.first = (int)((a.tail ? a.b * p.RB : 0) + block * 2 * kAtTile);
    a.end = (int)(a.tail ? (a.b + 1) * p.RB : p.R);
    const uint32_t nt = (uint32_t)(a.n + kAtTile - 1) / kAtTile;     // below 2^16, S at most 64
    a.j0 = (int)(nt * range / S);
    a.steps = (int)(nt * (range + 1) / S) - a.j0;
  } else {
    const uint32_t per = (uint32_t)(p.nt1 + 1) / 2;
    a.tail = false;
    const uint32_t S = (uint32_t)p.row_cuts, cut = blockIdx.x % S, e = blockIdx.x / S;
    a.hl = (int)(e / per);
    a.b = 0;
    a.slot = (int)cut;
    a.n = (int)p.Nk;
    a.first = (int)(e % per) * 2 * kAtTile;
    a.end = a.n;
    const uint32_t nt = (uint32_t)(p.R + kAtTile - 1) / kAtTile;
    a.j0 = (int)(nt * cut / S);
    a.steps = (int)(nt * (cut + 1) / S) - a.j0;
  }
  a.h = p.h0 + a.hl;
  a.groups = a.end - a.first > kAtTile ? 2 : 1;
  return a;
}

template <bool STATS>
__global__ void __launch_bounds__(kWtThreads, 1) qvg_batch_weights(const BatchParams p, const float* lse, const int* limits,
                                                                  const float* received, float* out) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* own = smem;                              // resident tile g: high half at 2g tiles, low half after it
  uint8_t* ring = own + 4 * kAtOpBytes;
  WtShared* sh = reinterpret_cast<WtShared*>(ring + kWtSlots * kAtOpBytes);
  volatile int* abort_flag = &sh->abort_flag;
  WtPlace a = wt_place<STATS>(p);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWtSlots; ++i) { bar_init(&sh->full[i], 1); bar_init(&sh->empty[i], 1); }
    bar_init(&sh->resident, 1);
    bar_init(&sh->drained, 1);
    for (int i = 0; i < 2; ++i) {
      for (int g = 0; g < 2; ++g) { bar_init(&sh->s_done[g][i], 1); bar_init(&sh->s_free[g][i], 8); }
      bar_init(&sh->v_full[i], 1);
      bar_init(&sh->v_free[i], (uint32_t)(a.groups * 8));
    }
    sh->abort_flag = 0;
    sh->failed = !STATS && *static_cast<const volatile uint32_t*>(p.status) != 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh->tmem_base)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  // After a wait that ran out (in the first pass above all) the rows' logarithms may
  // be anything: no rows then, so that every key keeps what it received before.
  if (!STATS && sh->failed) a.steps = 0;
  const uint32_t tmem = uniform(sh->tmem_base);              // scores of resident tile g in buffer i at column 256 g + 128 i

  if (warp == 17) {
    // ---------------------------------------------------------------- loader
    if (lane == 0 && a.steps > 0) {
      // key tiles are whole images; row tiles are two halves of 64 channels, Rp or RBp rows apart
      const int64_t unit = (a.tail ? (int64_t)a.b * p.Hn : 0) + a.hl;
      const int64_t nt = a.tail ? p.nt2 : p.nt1, pad = a.tail ? p.RBp : p.Rp;
      auto load_keys = [&](uint32_t dst, int64_t tile, bool low, uint64_t* bar) {
        bulk_load(dst, (low ? p.val_img : p.key_img)[a.tail] + (unit * nt + tile) * kImageBytes, (uint32_t)kImageBytes, bar);
      };
      auto load_rows = [&](uint32_t dst, int64_t row, bool low, uint64_t* bar) {
        const uint8_t* src = (low ? p.row_lo : p.row_img)[a.tail] + (unit * 2 * pad + row) * 128;
        bulk_load(dst, src, kAtHalfBytes, bar);
        bulk_load(dst + kAtHalfBytes, src + pad * 128, kAtHalfBytes, bar);
      };
      expect_bytes(&sh->resident, (uint32_t)(2 * a.groups * kAtOpBytes));
      for (int g = 0; g < a.groups; ++g)
        for (int low = 0; low < 2; ++low) {
          const uint32_t dst = smem_addr(own) + (2 * g + low) * kAtOpBytes;
          if (STATS) load_rows(dst, a.first - (a.tail ? a.b * p.RB : 0) + g * kAtTile, low != 0, &sh->resident);
          else load_keys(dst, a.first / kAtTile + g, low != 0, &sh->resident);
        }
      int issued = 0, vectors = 0;
      for (int i = 0; i < 2 * a.steps; ++i) {
        const int slot = i % kWtSlots, turn = i / kWtSlots, j = i >> 1;
        if (turn > 0 && !bar_wait_or_abort(&sh->empty[slot], (uint32_t)((turn - 1) & 1), abort_flag)) { *abort_flag = 1; break; }
        expect_bytes(&sh->full[slot], (uint32_t)kAtOpBytes);
        const uint32_t dst = smem_addr(ring) + slot * kAtOpBytes;
        if (STATS) load_keys(dst, a.j0 + j, (i & 1) != 0, &sh->full[slot]);
        else load_rows(dst, (int64_t)(a.j0 + j) * kAtTile, (i & 1) != 0, &sh->full[slot]);
        ++issued;
        if (!STATS && (i & 1) == 0) {
          if (j > 1 && !bar_wait_or_abort(&sh->v_free[j & 1], (uint32_t)(((j >> 1) - 1) & 1), abort_flag)) { *abort_flag = 1; break; }
          const int64_t at = (int64_t)a.hl * p.Rp + (int64_t)(a.j0 + j) * kAtTile;
          expect_bytes(&sh->v_full[j & 1], kAtTile * 4);
          bulk_load(smem_addr(sh->lse[j & 1]), lse + at, kAtTile * 4, &sh->v_full[j & 1]);
          ++vectors;
        }
      }
      // no copy may be in flight when the CTA leaves
      bar_wait(&sh->resident, 0);
      for (int i = issued > kWtSlots ? issued - kWtSlots : 0; i < issued; ++i)
        bar_wait(&sh->full[i % kWtSlots], (uint32_t)((i / kWtSlots) & 1));
      for (int j = vectors > 2 ? vectors - 2 : 0; j < vectors; ++j) bar_wait(&sh->v_full[j & 1], (uint32_t)((j >> 1) & 1));
    }
  } else if (warp == 16) {
    // ---------------------------------------------------------------- issuer
    const int steps = uniform(a.steps), groups = uniform(a.groups);
    // after a failed wait the loop runs on without waiting or issuing
    if (steps > 0) {
      bool dead = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !bar_wait_or_abort(bar, parity, abort_flag);
        dead = __any_sync(0xffffffffu, dead);
        fence_after();
      };
      const uint64_t own0 = op_desc(smem_addr(own)), ring0 = op_desc(smem_addr(ring));
      constexpr uint32_t kTile = kAtOpBytes >> 4;
      // columns (+)= resident half `low` of tile g times the half tile in `slot`
      auto product = [&](int g, int low, uint32_t slot, uint32_t columns, bool add) {
        const uint64_t a0 = own0 + (2 * g + low) * kTile, b0 = ring0 + slot * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_as(columns + 256 * g, a0 + desc_step(kk), b0 + desc_step(kk), kIdescScores, add || kk > 0 ? 1u : 0u);
      };
      wait(&sh->resident, 0);
      uint32_t hi = 0, lo = 1, hi_turn = 0, lo_turn = 0;     // slots of the two halves, and which pass over the ring
      auto onward = [](uint32_t& slot, uint32_t& turn) {
        slot += 2;
        if (slot >= kWtSlots) { slot -= kWtSlots; turn ^= 1u; }
      };
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const uint32_t buf = (uint32_t)j & 1u, columns = tmem + 128 * buf;
        wait(&sh->full[hi], hi_turn);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g >= groups) continue;
          if (j > 1) wait(&sh->s_free[g][buf], (uint32_t)(((j >> 1) - 1) & 1));
          if (!dead && elect_one()) {
            product(g, 0, hi, columns, false);
            product(g, 1, hi, columns, true);
            if (g == groups - 1) mma_commit(&sh->empty[hi]);
          }
          __syncwarp();
        }
        wait(&sh->full[lo], lo_turn);
        if (!dead && elect_one()) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= groups) continue;
            product(g, 0, lo, columns, true);
            mma_commit(&sh->s_done[g][buf]);
          }
          mma_commit(&sh->empty[lo]);
        }
        __syncwarp();
        onward(hi, hi_turn);
        onward(lo, lo_turn);
      }
      if (dead) *abort_flag = 1;
      // every product has finished (bounded) before the tensor memory is freed
      if (elect_one()) mma_commit(&sh->drained);
      __syncwarp();
      bar_wait(&sh->drained, 0);
    }
  } else if ((warp >> 3) < a.groups) {
    // ---------------------------------------------------------------- a thread's row (STATS) or key over the stream
    // two threads of warps four apart take columns 0 .. 63 and 64 .. 127
    const int g = warp >> 3, side = (warp >> 2) & 1, mine = a.first + g * kAtTile + (threadIdx.x & 127);
    const uint32_t tD = tmem + 256 * g + 64 * side + ((uint32_t)(32 * (warp & 3)) << 16);
    const bool in = mine < a.end;
    const float2 sl2 = make_float2(p.sl, p.sl);
    // STATS: the row's limit and the least of the warp's live rows; otherwise
    // the key's position and the largest of the warp's keys
    int limit = kLimitNone, bound = 0;
    if (STATS) {
      limit = in ? row_limit(p, query_pos(p, mine)) : kLimitNone;
      bound = __reduce_min_sync(0xffffffffu, limit != kLimitNone ? limit : kPosNever);
    } else {
      limit = mask_pos(p, false, a.h, 0, in ? mine : a.n - 1, a.n);
      bound = __reduce_max_sync(0xffffffffu, limit);
    }
    const bool in_order = STATS && !a.tail && p.k_pos == nullptr;
    float m_run = kNoMax, total = 0.0f;
    bool ok = true;
    for (int j = 0; j < a.steps; ++j) {
      const int buf = j & 1;
      bool masked = false;
      int kp[2];                                     // positions of the streamed keys, or limits of the streamed rows
      if (STATS) {
        const int k0 = (a.j0 + j) * kAtTile, valid = min(a.n - k0, kAtTile);
        masked = valid < kAtTile || (p.causal && in_order && k0 + valid - 1 > bound);
        if (masked || (p.causal && !in_order)) {
          bool over = false;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            kp[c] = mask_pos(p, a.tail, a.h, a.b, k0 + 64 * side + 32 * c + lane, a.n);
            over |= kp[c] > bound;
          }
          masked = __any_sync(0xffffffffu, over);
        }
      } else {
        if (p.causal) {
          bool under = false;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            kp[c] = __ldg(limits + (int64_t)a.hl * p.Rp + (a.j0 + j) * kAtTile + 64 * side + 32 * c + lane);
            under |= kp[c] < bound;
          }
          masked = __any_sync(0xffffffffu, under);
        }
        ok = bar_wait_or_abort(&sh->v_full[buf], (uint32_t)((j >> 1) & 1), abort_flag);
      }
      ok = ok && bar_wait_or_abort(&sh->s_done[g][buf], (uint32_t)((j >> 1) & 1), abort_flag);
      if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
      fence_after();
      uint32_t s[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) tld32_start(tD + 128 * buf + 32 * c, s[c]);
      tld_wait();
#pragma unroll
      for (int c = 0; c < 2; ++c) hold32(s[c]);
      fence_before();
      warp_arrive(&sh->s_free[g][buf], lane);         // the scores are in registers
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      if (STATS) {
        if (masked) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (__shfl_sync(0xffffffffu, kp[c], e) > limit) s[c][e] = 0xFF800000u;       // -inf
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(s[c >> 1][16 * (c & 1)]);
#pragma unroll
          for (int e = 1; e < 16; ++e) mx[c] = fmaxf(mx[c], __uint_as_float(s[c >> 1][16 * (c & 1) + e]));
        }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.sl;
        const float m_new = fmaxf(m_run, mt);
        const float2 nm2 = make_float2(-m_new, -m_new);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), sl2, nm2);
            sum[e & 1] = __fadd2_rn(sum[e & 1], make_float2(exp2_approx(x.x), exp2_approx(x.y)));
          }
        total = total * exp2_approx(m_run - m_new) + ((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y));
        m_run = m_new;
      } else {
        const float4* rows = reinterpret_cast<const float4*>(sh->lse[buf] + 64 * side);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 l = rows[8 * c + e];
            float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e]), __uint_as_float(s[c][4 * e + 1])), sl2, make_float2(-l.x, -l.y));
            float2 y = __ffma2_rn(make_float2(__uint_as_float(s[c][4 * e + 2]), __uint_as_float(s[c][4 * e + 3])), sl2, make_float2(-l.z, -l.w));
            if (masked) {
              if (limit > __shfl_sync(0xffffffffu, kp[c], 4 * e)) x.x = -INFINITY;
              if (limit > __shfl_sync(0xffffffffu, kp[c], 4 * e + 1)) x.y = -INFINITY;
              if (limit > __shfl_sync(0xffffffffu, kp[c], 4 * e + 2)) y.x = -INFINITY;
              if (limit > __shfl_sync(0xffffffffu, kp[c], 4 * e + 3)) y.y = -INFINITY;
            }
            sum[0] = __fadd2_rn(sum[0], make_float2(exp2_approx(x.x), exp2_approx(x.y)));
            sum[1] = __fadd2_rn(sum[1], make_float2(exp2_approx(y.x), exp2_approx(y.y)));
          }
        total += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        warp_arrive(&sh->v_free[buf], lane);
      }
    }
    if (!ok) *abort_flag = 1;
    // the row's or key's two halves joined, through the resident tile, which no
    // product reads any more
    float2* half = reinterpret_cast<float2*>(own + 2 * g * kAtOpBytes) + (threadIdx.x & 127);
    __syncwarp();
    if (STATS) {
      if (side == 1) *half = make_float2(m_run, total);
      ok = !named_bar_or(1 + g, 256, !ok);
      if (side == 0) {
        const float2 other = *half;
        const float M = fmaxf(m_run, other.x);
        total = total * exp2_approx(m_run - M) + other.y * exp2_approx(other.x - M);
        m_run = M;
      }
    } else {
      if (side == 1) half->x = total;
      ok = !named_bar_or(1 + g, 256, !ok);
      if (side == 0) total = ok ? total + half->x : 0.0f;          // after a failed wait: nothing is added
    }
    // a single range: nothing for qvg_batch_lse to join
    if (STATS && ok && side == 0 && p.slots == 1) {
      const bool seen = limit != kLimitNone && total != 0.0f;
      const int64_t at = (int64_t)a.hl * p.Rp + mine;
      p.lse[at] = seen ? m_run + log2f(total) : INFINITY;
      p.limits[at] = seen ? limit : in ? unseen_limit(p, query_pos(p, mine)) : kLimitAll;
    }
    if ((ok || !STATS) && in && side == 0) {
      if (STATS) {
        if (p.slots > 1) p.part_ml[((int64_t)a.slot * p.Hn + a.hl) * p.R + mine] = make_float2(m_run, limit == kLimitNone ? 0.0f : total);
      } else if (p.row_cuts > 1) {
        p.part_w[((int64_t)a.slot * p.Hn + a.hl) * p.Nkp + mine] = total;
      } else {
        const int64_t at = (int64_t)a.h * p.Nk + mine;
        out[at] = (received != nullptr ? received[at] : 0.0f) + total;
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

// The rows' lse from the partial results, and their limits, for the second
// pass: lse = +inf (every weight 0) for a row that sees nothing and behind the
// last row.
__global__ void __launch_bounds__(256) qvg_batch_lse(const BatchParams p, float* lse, int* limits) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= p.Hn * p.Rp) return;
  const int hl = (int)(e / p.Rp);
  const int64_t r = e - hl * p.Rp, row = (int64_t)hl * p.R + r, stride = (int64_t)p.Hn * p.R;
  float x = INFINITY;
  int limit = kLimitAll;
  if (r < p.R) {
    float M = kNoMax, L = 0.0f;
    for (int s = 0; s < p.slots; ++s) M = fmaxf(M, __ldg(p.part_ml + s * stride + row).x);
    for (int s = 0; s < p.slots; ++s) {
      const float2 ml = __ldg(p.part_ml + s * stride + row);
      L += ml.y * exp2_approx(ml.x - M);
    }
    const int64_t pos = query_pos(p, r);
    limit = unseen_limit(p, pos);
    if (L != 0.0f) {
      x = M + log2f(L);
      limit = row_limit(p, pos);
    }
  }
  lse[e] = x;
  limits[e] = limit;
}

// out = received + the sums of the cuts of the rows, in their order.
__global__ void __launch_bounds__(256) qvg_batch_sums(const BatchParams p, const float* received, float* out) {
  const uint32_t per = (uint32_t)(p.Nk + 255) / 256;
  const int hl = (int)(blockIdx.x / per);
  const int64_t j = (int64_t)(blockIdx.x % per) * 256 + threadIdx.x;
  if (j >= p.Nk) return;
  const float* part = p.part_w + (int64_t)hl * p.Nkp + j;
  float sum = 0.0f;
#pragma unroll 8
  for (int s = 0; s < p.row_cuts; ++s) sum += __ldg(part + (int64_t)s * p.Hn * p.Nkp);
  const int64_t at = (int64_t)(p.h0 + hl) * p.Nk + j;
  out[at] = (received != nullptr ? received[at] : 0.0f) + sum;
}

size_t wt_smem_bytes() { return 1024 + (size_t)(4 + kWtSlots) * kAtOpBytes + sizeof(WtShared); }

}  // namespace

cudaError_t launch_batch_stats(const BatchParams& p, cudaStream_t s) {
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_batch_weights<true>), wt_smem_bytes());
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(p.S1 * p.tiles1 * p.Hn + p.S2 * p.tiles2 * p.Hn * p.B);
  qvg_batch_weights<true><<<grid, kWtThreads, wt_smem_bytes(), s>>>(p, nullptr, nullptr, nullptr, nullptr);
  return cudaGetLastError();
}

cudaError_t launch_batch_weights(const BatchParams& p, float* lse, int* limits, const float* received, float* out, cudaStream_t s) {
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(qvg_batch_weights<false>), wt_smem_bytes());
  if (e != cudaSuccess) return e;
  if (p.slots > 1) {
    qvg_batch_lse<<<(unsigned)((p.Hn * p.Rp + 255) / 256), 256, 0, s>>>(p, lse, limits);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  qvg_batch_weights<false><<<(unsigned)((p.nt1 + 1) / 2 * p.Hn * p.row_cuts), kWtThreads, wt_smem_bytes(), s>>>(p, lse, limits, received, out);
  if (p.row_cuts == 1 || (e = cudaGetLastError()) != cudaSuccess) return e != cudaSuccess ? e : cudaGetLastError();
  qvg_batch_sums<<<(unsigned)((p.Nk + 255) / 256 * p.Hn), 256, 0, s>>>(p, received, out);
  return cudaGetLastError();
}

}  // namespace qvg
