// attention_tc.cuh -- what the tcgen05 attention kernels share: their shape,
// bounded barrier waits, operand layout, tensor-core and tensor-memory
// wrappers, distributed shared memory, and the reconstruction of cached tokens
// in registers.
#pragma once

#include "qvg_common.cuh"

namespace qvg {
namespace {

constexpr int kAtThreads = 768;                 // 24 warps
constexpr int kAtQTiles = 2;                    // query tiles per CTA (each reconstructed K/V tile serves both)
constexpr int kAtSoftmaxThreads = 256;          // warps 0-7: softmax of the two query tiles (threads 0 and 128 issue the MMAs)
constexpr int kAtReconThreads = 512;            // warps 8-23: reconstruction into the K/V ring
constexpr int kAtTile = 128;                    // queries per query tile, cached tokens per tile
constexpr int kAtOpBytes = kAtTile * kD * 2;    // one 128 x 128 bf16 operand: 32 KB
constexpr uint64_t kAtWaitNs = 2000000000ull;   // 2 s per bounded wait

struct __align__(8) AtBars {
  uint64_t s_done[2];       // S product of query tile g complete (tcgen05.commit)
  uint64_t o_done[2];       // O product of query tile g complete (tcgen05.commit)
  uint64_t kv_full[2];      // ring stage reconstructed (lane 0 of every reconstruction warp of each CTA that writes it)
  uint64_t kv_empty[2];     // ring stage free again: the O products of every CTA that read it completed
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// The clock (and the abort flag) are looked at only after 63 tries: reading the
// timer takes longer than most waits.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_addr(bar);
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u) {
      uint64_t now;
      asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAtWaitNs) return false;
    }
  }
}

// bar_wait that also gives up as soon as another role of the CTA has
// recorded an abort (so that no role waits out the full limit for a
// partner that has stopped).
__device__ __forceinline__ bool bar_wait_or_abort(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  const uint32_t addr = smem_addr(bar);
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u) {
      if (*abort_flag) return false;
      uint64_t now;
      asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAtWaitNs) return false;
    }
  }
}
// bar_wait_or_abort with acquire at cluster scope: the barrier also takes
// arrivals (and the writes they release) from the other CTA of a pair.
__device__ __forceinline__ bool bar_wait_cluster(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  const uint32_t addr = smem_addr(bar);
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u) {
      if (*abort_flag) return false;
      uint64_t now;
      asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > kAtWaitNs) return false;
    }
  }
}
// Named barrier over `count` threads with an OR of `pred` (every participant
// gets the same answer).
__device__ __forceinline__ bool named_bar_or(int id, int count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// one arrival for a converged warp, after what its lanes did: the lanes' own
// arrivals on one barrier would go one after another (256 of them took longer
// than the tile's products)
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// arrive on a barrier of another CTA of the cluster (shared::cluster
// address), releasing this thread's earlier writes at cluster scope
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr_of_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr_of_bar) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_cluster_b32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Shared-memory operand descriptor, K-major, 128-byte swizzle: a 128 x 128
// bf16 operand is two 64-column halves of 128 rows x 128 bytes (16 KB apart),
// and in each 8-row group of 1,024 bytes (SBO) the 16-byte chunk c of row r
// sits at chunk position c ^ (r mod 8).  The swizzle spreads a warp's stores
// of one chunk column over all banks.
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)1 << 16;                 // LBO (unused with this swizzle)
  d |= (uint64_t)(1024 >> 4) << 32;       // SBO
  d |= (uint64_t)1 << 46;                 // version
  d |= (uint64_t)2 << 61;                 // SWIZZLE_128B
  return d;
}
constexpr int kAtHalfBytes = kAtTile * 128;     // one 64-column half of an operand
// Byte offset of element (row, k) of a 128 x 128 operand (k even for the
// 4-byte stores, a multiple of 8 for the 16-byte ones).
__device__ __forceinline__ int op_off(int row, int k) {
  return (k >> 6) * kAtHalfBytes + row * 128 + ((((k & 63) >> 3) ^ (row & 7)) << 4) + (k & 7) * 2;
}
// Descriptor of K-step kk (16 columns) of the operand at saddr.
__device__ __forceinline__ uint64_t op_desc_k(uint32_t saddr, int kk) {
  return op_desc(saddr + (uint32_t)((kk >> 2) * kAtHalfBytes + (kk & 3) * 32));
}

// kind::f16, A = B = bf16, D = f32, both K-major, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 3) << 17) |
                            ((uint32_t)(128 >> 4) << 24);

__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(kIdesc), "r"(accumulate)
      : "memory");
}
// The same product with A read from tensor memory (lane i = row i, K
// elements packed two per 32-bit column, the lower half first).
__device__ __forceinline__ void mma_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(kIdesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// the same arrival on the barrier at this offset in every CTA of `mask`
// (bit i = cluster rank i)
__device__ __forceinline__ void mma_commit_mc(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  // the registers pass through the wait so that no use moves above it
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
        "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
        "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}

__device__ __forceinline__ void tld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  // the registers pass through the wait so that no use moves above it
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}
__device__ __forceinline__ void tst16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tst8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Distributed shared memory of the CTA's cluster: the address of the same
// shared-memory location in CTA `rank`, loads from it, and the cluster-wide
// barrier (every thread of every CTA arrives; release/acquire order the
// shared-memory writes before it with the reads after it).
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Two E4M3 bytes (low byte first) as fp32 values, through the hardware
// conversion to f16 (exact for every finite E4M3 value) and then to fp32.
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t pair16) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(pair16));
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

// Bulk copies into shared memory (16-byte multiples), counted by a barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count));
}

// 32 columns of the thread's lane, without the wait
__device__ __forceinline__ void tld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// the registers of a started load, not to be used before this
__device__ __forceinline__ void hold32(uint32_t (&r)[32]) {
  asm volatile(
      ""
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
        "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
        "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Products issued by a converged warp, in a branch that one elected lane takes.
// The instruction wants its operands in uniform registers.  When the compiler
// can tell that the warp's index, the tensor-memory address and the loop's
// bounds are uniform (they come from a shuffle) and that one lane is in the
// branch (elect.sync), a 128 x 128 x 16 product issues every 64 cycles, the tensor
// core's rate; from `lane == 0` in a branch on threadIdx it took 85 to 140.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
template <class T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
// D += A B as mma and mma_ta, for another instruction descriptor
__device__ __forceinline__ void mma_as(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ta_as(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
constexpr uint32_t kIdescScores = kIdesc & ~((7u << 7) | (7u << 10));   // A = B = f16
// The steps of an operand tile's descriptor: K-step kk (16 columns) of a K-major one.
__device__ __forceinline__ uint64_t desc_step(int kk) {
  return (uint64_t)((kk >> 2) * (kAtHalfBytes >> 4) + (kk & 3) * 2);
}

// Reconstruction of channels c0 .. c0+7 of the NR tokens tok0 .. tok0+NR-1
// (those below Nk) of cache `which` (0 = K, 1 = V) of head h: y = s*q + m
// (or s*(u - 2)), plus the centroids of stages T, ..., 1 in that order, each
// an fp32 add, then one rounding to bf16 -- the arithmetic of
// qvg_dequant_fused.  The results are fp32 values of the rounded bf16
// numbers (zero for tokens past the end).  In three steps, so that a thread
// can issue the loads of several blocks before it waits for any: the
// per-token codes, scale/zero bytes and assignments; the centroid rows they
// select (TT > 0, a fixed stage count of at most 4); the arithmetic.
template <int TT, int NR, class P>
struct ReconBlock {
  static constexpr int TR = TT > 0 ? TT : 1;
  int tok0, c0, which;
  uint32_t code[NR], sz[NR];
  int kk[NR][TR];
  uint4 rows[NR][TR];

  // the head's streams (the same for the whole CTA), then 32-bit offsets
  // within them (a block has fewer than 2^23 tokens)
  __device__ __forceinline__ void load_tokens(const P& p, int w, int h, int t0, int ch) {
    which = w; tok0 = t0; c0 = ch;
    const int ng = kD / p.G;
    const int64_t hN = (int64_t)h * p.Nk;
    const uint8_t* codes = p.codes[w] + hN * (kD / 4) + c0 / 4;
    const uint8_t* scl = p.scale[w] + hN * ng + c0 / p.G;
    const uint8_t* zr = p.zero[w] + hN * ng + c0 / p.G;
    const uint8_t* asg = p.assign[w] + hN;
    const int64_t asg_stage = (int64_t)p.H * p.Nk;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint32_t tok = (uint32_t)(tok0 + r < p.Nk ? tok0 + r : p.Nk - 1);   // past the end: a valid token, result unused
      code[r] = __ldg(reinterpret_cast<const unsigned short*>(codes + tok * (kD / 4)));
      sz[r] = (uint32_t)__ldg(scl + tok * (uint32_t)ng) | (p.sym ? 0u : ((uint32_t)__ldg(zr + tok * (uint32_t)ng) << 8));
#pragma unroll
      for (int t = 0; t < TR; ++t)
        if (TT > 0) kk[r][t] = min((int)__ldg(asg + t * asg_stage + tok), p.K - 1);
    }
  }
  // the per-token part of another block (loaded one step ahead)
  __device__ __forceinline__ void take_tokens(const ReconBlock& o) {
    which = o.which; tok0 = o.tok0; c0 = o.c0;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      code[r] = o.code[r];
      sz[r] = o.sz[r];
#pragma unroll
      for (int t = 0; t < TR; ++t) kk[r][t] = o.kk[r][t];
    }
  }
  __device__ __forceinline__ void load_rows(const P& p, int h) {
    if (TT <= 0) return;
    const __nv_bfloat16* tab = p.tab[which] + (int64_t)h * p.K * kD + c0;
    const int64_t tab_stage = (int64_t)p.H * p.K * kD;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int t = 0; t < TR; ++t)
        rows[r][t] = __ldg(reinterpret_cast<const uint4*>(tab + t * tab_stage + (uint32_t)kk[r][t] * kD));
  }
  __device__ __forceinline__ void finish(const P& p, const float2* nlut, int h, float (&y)[NR][8]) const {
    const int T = TT >= 0 ? TT : p.T;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      // y = s*q + m (or s*(u - 2)), exact in fp32, two channels per op through
      // the nibble table (which holds q, or u - 2 in the symmetric mode)
      const float2 sm = e4m3x2_to_f2(sz[r]);
      const float2 s2 = make_float2(sm.x, sm.x), m2 = make_float2(sm.y, sm.y);
      float2 y2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y2[e] = p.sym ? __fmul2_rn(s2, nlut[(code[r] >> (4 * e)) & 0xFu])
                      : __ffma2_rn(s2, nlut[(code[r] >> (4 * e)) & 0xFu], m2);
      auto add_row = [&](const uint4 w) {
        y2[0] = __fadd2_rn(y2[0], make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u)));
        y2[1] = __fadd2_rn(y2[1], make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)));
        y2[2] = __fadd2_rn(y2[2], make_float2(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u)));
        y2[3] = __fadd2_rn(y2[3], make_float2(__uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u)));
      };
      if (TT > 0) {
#pragma unroll
        for (int t = TR - 1; t >= 0; --t) add_row(rows[r][t]);
      } else if (TT < 0) {
        const uint32_t tok = (uint32_t)(tok0 + r < p.Nk ? tok0 + r : p.Nk - 1);
        const uint8_t* asg = p.assign[which] + (int64_t)h * p.Nk;
        const __nv_bfloat16* tab = p.tab[which] + (int64_t)h * p.K * kD + c0;
        for (int t = T - 1; t >= 0; --t) {
          const int k = min((int)__ldg(asg + t * (int64_t)p.H * p.Nk + tok), p.K - 1);
          add_row(__ldg(reinterpret_cast<const uint4*>(tab + t * (int64_t)p.H * p.K * kD + (uint32_t)k * kD)));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) { y[r][2 * e] = y2[e].x; y[r][2 * e + 1] = y2[e].y; }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t b = pack_bf16(y[r][e], y[r][e + 1]);
        y[r][e] = tok0 + r < p.Nk ? __uint_as_float(b << 16) : 0.0f;
        y[r][e + 1] = tok0 + r < p.Nk ? __uint_as_float(b & 0xFFFF0000u) : 0.0f;
      }
    }
  }
};

}  // namespace
}  // namespace qvg
