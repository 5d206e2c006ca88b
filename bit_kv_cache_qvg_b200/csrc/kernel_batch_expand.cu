// kernel_batch_expand.cu -- the tensor-core operands of qvg_attention_batch and
// qvg_attention_weights for many rows, written once for all of them.
//
// The attention kernels read a key tile once for every 256 rows.  With more
// rows than that, rebuilding it each time costs more than the products: a
// kernel that rebuilt the tiles on the fly, as qvg_attention does, took 2.58 ms
// for 1,520 rows over 38,000 tokens of 32 heads.  So a tile is rebuilt once,
// into the workspace, as the 32 KB image that a bulk copy brings into shared
// memory as it is: 128 keys x 128 channels (K in fp16, V in bf16), two halves of 64 channels,
// a key's 128 bytes of a half swizzled by key mod 8 (attention_tc.cuh).  K is
// the K-major operand of S = Q K'^T in this layout and V the N-major one of
// O = P V.  The rows are rotated once, too.
//
// The floor is the 512 bytes written a token: 95 us for 32 heads of 38,000
// tokens.  It takes 220 us (K = 256, T = 2, G = 64; 47 us for 12 heads of
// 14,040): the rebuilding (rebuild.cuh) keeps the issue slots, the ALU and the L1
// data path each a half busy, and the latency of the centroid rows does the
// rest.  So small CTAs, six to an SM: with one of 1,024 threads that keeps
// one head's tables in the SM's L1 and loads a step ahead it took 289 us.
#include "attention_tc.cuh"
#include "batch.cuh"
#include "rebuild.cuh"

namespace qvg {
namespace {

constexpr int kExThreads = 256;
constexpr int kExKeys = kExThreads / 8;           // keys per pass
constexpr int kExPasses = kAtTile / kExKeys;

// 128 rows of a head, or of one sequence, rotated at their positions; zeros
// behind the last one and for padding rows, whatever their queries hold: the
// sums by key take every row's scores, and 2^(x - inf) is 0 for a finite x only.
template <bool PRECISE>
__device__ __forceinline__ void expand_rows(const BatchParams& p, bool by_sequence, int hl, int b, int64_t tile) {
  const int which = by_sequence ? 1 : 0;
  const int64_t rows = by_sequence ? p.RB : p.R, pad = by_sequence ? p.RBp : p.Rp;
  const int64_t base = ((by_sequence ? (int64_t)b * p.Hn : 0) + hl) * 2 * pad;
  const int cb = threadIdx.x & 15;
#pragma unroll 2
  for (int i = 0; i < 128 * 16 / kExThreads; ++i) {
    const int64_t r = tile * 128 + (threadIdx.x >> 4) + i * (kExThreads / 16);
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (r < rows) {
      const int64_t row = by_sequence ? b * p.RB + r : r;
      const int64_t pos = query_pos(p, row);
      uint4 x = __ldg(reinterpret_cast<const uint4*>(p.Q + query_row(p, p.h0 + hl, row) * kD + 8 * cb));
      if (pos < 0) x = make_uint4(0, 0, 0, 0);
      turn_chunk<PRECISE>(p.rope + rope_row(p, pos) * (kD / 2) + 4 * cb, x, hi, lo);
    }
    const int64_t at = (base + (cb >> 3) * pad + r) * 128 + (((cb & 7) ^ (int)(r & 7)) << 4);
    *reinterpret_cast<uint4*>(p.row_img[which] + at) = hi;
    if (PRECISE) *reinterpret_cast<uint4*>(p.row_lo[which] + at) = lo;
  }
}

// One tile of K (rotated; PRECISE: and its low halves) or of V.
template <int TT, bool KEYS, bool PRECISE>
__device__ __forceinline__ void expand_tile(const BatchParams& p, uint8_t* smem, bool tail, int h, int b, int tile0, int n,
                                            uint8_t* img, uint8_t* img_lo) {
  float2* nlut = reinterpret_cast<float2*>(smem);
  uint32_t* turn = reinterpret_cast<uint32_t*>(nlut + 16);           // rows of the rotary table
  Tokens<TT, kAtTile>& tokens = *reinterpret_cast<Tokens<TT, kAtTile>*>(turn + kAtTile);
  constexpr int w = KEYS ? 0 : 1;
  // a thread per token: its bytes, or its position
  if (threadIdx.x < kAtTile) {
    const int key = min(tile0 + (int)threadIdx.x, n - 1);            // past the end: the last token, finite and not used
    if (!tail) {
      TokenBytes<TT> x;
      load_token<TT>(p, w, h, key, x);
      store_token<TT, kAtTile>(p, w, h, key, x, tokens, threadIdx.x);
    }
  } else if (KEYS) {
    const int at = threadIdx.x - kAtTile, key = min(tile0 + at, n - 1);
    turn[at] = (uint32_t)rope_row(p, raw_key_pos(p, tail, h, b, key));
  }
  if (!tail) {
    const int key = min(tile0 + (int)(threadIdx.x >> 1), n - 1);
    tokens.codes[threadIdx.x] = __ldg(reinterpret_cast<const uint4*>(p.codes[w] + ((int64_t)h * p.Nk + key) * (kD / 4)) + (threadIdx.x & 1));
    fill_nlut(p, nlut);
  }
  __syncthreads();
  const int c = threadIdx.x & 7, key0 = threadIdx.x >> 3;
  // a lane's place in the image does not depend on the pass: 32 keys on, the swizzle is the same
  const uint32_t place = (uint32_t)(key0 * 128 + ((c ^ (key0 & 7)) << 4));
  auto put = [&](int pass, uint4 (&x)[2]) {
    uint8_t* dst = img + place + pass * (kExKeys * 128);
    if (!KEYS) {
      *reinterpret_cast<uint4*>(dst) = x[0];
      *reinterpret_cast<uint4*>(dst + kAtHalfBytes) = x[1];
      return;
    }
    const float2* cs = p.rope + (int64_t)turn[pass * kExKeys + key0] * (kD / 2) + 4 * c;
    uint4 hi[2], lo[2];
    turn_chunk<PRECISE>(cs, x[0], hi[0], lo[0]);
    turn_chunk<PRECISE>(cs + 32, x[1], hi[1], lo[1]);
    *reinterpret_cast<uint4*>(dst) = hi[0];
    *reinterpret_cast<uint4*>(dst + kAtHalfBytes) = hi[1];
    if (PRECISE) {
      uint8_t* dl = img_lo + place + pass * (kExKeys * 128);
      *reinterpret_cast<uint4*>(dl) = lo[0];
      *reinterpret_cast<uint4*>(dl + kAtHalfBytes) = lo[1];
    }
  };
  if (!tail) {
    const Rebuild<TT, kAtTile> rebuild(p, w, h, c);
#pragma unroll 1
    for (int pass = 0; pass < kExPasses; ++pass) {
      uint4 x[2];
      rebuild(nlut, tokens, pass * kExKeys + key0, x);
      put(pass, x);
    }
  } else {
    // a tail's tokens are bf16 rows already; behind its length zeros
    const __nv_bfloat16* rows = p.tail[w] + ((int64_t)b * p.H + h) * p.Nt * kD + 8 * c;
#pragma unroll 1
    for (int pass = 0; pass < kExPasses; ++pass) {
      const int key = tile0 + pass * kExKeys + key0;
      uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (key < n) {
        const uint4* row = reinterpret_cast<const uint4*>(rows + (int64_t)key * kD);
        x[0] = __ldg(row);
        x[1] = __ldg(row + 8);
      }
      put(pass, x);
    }
  }
}

// CTAs: the prefix's tiles (K, then V unless PRECISE, of every key tile), the
// tails', the rows by head, the rows by sequence.  PRECISE: the second image
// of a tile holds the keys' low halves instead of the values.
template <int TT, bool PRECISE>
__global__ void __launch_bounds__(kExThreads, TT >= 0 && TT <= 2 ? 6 : 4) qvg_batch_expand(const BatchParams p, const uint32_t tiles_p, const uint32_t tiles_t,
                                                              const uint32_t row_tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kKinds = PRECISE ? 1 : 2;
  uint32_t id = blockIdx.x;
  if (id >= kKinds * (tiles_p + tiles_t)) {
    id -= kKinds * (tiles_p + tiles_t);
    const bool by_sequence = id >= row_tiles;
    if (by_sequence) id -= row_tiles;
    const uint32_t per = (uint32_t)(by_sequence ? p.RBp : p.Rp) / 128, unit = id / per;
    expand_rows<PRECISE>(p, by_sequence, (int)(unit % (uint32_t)p.Hn), (int)(unit / (uint32_t)p.Hn), id % per);
    return;
  }
  // all K tiles first, then all V tiles: neighbouring CTAs read the same tables
  const bool values = id >= tiles_p + tiles_t;
  if (values) id -= tiles_p + tiles_t;
  const bool tail = id >= tiles_p;
  if (tail) id -= tiles_p;
  const uint32_t nt = (uint32_t)(tail ? p.nt2 : p.nt1), unit = id / nt;
  const int j = (int)(id % nt), hl = (int)(unit % (uint32_t)p.Hn), b = (int)(unit / (uint32_t)p.Hn), h = p.h0 + hl;
  const int n = (int)(tail ? tail_length(p, b) : p.Nk);
  const int tile0 = j * kAtTile;
  if (tile0 >= n) return;                          // a tail's tile that nobody reads
  const int64_t at = (((tail ? (int64_t)b * p.Hn : 0) + hl) * nt + j) * kImageBytes;
  if (!values) expand_tile<TT, true, PRECISE>(p, smem, tail, h, b, tile0, n, p.key_img[tail] + at, p.val_img[tail] + at);
  else expand_tile<TT, false, false>(p, smem, tail, h, b, tile0, n, p.val_img[tail] + at, nullptr);
}

template <int TT>
cudaError_t expand_t(const BatchParams& p, bool precise, cudaStream_t s) {
  // the launch's key tiles and rows: none of a part that another kernel handles
  const int64_t tiles_p = p.S1 > 0 ? p.Hn * p.nt1 : 0, tiles_t = p.S2 > 0 ? p.B * p.Hn * p.nt2 : 0;
  const int64_t rows_h = p.S1 > 0 ? p.Hn * (p.Rp / 128) : 0, rows_s = p.S2 > 0 ? p.B * p.Hn * (p.RBp / 128) : 0;
  const unsigned grid = (unsigned)((precise ? 1 : 2) * (tiles_p + tiles_t) + rows_h + rows_s);
  const size_t smem = 16 * sizeof(float2) + kAtTile * sizeof(uint32_t) + Tokens<TT, kAtTile>::bytes(kD / p.G);
  const uint32_t np = (uint32_t)tiles_p, nt = (uint32_t)tiles_t, nr = (uint32_t)rows_h;
  if (precise) qvg_batch_expand<TT, true><<<grid, kExThreads, smem, s>>>(p, np, nt, nr);
  else qvg_batch_expand<TT, false><<<grid, kExThreads, smem, s>>>(p, np, nt, nr);
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
