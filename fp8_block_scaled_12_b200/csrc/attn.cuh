// attn.cuh -- attention of one new token per sequence over a paged FP8 key-value cache.
//
// For sequence b, query head h of key-value head c (G = Hq / Hkv heads share one), tokens t
// of the sequence (its length, its window and its valid pages decide which):
//   s_t = scale * sk_t * sum_d q_d dec(k_t[d])            p_t = exp(s_t - max s)
//   out = (sum_t p_t sv_t dec(v_t)) / sum_t p_t
// What bounds it: the cache is read once per chunk of up to 16 query heads of a kv head (8 with
// more than 128 channels), 2 D + 8 bytes a token and kv head, against 4 D G flops, so HBM does up
// to about a hundred heads per kv head.  The kernel is built so that no code byte is ever
// converted: both products run on the FP8 tensor cores straight from the tiles TMA has put into
// shared memory.
//   scores   S^T[128 tokens x heads] = K-tile (A, 128 x D) . q^T.  A bf16 q (8 significant
//            bits) is split into two E4M3 pieces q = (hi + lo / 16) 2^-e, 4 bits each with
//            e from the head's largest |q|: exact for every element above 2^-14 of the
//            largest and off by at most 2^-21 of the largest below that.  The pieces are
//            2 x heads columns of B; tensor memory then holds one token per lane, so the
//            token's scale is one register.
//   softmax  per tile: with 2^e_t > sv_t and E the tile's largest e_t, the maximum Y of
//            s_t + e_t - E over the 128 tokens (in powers of two; one redux per warp and head,
//            one exchange through shared memory), p = 2^(s - Y), and w = p sv 2^(8 - E), whose
//            largest then lies in [2^7, 2^8) for every head, whichever token it is.
//   output   O^T[D x heads] = V-tile^T (A, read "transposed" as stored: D contiguous) . w.
//            w is split into four E4M3 pieces w = c0 + c1/16 + c2/256 + c3/4096: off by at
//            most 2^-17 relative, or 2^-29 of the head's largest w of the tile.  (With p taken
//            from the largest score instead, w would be held to 2^-30 of the tile's largest sv:
//            a large scale with hardly any probability would cost the other tokens their bits.
//            The addition before the maximum costs 2.5 of 70 us with 16 heads a tile, nothing that
//            shows with 4 or 8.)
//            Each tile's product lands in fresh tensor-memory columns and is folded into fp32
//            registers (one channel d per thread) with the running maximum's factors.
// A CTA (one per SM): two warpgroups (warps 4-11) do softmax and accumulation, each working
// through a range of tiles of its own, for which one warp loads pages (TMA; one lane per box of
// gcd(page, 128) rows) and scales and another issues the MMAs.  K and V of a tile are halves that
// take slots of the warpgroup's own ring, K's free after the scores, V's after the outputs: the
// warpgroups never wait for one another.
//
// Split: the batch's tiles, row after row (a row is a sequence, kv head and chunk of GT query
// heads), form one list that is cut into ranges of equal cost, one per warpgroup ("worker"),
// whatever the lengths.  A row inside one range is finished there; a row cut by a border leaves
// partial sums (o, m, l) in the workspace, which k_attn_join adds up in the order of the tiles,
// so results do not depend on timing.
//
// Measured (32 query and 8 kv heads of 128, e4m3, ragged lengths; bytes of the cache over time,
// both kernels, replayed from a graph): 64 sequences of up to 24000 tokens in pages of 32,
// 1.63 GB, 247 us, 6.6 TB/s, the speed of a copy; 32 of up to 8192 in pages of 16, 286 MB, 54 us,
// 5.2 TB/s (~4 us until the first tiles are there, ~5 us for the join and its launch); 131071 +
// 50070 tokens of 64 / 8 heads, token-major, 383 MB, 77 us, 4.9 TB/s (rows of 128 bytes 1 KB
// apart; head-major pages 67 us).  With the two warpgroups on alternate tiles of one range and
// one ring the first two took 318 and 83 us, with one warpgroup 396 and 113.
//
// Masked tokens (beyond the length, before the window, or of a page id outside the cache):
// boxes without any valid token are zero-filled by TMA (an out-of-range page coordinate: no
// memory is read), rows of V that are masked inside a loaded box are zeroed in shared memory,
// their scales are not used, their scores are -inf.  Whatever bytes they hold never matter.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace fp8lin {

constexpr int kAttnThreads = 384;
constexpr int kAttnTile = 128;
// Tiles whose scales are held: a K-slot is filled for tile j only after the outputs of tile j - 4
// (or a later one) have left a V-slot, whatever the ring's length.
constexpr int kScaleRing = 4;
// Binades by which value scales of a tile may differ before the smaller ones count as this far
// from the largest.  Sums of p reach 2^kScaleSpread times the number of tokens (a token with
// nearly all of the probability and the smallest scale), which fp32 has to hold: a tile whose
// reference lies 2^126 below another's adds nothing, and it is at most 2^(kScaleSpread - 126) of
// the sum.  (Scales that count with their own exponent, without the tile's largest, would move
// the references of two tiles apart by twice the span and lose such a tile.)
constexpr int kScaleSpread = 90;
// Register split of the variant with 16 heads (the pool is kLaunchRegs a thread).
constexpr uint32_t kAttnLoadRegs = 88, kAttnSoftmaxRegs = 208;
static_assert(128 * kAttnLoadRegs + 256 * kAttnSoftmaxRegs <= 384 * kLaunchRegs, "register split exceeds pool");
static_assert(kAttnThreads == 384, "the split is of 384 threads");

struct AttnArgs {
  const uint16_t* q;       // bf16 [B][Hq][D], strides below
  const float* ks;         // [pages][H][P]
  const float* vs;
  const int32_t* table;    // [B][max_pages], row stride table_stride
  const int32_t* lens;     // [B]
  uint16_t* out;           // bf16 [B][Hq][D]
  float* lse;              // [B][Hq] or nullptr
  float* ws_o;             // [2 * workers][GT][D]: a worker's first and last segment
  float* ws_ml;            // [2 * workers][2][GT]
  int2* ws_join;           // rows to join: (row, slot of its first partial << 16 | worker of its last), or
                           // (-1, -1); [rows] by row or [workers] by the worker in which the row begins
  int64_t q_row, q_head, table_stride;
  int64_t window, cap;     // tokens; window 0 = none; cap = max_pages * P
  int64_t pages;
  float scale;
  int B, H, G, HC, D, P, BR;   // HC chunks of query heads per kv head; BR rows per box
  int slots;               // partial sums that the workspace holds
  int by_row;              // how ws_join is ordered
};

template <int GT_, int DCH_>
struct AttnCfg {
  static constexpr int GT = GT_, DCH = DCH_;
  static constexpr uint32_t KV_BYTES = kAttnTile * 128 * DCH;   // of K or V of one tile: a slot
  // Slots of each warpgroup's ring.  More in flight do not help: with 6 of 16 KB the requests
  // disturb one another (8 sequences of up to 64000 tokens: 108 us; 103 us with 5, 101 us with 4,
  // 105 us with 3), with fewer the loads show as soon as the clock drops (64 sequences of up to
  // 24000 tokens back to back for 80 ms: 252 us with 5, 258 us with 4, 280 us with 3).
  static constexpr int SLOTS = DCH == 2 ? 3 : 5;
  static constexpr uint32_t Q_ROWS = GT == 4 ? 16 : 2 * GT;    // two pieces; at least the MMA's smallest N
  static constexpr uint32_t Q_BYTES = Q_ROWS * 128 * DCH;
  static constexpr uint32_t P_ROW = 4 * GT;                  // bytes per token of the split weights
  static constexpr uint32_t P_BYTES = kAttnTile * P_ROW;
  static constexpr uint32_t OFF_Q = 2 * SLOTS * KV_BYTES;
  static constexpr uint32_t OFF_P = OFF_Q + 4 * Q_BYTES;     // queries: two buffers a warpgroup
  static constexpr uint32_t OFF_S = OFF_P + 2 * P_BYTES;     // scales: [warpgroup][kScaleRing][2][128] fp32
  static constexpr uint32_t OFF_STATE = OFF_S + 2 * kScaleRing * 1024;
  static constexpr uint32_t S_COLS = Q_ROWS, O_COLS = 4 * GT;
  static constexpr uint32_t TMEM_USED = 2 * (2 * S_COLS + DCH * O_COLS);     // two score buffers a warpgroup
  static constexpr uint32_t TMEM_COLS = TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : 256;
};

// What a warpgroup has to know of the batch.
struct AttnRange {
  int tiles;                 // of the batch
  int b, off, count;         // its first tile: sequence and place among its tiles; how many it takes
};

template <int GT, int SLOTS>
struct alignas(16) AttnState {            // arrays [2]: by warpgroup
  float red[2][2][4][GT];  // [parity of its tile]: per-warp maxima
  float lsum[2][4][GT];    // per-warp sums of p
  float cq[2][2][GT];      // per-head factor of the staged queries
  uint64_t full[2][SLOTS];
  uint64_t empty[2][SLOTS];
  uint64_t scales[2][kScaleRing];
  uint64_t qfull[2][2];    // [buffer]
  uint64_t sfull[2][2];    // [parity of its tile]
  uint64_t pfull[2], ofull[2];
  uint64_t meet[2];        // the warpgroup's warps
  uint64_t drain[2];
  uint32_t boxes[2][kScaleRing];           // which boxes of the tile hold a valid page
  int seg[2][kScaleRing];                  // its segment of the worker's range
  uint32_t tmem_base;
  int abort;
  AttnRange range[2];
};

template <class C>
constexpr size_t attn_smem_bytes() {
  return 1024 + C::OFF_STATE + sizeof(AttnState<C::GT, C::SLOTS>);
}

// Tokens [st, len) of a sequence, and its tiles [ft, ft + n): at least one, so that an empty
// row is written too.
struct AttnSeq {
  int len, st, ft, n;
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  AttnSeq s;
  const int64_t l = min(int64_t(max(__ldg(a.lens + b), 0)), a.cap);
  s.len = int(l);
  s.st = a.window > 0 && l > a.window ? int(l - a.window) : 0;
  s.ft = s.st / kAttnTile;
  s.n = max(1, (s.len + kAttnTile - 1) / kAttnTile - s.ft);
  return s;
}

// The ranges of the list of tiles.  Where a worker has several tiles to take, each row counts
// kAttnRowCost tiles more than it has, which stand before its first, for its queries, sums and
// outputs (with equal tiles the workers of many short rows ended up
// to 8 of 47 us after the others in a batch of 32 ragged sequences: 59 us in all, 57 us counting
// one, 55.6 us two or three; 8 rows of 8 tiles, one a worker, take 8.0 us without and 9.1 us
// with the extra). Worker k of n takes [total k / n, total (k + 1) / n) of this list.  Workers
// of one CTA are grid.x apart, so few tiles spread over the SMs first.
constexpr int kAttnRowCost = 2;
struct AttnPlan {
  int tiles, workers, cost, total;
  __device__ __forceinline__ AttnPlan(int tiles_, int rows) : tiles(tiles_) {
    workers = min(2 * int(gridDim.x), tiles);
    cost = tiles >= 4 * workers ? kAttnRowCost : 0;
    total = tiles + cost * rows;
  }
  __device__ __forceinline__ int begin(int k) const { return int(int64_t(total) * min(k, workers) / workers); }
  __device__ __forceinline__ int worker(int wg) const { return int(blockIdx.x) + wg * int(gridDim.x); }
};

// The walk over a worker's range, tile by tile (next_tile) or segment by segment (a segment:
// the part of one row inside the range).  Every role walks the same sequence.
struct AttnWalk {
  int b, c, hc;              // the row: sequence, kv head, chunk of query heads
  int t, t1, left;           // tiles [t, t1) of the segment are still to come, `left` after it
  AttnSeq s;
  __device__ __forceinline__ void start(const AttnArgs& a, int first_b, int off, int count) {
    b = first_b;
    s = attn_seq(a, b);
    const int rr = off / s.n;
    c = rr / a.HC;
    hc = rr - c * a.HC;
    t = off - rr * s.n;
    t1 = min(s.n, t + count);
    left = count - (t1 - t);
  }
  __device__ __forceinline__ bool next_segment(const AttnArgs& a) {
    if (left <= 0) return false;
    if (++hc == a.HC) {
      hc = 0;
      if (++c == a.H) {
        c = 0;
        s = attn_seq(a, ++b);
      }
    }
    t = 0;
    t1 = min(s.n, left);
    left -= t1;
    return true;
  }
  // to the next tile; true if it begins another segment
  __device__ __forceinline__ bool next_tile(const AttnArgs& a) { return ++t == t1 && next_segment(a); }
};

// Sums over the warp of N values a lane, N a power of two: in each step a lane passes half of
// them on and adds what it gets to the other half.  Lane i returns the sum of value
// i / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  float r = v[0];
  int d = 16;
  if constexpr (N > 1) {
    float h[N / 2];
    const bool up = (lane & 16) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      h[i] = (up ? v[N / 2 + i] : v[i]) + __shfl_xor_sync(~0u, up ? v[i] : v[N / 2 + i], 16);
    // the same with the next lower bit of the lane in the place of this one
    int n = N / 2;
    for (d = 8; n > 1; d >>= 1) {
      n >>= 1;
      const bool u = (lane & d) != 0;
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        if (i < n) h[i] = (u ? h[n + i] : h[i]) + __shfl_xor_sync(~0u, u ? h[i] : h[n + i], d);
    }
    r = h[0];
  }
  for (; d > 0; d >>= 1) r += __shfl_xor_sync(~0u, r, d);
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// ln(l 2^m), -infinity for l = 0.  l's exponent joins m first: l may be far from 1 and m as far on
// the other side, and a logarithm of all of l would be off by its last place there.
__device__ __forceinline__ float log_sum(float m, float l) {
  if (l == 0.0f) return -INFINITY;
  if (!(l < INFINITY)) return l + m;
  const uint32_t b = __float_as_uint(l);
  return ((m + float(int(b >> 23) - 127)) + __log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u))) *
         0.69314718055994530942f;
}
// Arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Shared-memory descriptors.  K-major operands have rows of 128 bytes (the layout of
// sw128_kmajor_desc); MN-major ones have rows along K that hold `row` bytes of the whole M or N,
// written with the swizzle of that width (none for 16).  Either way 8-row groups are row * 8
// bytes apart: the stride offset, or, without a swizzle, the leading one, which nothing else
// uses here.  The low word holds the address in units of 16 bytes, so that steps are additions
// of constants to it.
__device__ __forceinline__ uint32_t attn_desc_lo(uint32_t addr, uint32_t row = 128) {
  return (addr >> 4) | ((row == 16 ? (row * 8) >> 4 : 1u) << 16);
}
__device__ __forceinline__ uint64_t attn_desc(uint32_t lo, uint32_t row) {
  const uint32_t layout = row == 128 ? 2u : row == 64 ? 4u : row == 32 ? 6u : 0u;    // 128-, 64-, 32-byte swizzle
  const uint32_t hi = ((row * 8) >> 4) | (1u << 14) | (layout << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// Columns of tensor memory, N a thread.  The loads are for whole warps (.sync.aligned), so lanes
// that a mask or a wait has parted meet first.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, uint32_t (&r)[N]) {
  __syncwarp();
  if constexpr (N == 8) {
    tmem_ld8(taddr, r);
  } else if constexpr (N == 16) {
    tmem_ld16(taddr, r);
  } else if constexpr (N == 32) {
    tmem_ld32(taddr, r);
  } else {
    static_assert(N == 64, "columns a thread loads");
    tmem_ld32(taddr, reinterpret_cast<uint32_t(&)[32]>(r[0]));
    tmem_ld32(taddr + 32, reinterpret_cast<uint32_t(&)[32]>(r[32]));
  }
  tmem_ld_wait();
  tmem_regs_ready(r);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Instruction descriptor with A in the cache's format (0 E4M3, 1 E5M2), B E4M3; `mn`: both
// operands MN-major.
__device__ __forceinline__ constexpr uint32_t attn_idesc(int fmt, uint32_t n, bool mn) {
  return idesc_f8_e4m3_f32(128, n) | (uint32_t(fmt) << 7) | (mn ? (3u << 15) : 0u);
}

// fp32 pair -> two E4M3 codes, and what they leave, times 16 (exact), in its place.
__device__ __forceinline__ uint32_t code2(uint64_t v) {
  const float2 f = unpack2(v);
  return cvt2<kE4M3>(f.x, f.y);
}
__device__ __forceinline__ uint32_t split16(uint64_t& v) {
  const uint32_t c = code2(v);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(c)));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  v = fma2(pack2(f.x, f.y), pack2(-16.0f, -16.0f), mul2(v, pack2(16.0f, 16.0f)));
  return c;
}

// Scan of the batch by one warp: the list's length, then the tiles at both ends of the range.
// The first pass has its loads in flight together and one sum at the end; the second takes 32
// sequences at a time and looks inside only where the range begins or ends.  (512 sequences of up
// to 1000 tokens: 118 us; 127 us with a sum and a full look at every 32, the loads one by one.)
__device__ __forceinline__ void attn_scan(const AttnArgs& a, int lane, int wg, AttnRange* out) {
  const int rows = a.H * a.HC;
  int tiles = 0;
#pragma unroll 8
  for (int i = lane; i < a.B; i += 32) tiles += attn_seq(a, i).n;
  tiles = __reduce_add_sync(~0u, tiles) * rows;
  const AttnPlan plan(tiles, a.B * rows);
  const int k = plan.worker(wg), x0 = plan.begin(k), x1 = plan.begin(k + 1);
  int run = 0;                                             // tiles of the sequences before these 32
  int first = 0, last = 0;                                 // numbers of the range's first tile and the next range's
  if (lane == 0) {
    out->tiles = tiles;
    out->b = out->off = out->count = 0;
  }
  for (int i = 0; x0 < x1 && i < a.B; i += 32) {
    const int n = i + lane < a.B ? attn_seq(a, i + lane).n : 0;
    const int all = __reduce_add_sync(~0u, n) * rows;
    const int e0 = run + plan.cost * i * rows;             // their entries of the list: [e0, e1)
    const int e1 = e0 + all + plan.cost * min(32, a.B - i) * rows;
    if ((x0 >= e0 && x0 < e1) || (x1 >= e0 && x1 < e1)) {
      int inc = n * rows;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += y;
      }
      const int before = run + inc - n * rows;             // tiles and list entries before this sequence
      const int entry = before + plan.cost * (i + lane) * rows, per = n + plan.cost;
      auto locate = [&](int x) {                           // place of list entry x among this sequence's tiles
        const int row = (x - entry) / per;
        return row * n + max(0, x - entry - row * per - plan.cost);
      };
      const bool has0 = n > 0 && x0 >= entry && x0 < entry + rows * per;
      const bool has1 = n > 0 && x1 >= entry && x1 < entry + rows * per;
      if (has0) {
        out->b = i + lane;
        out->off = locate(x0);
      }
      first += __reduce_add_sync(~0u, has0 ? before + locate(x0) : 0);
      last += __reduce_add_sync(~0u, has1 ? before + locate(x1) : 0);
      if (x1 < e1) break;
    }
    run += all;
  }
  __syncwarp();
  if (lane == 0 && x0 < x1) out->count = (x1 == plan.total ? tiles : last) - first;
}

// Queries of a segment -> two E4M3 pieces as K-major rows (hi: head g, lo: head GT + g) in
// shared memory, and the factor that turns their products into base-2 exponents.  A thread
// owns 4, 8 or 16 channels of a head; loading and storing are apart, so that a tile's work hides
// the loads' latency.
template <class C>
struct AttnQuery {
  static constexpr int UNIT = C::GT * C::DCH;                // 128 threads share GT heads of 128 DCH channels
  static constexpr int UPH = 128 * C::DCH / UNIT;            // units per head
  static_assert(C::GT * UPH == 128 && (UNIT == 4 || UNIT == 8 || UNIT == 16), "one unit a thread");
  uint32_t x[UNIT / 2];
  __device__ __forceinline__ void load(const AttnArgs& a, const AttnWalk& w, int tid) {
    const int g = w.hc * C::GT + tid / UPH, ch = tid % UPH * UNIT;
#pragma unroll
    for (int i = 0; i < UNIT / 2; ++i) x[i] = 0u;
    if (g < a.G && ch < a.D) {
      const uint16_t* p = a.q + int64_t(w.b) * a.q_row + int64_t(w.c * a.G + g) * a.q_head + ch;
      if constexpr (UNIT == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        x[0] = v.x;
        x[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < UNIT / 8; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
          x[4 * i] = v.x;
          x[4 * i + 1] = v.y;
          x[4 * i + 2] = v.z;
          x[4 * i + 3] = v.w;
        }
      }
    }
  }
  __device__ __forceinline__ void store(const AttnArgs& a, uint8_t* sq, float* cq, int tid) const {
    const int head = tid / UPH, ch = tid % UPH * UNIT;
    uint32_t mx = 0;                         // largest |q| as bf16 bits: NaN and Inf sort above all
#pragma unroll
    for (int i = 0; i < UNIT / 2; ++i) mx = max(mx, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int d = 1; d < UPH; d <<= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, d));
    const bool bad = mx >= 0x7F80u;          // a NaN or infinity: the head's output is NaN
    const int e = min(7 - (int(mx >> 7) - 127), 126);       // q 2^e in [128, 256)
    const float up = __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
    uint32_t hi[UNIT / 4], lo[UNIT / 4];
#pragma unroll
    for (int i = 0; i < UNIT / 4; ++i) {
      uint64_t p0 = mul2(pack2(bf16_lo(x[2 * i]), bf16_hi(x[2 * i])), pack2(up, up));
      uint64_t p1 = mul2(pack2(bf16_lo(x[2 * i + 1]), bf16_hi(x[2 * i + 1])), pack2(up, up));
      const uint32_t h0 = split16(p0), h1 = split16(p1);
      hi[i] = bad ? 0x7F7F7F7Fu : h0 | (h1 << 16);
      lo[i] = bad ? 0x7F7F7F7Fu : code2(p0) | (code2(p1) << 16);
    }
    // rows of 128 bytes with the 128-byte swizzle
    uint8_t* chunk = sq + (ch >> 7) * (C::Q_ROWS * 128) + (ch & 15);
    const int c16 = (ch >> 4) & 7, low = C::GT + head;
    uint8_t* at = chunk + head * 128 + ((c16 ^ (head & 7)) * 16);
    uint8_t* at_lo = chunk + low * 128 + ((c16 ^ (low & 7)) * 16);
    if constexpr (UNIT == 4) {
      *reinterpret_cast<uint32_t*>(at) = hi[0];
      *reinterpret_cast<uint32_t*>(at_lo) = lo[0];
    } else if constexpr (UNIT == 8) {
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(at_lo) = make_uint2(lo[0], lo[1]);
    } else {
      *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(at_lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (ch == 0) cq[head] = a.scale * 1.44269504088896340736f / up;
  }
};

// A wait by a whole warp, with mbar_wait's bounds.  Every branch in it is taken by all lanes or
// none: a wait that lanes leave one by one, or that some of them skip (those of unmasked tokens,
// say), can leave the warp in parts, and a part that reaches a barrier counts as the warp -- the
// barrier then lets the other warps go without the rest, whose own wait there never ends.
// The limit is read once per kernel and the clock only now and then: either costs more than
// most of the waits.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; i < FP8LIN_WAIT_ITERS && limit_ns >= 1000; ++i) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    if ((i & 31u) == 0u) {
      if (__any_sync(~0u, *abort != 0)) return false;
      const uint64_t now = __shfl_sync(~0u, globaltimer_ns(), 0);
      if (since == 0) since = now;
      if (now - since > limit_ns) break;
    }
  }
  if ((threadIdx.x & 31) == 0) {
    *abort = 1;
    atomicOr(&g_device_error, 1u);
  }
  __syncwarp();
  return false;
}

// Meeting of a warpgroup's four warps on an mbarrier (bounded, unlike a hardware barrier): what
// they wrote to shared memory before it is visible after it.  False if a warp has given up.
__device__ __forceinline__ bool attn_meet(uint32_t bar, int& turn, bool ok, volatile int* abort, uint64_t limit_ns) {
  __syncwarp();
  if (ok && (threadIdx.x & 31) == 0) mbar_arrive(bar);
  return attn_wait(bar, uint32_t(turn++) & 1u, abort, limit_ns) && ok;
}

template <int FMT, class C>
__global__ void __launch_bounds__(kAttnThreads, 1)
    k_paged_attention(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const AttnArgs a) {
  constexpr int GT = C::GT, NP = GT / 2, DCH = C::DCH, SLOTS = C::SLOTS;
  using State = AttnState<GT, SLOTS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  State* ps = reinterpret_cast<State*>(gbase + C::OFF_STATE);
  volatile int* abort = &ps->abort;
  const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_wait_limit_ns);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < SLOTS; ++s) {
        mbar_init(smem_u32(&ps->full[i][s]), 1);
        mbar_init(smem_u32(&ps->empty[i][s]), 1);
      }
      for (int s = 0; s < kScaleRing; ++s) mbar_init(smem_u32(&ps->scales[i][s]), 1 + 32);   // `boxes`, copies
      for (int s = 0; s < 2; ++s) {
        mbar_init(smem_u32(&ps->qfull[i][s]), 4);
        mbar_init(smem_u32(&ps->sfull[i][s]), 1);
      }
      mbar_init(smem_u32(&ps->pfull[i]), 4);
      mbar_init(smem_u32(&ps->ofull[i]), 1);
      mbar_init(smem_u32(&ps->meet[i]), 4);
      mbar_init(smem_u32(&ps->drain[i]), 1);
    }
    ps->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ps->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 2 || warp == 3) attn_scan(a, lane, warp - 2, &ps->range[warp - 2]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ps->tmem_base;                 // scores of both warpgroups, then outputs
  int u = 0;                                           // loaders: half tiles (K, then V) given a slot
  // (8 heads fit the registers of an even split)
  if (warp < 4) {
    if constexpr (GT > 8) setmaxnreg_dec<kAttnLoadRegs>();
    const int g = warp & 1, n = ps->range[g].count;      // the warpgroup it works for
    const uint32_t ring = base + uint32_t(g * SLOTS) * C::KV_BYTES;
    if (warp < 2) {
      // ------------------------------------------------ pages and scales -> shared memory
      // a lane owns a box of the tile and the scales of four tokens (rows of a box come in
      // multiples of eight)
      if (n > 0) {
        AttnWalk w;
        w.start(a, ps->range[g].b, ps->range[g].off, n);
        const int nb = kAttnTile / a.BR;
        const int sbox = lane * 4 / a.BR, srow = lane * 4 - sbox * a.BR;
        const int step_p = kAttnTile / a.P, step_r = kAttnTile - step_p * a.P;   // a tile further in pages and rows
        int seg = 0, h, tok, pi, row, page;
        const int32_t* trow;
        auto lookup = [&]() {              // the page of this lane's box, -1 if none of its tokens counts
          page = -1;
          if (lane < nb && tok < w.s.len && tok + a.BR > w.s.st) page = __ldg(trow + pi);
        };
        auto enter = [&]() {               // a segment's first tile
          h = w.c;
          tok = (w.s.ft + w.t) * kAttnTile + lane * a.BR;
          pi = tok / a.P;
          row = tok - pi * a.P;
          trow = a.table + int64_t(w.b) * a.table_stride;
          lookup();
        };
        enter();
        for (int j = 0; j < n; ++j) {
          const int pg = page, rw = row, ch = h, sg = seg;
          if (j + 1 < n) {
            if (w.next_tile(a)) {
              ++seg;
              enter();
            } else {
              tok += kAttnTile;
              pi += step_p;
              row += step_r;
              if (row >= a.P) {
                row -= a.P;
                ++pi;
              }
              lookup();
            }
          }
          const bool ok = pg >= 0 && pg < a.pages;
          const int pc = ok ? pg : int(a.pages);
          const uint32_t boxes = __ballot_sync(~0u, ok);
          const int64_t spage = __shfl_sync(~0u, pg, sbox);
          const int sr = __shfl_sync(~0u, rw, sbox) + srow;
          int s = u % SLOTS;
          if (!attn_wait(smem_u32(&ps->empty[g][s]), ((u / SLOTS) & 1u) ^ 1u, abort, limit)) break;
          const int e = j % kScaleRing;
          if (lane == 0) {
            ps->boxes[g][e] = boxes;
            ps->seg[g][e] = sg;
            mbar_arrive(smem_u32(&ps->scales[g][e]));
            mbar_arrive_expect_tx(smem_u32(&ps->full[g][s]), C::KV_BYTES);
          }
          __syncwarp();
          if (lane < nb) {
#pragma unroll
            for (int c = 0; c < DCH; ++c)
              tma_load_4d(ring + s * C::KV_BYTES + c * (kAttnTile * 128) + uint32_t(lane * a.BR) * 128u, &tmK,
                          smem_u32(&ps->full[g][s]), c * 128, rw, ch, pc);
          }
          if ((boxes >> sbox) & 1u) {
            const int64_t at = (spage * a.H + ch) * a.P + sr;
            const uint32_t sc = base + C::OFF_S + (g * kScaleRing + e) * 1024 + lane * 16;
            cp_async16(sc, a.ks + at);
            cp_async16(sc + 512, a.vs + at);
          }
          cp_async_arrive(smem_u32(&ps->scales[g][e]));
          ++u;
          s = u % SLOTS;
          if (!attn_wait(smem_u32(&ps->empty[g][s]), ((u / SLOTS) & 1u) ^ 1u, abort, limit)) break;
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&ps->full[g][s]), C::KV_BYTES);
          __syncwarp();
          if (lane < nb) {
#pragma unroll
            for (int c = 0; c < DCH; ++c)
              tma_load_4d(ring + s * C::KV_BYTES + c * (kAttnTile * 128) + uint32_t(lane * a.BR) * 128u, &tmV,
                          smem_u32(&ps->full[g][s]), c * 128, rw, ch, pc);
          }
          ++u;
        }
      }
      if (warp == 0) pdl_trigger();
    } else {
      // ------------------------------------------------ MMAs
      // the whole warp walks, one elected lane issues: operands then stay in uniform registers
      constexpr uint32_t id_s = attn_idesc(FMT, C::Q_ROWS, false), id_o = attn_idesc(FMT, 4 * GT, true);
      const int steps = (a.D + 31) / 32;
      const uint32_t rlo = attn_desc_lo(ring);
      const uint32_t qlo = attn_desc_lo(base + C::OFF_Q + 2 * g * C::Q_BYTES);
      const uint32_t plo = attn_desc_lo(base + C::OFF_P + g * C::P_BYTES, C::P_ROW);
      const uint32_t tmem_s = tmem + 2 * g * C::S_COLS, tmem_o = tmem + 4 * C::S_COLS + g * (DCH * C::O_COLS);
      // Whichever product's operands are there goes first: in tile order, outputs whose weights
      // are ready would wait for a later tile's K and keep V's slot meanwhile.  Scores run up to
      // two tiles ahead of the outputs: the scores of tile j - 2 were read before its weights
      // were announced.
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(~0u, mbar_test_wait(smem_u32(bar), parity)) != 0;
      };
      bool ok = true;
      uint32_t polls = 0;
      uint64_t since = 0;
      for (int js = 0, jo = 0; jo < n;) {
        if (js < n && js <= jo + 1) {
          const int u = 2 * js, s = u % SLOTS, par = js & 1;
          if (ready(&ps->full[g][s], (u / SLOTS) & 1u)) {
            const int seg = ps->seg[g][js % kScaleRing];
            if (ready(&ps->qfull[g][seg & 1], (seg >> 1) & 1u)) {
              tc_fence_after();
              if (elect_one()) {
                const uint32_t k0 = rlo + uint32_t(s) * (C::KV_BYTES / 16);
                const uint32_t q0 = qlo + uint32_t(seg & 1) * (C::Q_BYTES / 16);
#pragma unroll
                for (int k = 0; k < 4 * DCH; ++k)
                  if (k < steps)
                    mma_f8(tmem_s + par * C::S_COLS, attn_desc(k0 + (k / 4) * (kAttnTile * 8) + (k % 4) * 2, 128),
                           attn_desc(q0 + (k / 4) * (C::Q_ROWS * 8) + (k % 4) * 2, 128), id_s, k > 0 ? 1u : 0u);
                mma_commit(smem_u32(&ps->sfull[g][par]));
                mma_commit(smem_u32(&ps->empty[g][s]));
              }
              __syncwarp();
              ++js;
              polls = 0;
            }
          }
        }
        if (jo < js && ready(&ps->pfull[g], jo & 1u)) {
          const int u = 2 * jo + 1, s = u % SLOTS;
          if (ready(&ps->full[g][s], (u / SLOTS) & 1u)) {
            tc_fence_after();
            if (elect_one()) {
              const uint32_t v0 = rlo + uint32_t(s) * (C::KV_BYTES / 16);
#pragma unroll
              for (int c = 0; c < DCH; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_f8(tmem_o + c * C::O_COLS, attn_desc(v0 + c * (kAttnTile * 8) + k * (32 * 8), 128),
                         attn_desc(plo + k * (2 * C::P_ROW), C::P_ROW), id_o, k > 0 ? 1u : 0u);
              mma_commit(smem_u32(&ps->ofull[g]));
              mma_commit(smem_u32(&ps->empty[g][s]));
            }
            __syncwarp();
            ++jo;
            polls = 0;
          }
        }
        // the wait's bounds, as in mbar_wait
        if ((++polls & 63u) == 0u || (limit < 1000 && polls > 1)) {
          const uint64_t now = globaltimer_ns();
          if (polls <= 64u) since = now;
          const bool out = limit < 1000 || now - since > limit || polls > FP8LIN_WAIT_ITERS;
          if (out && lane == 0) {
            *abort = 1;
            atomicOr(&g_device_error, 1u);
          }
          ok = !__any_sync(~0u, out || *abort);
          if (!ok) break;
        }
      }
      for (int u = max(0, 2 * n - 2); ok && u < 2 * n; ++u)       // the last commits have arrived
        ok = attn_wait(smem_u32(&ps->empty[g][u % SLOTS]), (u / SLOTS) & 1u, abort, limit);
    }
  } else {
    if constexpr (GT > 8) setmaxnreg_inc<kAttnSoftmaxRegs>();
    const int wg = (warp - 4) >> 2;
    const int mine = ps->range[wg].count;
    if (!a.by_row && (threadIdx.x & 127) == 0)               // until a row begins here that ends elsewhere
      a.ws_join[int(blockIdx.x) + wg * int(gridDim.x)] = make_int2(-1, -1);
    if (mine > 0) {
      // ------------------------------------------------ softmax and accumulation
      const int quad = warp & 3;                   // tensor-memory lanes of this warp
      const int tok = quad * 32 + lane;            // token of the tile; channel of the output
      const uint32_t all_boxes = (2u << (kAttnTile / a.BR - 1)) - 1u;
      const int box4 = 4 * lane / a.BR;            // the box of tokens 4 lane .. 4 lane + 3
      const uint32_t tlane = uint32_t(quad * 32) << 16;
      const uint32_t tmem_s = tmem + tlane + 2 * wg * C::S_COLS;
      const uint32_t tmem_o = tmem + tlane + 4 * C::S_COLS + wg * (DCH * C::O_COLS);
      const AttnPlan plan(ps->range[wg].tiles, a.B * a.H * a.HC);
      const int worker = plan.worker(wg);
      AttnWalk w;
      w.start(a, ps->range[wg].b, ps->range[wg].off, mine);
      AttnWalk ahead = w;                          // the next segment whose queries are staged
      AttnQuery<C> qn;
      auto stage = [&](int buf) {
        qn.store(a, gbase + C::OFF_Q + (2 * wg + buf) * C::Q_BYTES, ps->cq[wg][buf], tok);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ps->qfull[wg][buf]));
      };
      qn.load(a, ahead, tok);
      stage(0);
      int turn = 0;
      auto meet = [&](bool ok_) { return attn_meet(smem_u32(&ps->meet[wg]), turn, ok_, abort, limit); };
      bool ok = meet(true);                        // the first segment's factors are visible
      int j = 0;                                   // this warpgroup's tile
      for (int seg = 0;; ++seg) {
        bool staging = ahead.next_segment(a);
        if (staging) qn.load(a, ahead, tok);
        // pairs of heads; fa, fb: the last tile's factors.  Lane i of every warp keeps the running
        // maximum of head i % GT.
        uint64_t cq[NP], l[NP], o[DCH][NP], fa[NP], fb[NP];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          cq[i] = pack2(ps->cq[wg][seg & 1][2 * i], ps->cq[wg][seg & 1][2 * i + 1]);
          l[i] = fa[i] = fb[i] = 0u;
#pragma unroll
          for (int c = 0; c < DCH; ++c) o[c][i] = 0u;
        }
        // o = o * fa + (product of this warpgroup's tile j) * fb
        auto accumulate = [&](int j_) {
          ok &= attn_wait(smem_u32(&ps->ofull[wg]), j_ & 1u, abort, limit);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < DCH; ++c) {
            uint32_t r[4 * GT];
            tmem_cols(tmem_o + c * C::O_COLS, r);
            auto piece = [&](int k, int i) {
              return pack2(__uint_as_float(r[k * GT + 2 * i]), __uint_as_float(r[k * GT + 2 * i + 1]));
            };
            const uint64_t k16 = pack2(0.0625f, 0.0625f), k256 = pack2(0.00390625f, 0.00390625f);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const uint64_t x = fma2(piece(1, i), k16, piece(0, i)), y = fma2(piece(3, i), k16, piece(2, i));
              o[c][i] = fma2(o[c][i], fa[i], mul2(fma2(y, k256, x), fb[i]));
            }
          }
        };
        const int t_first = w.t;
        for (int t = t_first; ok && t < w.t1; ++t, ++j) {
          const int par = j & 1, e = j % kScaleRing;
          ok &= attn_wait(smem_u32(&ps->scales[wg][e]), (j / kScaleRing) & 1u, abort, limit);
          const float* sc = reinterpret_cast<const float*>(gbase + C::OFF_S + (wg * kScaleRing + e) * 1024);
          const int t0 = (w.s.ft + t) * kAttnTile;
          const uint32_t boxes = ps->boxes[wg][e];
          const bool live = t0 + tok >= w.s.st && t0 + tok < w.s.len && ((boxes >> (tok / a.BR)) & 1u);
          const float sk = live ? sc[tok] : 0.0f, sv = live ? sc[128 + tok] : 0.0f;
          // the tile's largest sv, four tokens a lane (every warp for itself: no exchange), 2^E >= it
          // (E >= -118, for which 2^(8 - E) is a number; a scale of 2^-126 is held to 2^-22), and
          // this token's e_t - E
          float top;
          {
            const float4 s4 = *reinterpret_cast<const float4*>(sc + 128 + 4 * lane);
            // (64 x up to 8000 tokens, 2 heads of 64 a kv head: 69.3 us with the masks skipped in a tile
            // that has none, 70.3 us without)
            float v0 = fabsf(s4.x), v1 = fabsf(s4.y), v2 = fabsf(s4.z), v3 = fabsf(s4.w);
            if (t0 < w.s.st || t0 + kAttnTile > w.s.len || boxes != all_boxes) {
              const int t4 = t0 + 4 * lane, lo = w.s.st - t4;
              const int hi = (boxes >> box4) & 1u ? w.s.len - t4 : 0;
              v0 = lo <= 0 && hi > 0 ? v0 : 0.0f;
              v1 = lo <= 1 && hi > 1 ? v1 : 0.0f;
              v2 = lo <= 2 && hi > 2 ? v2 : 0.0f;
              v3 = lo <= 3 && hi > 3 ? v3 : 0.0f;
            }
            top = warp_max(fmaxf(fmaxf(v0, v1), fmaxf(v2, v3)));
          }
          const int etop = int(__float_as_uint(top) >> 23), E = max(etop - 126, -118);
          const float apart =
              float(min(max(int(__float_as_uint(fabsf(sv)) >> 23) - etop, -kScaleSpread), 0));
          // (an infinite scale makes its token NaN: E4M3 would saturate without a trace)
          const float rsv = fabsf(sv) == INFINITY ? NAN : sv * __uint_as_float(uint32_t(8 - E + 127) << 23);
          const float down = __uint_as_float(uint32_t(E - 8 + 127) << 23);
          ok &= attn_wait(smem_u32(&ps->sfull[wg][par]), (j >> 1) & 1u, abort, limit);
          tc_fence_after();
          float x[GT];
          {
            uint32_t r[2 * GT];
            tmem_cols(tmem_s + par * C::S_COLS, r);
            float wm[GT];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const uint64_t hi = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
              const uint64_t lo = pack2(__uint_as_float(r[GT + 2 * i]), __uint_as_float(r[GT + 2 * i + 1]));
              const float2 v = unpack2(mul2(fma2(lo, pack2(0.0625f, 0.0625f), hi), mul2(cq[i], pack2(sk, sk))));
              x[2 * i] = live ? v.x : -INFINITY;
              x[2 * i + 1] = live ? v.y : -INFINITY;
              const float2 y = unpack2(add2(pack2(x[2 * i], x[2 * i + 1]), pack2(apart, apart)));
              wm[2 * i] = warp_max(y.x);
              wm[2 * i + 1] = warp_max(y.y);
            }
            if (lane == 0) {
#pragma unroll
              for (int g = 0; g < GT; g += 4)
                *reinterpret_cast<float4*>(&ps->red[wg][par][quad][g]) =
                    make_float4(wm[g], wm[g + 1], wm[g + 2], wm[g + 3]);
            }
          }
          if (t > t_first) accumulate(j - 1);
          ok = meet(ok);
          if (!ok) break;
          // lane i: the factors of head i % GT
          const int hg = lane & (GT - 1);
          const float tm = fmaxf(fmaxf(ps->red[wg][par][0][hg], ps->red[wg][par][1][hg]),
                                 fmaxf(ps->red[wg][par][2][hg], ps->red[wg][par][3][hg]));
          const float mn = fmaxf(m, tm);
          const float ref = mn == -INFINITY ? 0.0f : mn;        // nothing valid so far: every factor is 0
          const float la = ex2(m - ref), lb = ex2(tm - ref), lt = tm == -INFINITY ? 0.0f : tm;
          m = mn;
          uint64_t v[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float p0 = ex2(x[2 * i] - __shfl_sync(~0u, lt, 2 * i));
            const float p1 = ex2(x[2 * i + 1] - __shfl_sync(~0u, lt, 2 * i + 1));
            const uint64_t p = pack2(p0, p1);
            fa[i] = pack2(__shfl_sync(~0u, la, 2 * i), __shfl_sync(~0u, la, 2 * i + 1));
            const uint64_t be = pack2(__shfl_sync(~0u, lb, 2 * i), __shfl_sync(~0u, lb, 2 * i + 1));
            l[i] = fma2(l[i], fa[i], mul2(p, be));
            fb[i] = mul2(be, pack2(down, down));
            v[i] = mul2(p, pack2(rsv, rsv));
          }
          uint32_t pk[GT];                                      // [piece][heads], 4 codes a word
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < NP; i += 2) pk[k * (GT / 4) + i / 2] = split16(v[i]) | (split16(v[i + 1]) << 16);
#pragma unroll
          for (int i = 0; i < NP; i += 2) pk[3 * (GT / 4) + i / 2] = code2(v[i]) | (code2(v[i + 1]) << 16);
          uint8_t* pr = gbase + C::OFF_P + wg * C::P_BYTES + tok * C::P_ROW;
          const int sw = GT == 4 ? 0 : GT == 8 ? (tok >> 2) & 1 : (tok >> 1) & 3;
#pragma unroll
          for (int i = 0; i < GT / 4; ++i)
            *reinterpret_cast<uint4*>(pr + ((i ^ sw) * 16)) =
                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          const bool wipe = !live && ((boxes >> (tok / a.BR)) & 1u);
          if (__any_sync(~0u, wipe)) {                          // whatever the cache holds there times 0 is 0
            const int u = 2 * j + 1, s = u % SLOTS;
            ok &= attn_wait(smem_u32(&ps->full[wg][s]), (u / SLOTS) & 1u, abort, limit);
            if (wipe) {
              uint4* vr = reinterpret_cast<uint4*>(gbase + uint32_t(wg * SLOTS + s) * C::KV_BYTES + tok * 128);
#pragma unroll
              for (int c = 0; c < DCH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) vr[c * (kAttnTile * 8) + (i ^ (tok & 7))] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ps->pfull[wg]));
          if (staging) {                           // that buffer's reader, segment seg - 1, is done
            stage((seg + 1) & 1);
            staging = false;
          }
        }
        if (!ok) break;
        accumulate(j - 1);
        // sums of p over the tokens
        {
          float lg[GT];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float2 v = unpack2(l[i]);
            lg[2 * i] = v.x;
            lg[2 * i + 1] = v.y;
          }
          const float s1 = warp_sums(lg, lane);
          if ((lane & (32 / GT - 1)) == 0) ps->lsum[wg][quad][lane / (32 / GT)] = s1;
        }
        ok = meet(ok);
        if (!ok) break;
        const int g0 = w.hc * GT, heads = min(GT, a.G - g0);
        const bool whole = t_first == 0 && w.t1 == w.s.n;
        const int64_t head0 = (int64_t(w.b) * a.H + w.c) * a.G + g0;
        const int slot = 2 * worker + (seg > 0 ? 1 : 0);
        // lane i: the sum of head i % GT
        const int hg = lane & (GT - 1);
        const float sum = (ps->lsum[wg][0][hg] + ps->lsum[wg][1][hg]) + (ps->lsum[wg][2][hg] + ps->lsum[wg][3][hg]);
        if (tok < heads) {
          if (!whole) {
            a.ws_ml[int64_t(slot) * 2 * GT + tok] = m;
            a.ws_ml[int64_t(slot) * 2 * GT + GT + tok] = sum;
          } else if (a.lse != nullptr) {
            a.lse[head0 + tok] = log_sum(m, sum);
          }
        }
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);        // no valid token: zeros
#pragma unroll
        for (int ch = 0; ch < DCH; ++ch) {
          const bool on = ch * 128 + tok < a.D;
          if (whole) {
            __nv_bfloat16* po = reinterpret_cast<__nv_bfloat16*>(a.out) + head0 * a.D + ch * 128 + tok;
#pragma unroll
            for (int g = 0; g < GT; ++g) {
              const float2 og = unpack2(o[ch][g / 2]);
              const float v = (g & 1 ? og.y : og.x) * __shfl_sync(~0u, inv, g);
              if (on && g < heads) *po = __float2bfloat16_rn(v);
              po += a.D;
            }
          } else {
            float* pw = a.ws_o + int64_t(slot) * GT * a.D + ch * 128 + tok;
#pragma unroll
            for (int g = 0; g < GT; ++g) {
              const float2 og = unpack2(o[ch][g / 2]);
              if (on && g < heads) *pw = g & 1 ? og.y : og.x;
              pw += a.D;
            }
          }
        }
        if (t_first == 0 && tok == 0 && (a.by_row || !whole)) {
          const int row = (w.b * a.H + w.c) * a.HC + w.hc;
          int2 info = make_int2(-1, -1);
          if (!whole) {                            // the worker whose range holds the row's last tile
            const int64_t next = int64_t(plan.begin(worker + 1)) + w.s.n - w.t1;     // of the list: the next row
            info = make_int2(row, (slot << 16) | (int((next * plan.workers + plan.total - 1) / plan.total) - 1));
          }
          a.ws_join[a.by_row ? row : worker] = info;
        }
        if (!w.next_segment(a)) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // After a wait that ran out, loads and MMAs may still be under way, also those of warps that
  // had come to their end by then: all land before shared and tensor memory are given back.
  // (Nobody sets the flag any more, so all threads see the same.)
  if (*abort) {
    const int g = warp & 1;
    if (warp < 2) {
      for (int i = max(0, u - SLOTS); i < u; ++i)
        mbar_drain(smem_u32(&ps->full[g][i % SLOTS]), (i / SLOTS) & 1u);
      cp_async_wait_all();
    } else if (warp < 4) {
      if (elect_one()) {
        mma_commit(smem_u32(&ps->drain[g]));
        mbar_drain(smem_u32(&ps->drain[g]), 0u);
      }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Rows that more than one worker has a part of: their partial sums added up in the order of the
// tiles.  One block per row and head: first every partial's factor (its maximum against the
// largest), then the sums, the warps taking the partials in turn, 16 bytes a lane and several
// loads in flight.  Bound by the latency of these two dependent rounds of loads.
// A worker has at most one row that begins in its range and ends elsewhere, so that there are no
// more entries than workers: with a block for each of 4096 rows and 4 heads, nearly all with
// nothing to do, 512 sequences of up to 1000 tokens took 118 us, with entries by worker 104 us.
constexpr int kJoinThreads = 256;
constexpr int kJoinMax = 1024;      // partials of one row: at most two workers an SM

template <int GT>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const AttnArgs a) {
  constexpr int W = kJoinThreads / 32;
  __shared__ float sf[kJoinMax];
  __shared__ float sm[W], sl[W];
  __shared__ __align__(16) float so[W][256];
  pdl_trigger();
  pdl_wait();
  const int2 info = a.ws_join[blockIdx.x];
  const int row = info.x, slot0 = info.y >> 16, worker0 = slot0 >> 1, last = info.y & 0xFFFF;
  // nothing to join, or, after a wait that ran out, an entry that was never written
  if (row < 0 || row >= a.B * a.H * a.HC || slot0 < 0 || last < worker0 || last >= a.slots / 2) return;
  const int g = blockIdx.y, hc = row % a.HC;
  if (hc * GT + g >= a.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = min(last - worker0 + 1, kJoinMax);
  auto slot_of = [&](int i) { return int64_t(i == 0 ? slot0 : 2 * (worker0 + i)); };
  float m = -INFINITY, l = 0.0f;
  for (int i = threadIdx.x; i < n; i += kJoinThreads) {
    const float* p = a.ws_ml + slot_of(i) * 2 * GT + g;
    const float mi = p[0], li = p[GT];
    sf[i] = mi;
    const float mn = fmaxf(m, mi);
    l = l * ex2(m == mn ? 0.0f : m - mn) + li * ex2(mi == mn ? 0.0f : mi - mn);
    m = mn;
  }
  const float wm = warp_max(m);
  if (lane == 0) sm[warp] = wm;
  __syncthreads();
  float top = sm[0];
#pragma unroll
  for (int i = 1; i < W; ++i) top = fmaxf(top, sm[i]);
  const float ref = top == -INFINITY ? 0.0f : top;
  l *= ex2(m - ref);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
  if (lane == 0) sl[warp] = l;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  const bool on0 = lane * 4 < a.D, on1 = lane * 4 + 128 < a.D;
#pragma unroll 4
  for (int i = warp; i < n; i += W) {
    const float* p = a.ws_o + (slot_of(i) * GT + g) * a.D + lane * 4;
    const float f = ex2(sf[i] - ref);
    const float4 x = on0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 y = on1 ? *reinterpret_cast<const float4*>(p + 128) : make_float4(0.f, 0.f, 0.f, 0.f);
    o[0] = make_float4(fmaf(f, x.x, o[0].x), fmaf(f, x.y, o[0].y), fmaf(f, x.z, o[0].z), fmaf(f, x.w, o[0].w));
    o[1] = make_float4(fmaf(f, y.x, o[1].x), fmaf(f, y.y, o[1].y), fmaf(f, y.z, o[1].z), fmaf(f, y.w, o[1].w));
  }
  reinterpret_cast<float4*>(so[warp])[lane] = o[0];
  reinterpret_cast<float4*>(so[warp])[32 + lane] = o[1];
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) l += sl[i];
  const int64_t head = int64_t(row / a.HC) * a.G + hc * GT + g;
  const int d = threadIdx.x;
  if (d < a.D) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += so[i][d];
    reinterpret_cast<__nv_bfloat16*>(a.out)[head * a.D + d] = __float2bfloat16_rn(l == 0.0f ? 0.0f : v / l);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[head] = log_sum(top, l);
}

}  // namespace fp8lin
