// attn.cuh -- attention of one new token per sequence over a paged FP8 key-value cache.
//
// For sequence b, query head h of key-value head c (G = Hq / Hkv heads share one), tokens t
// of the sequence (its length, its window and its valid pages decide which):
//   s_t = scale * sk_t * sum_d q_d dec(k_t[d])            p_t = exp(s_t - max s)
//   out = (sum_t p_t sv_t dec(v_t)) / sum_t p_t
// What bounds it: the cache is read once, 2 D + 8 bytes a token and kv head, against 4 D G
// flops, so HBM does up to about a hundred heads per kv head.  The kernel is built so that
// no code byte is ever converted: both products run on the FP8 tensor cores straight from
// the tiles TMA has put into shared memory.
//   scores   S^T[128 tokens x heads] = K-tile (A, 128 x D) . q^T.  A bf16 q (8 significant
//            bits) is split into two E4M3 pieces q = (hi + lo / 16) 2^-e, 4 bits each with
//            e from the head's largest |q|: exact for every element above 2^-14 of the
//            largest and off by at most 2^-21 of the largest below that.  The pieces are
//            2 x heads columns of B; tensor memory then holds one token per lane, so the
//            token's scale is one register.
//   softmax  per tile: maximum over the 128 tokens (one redux per warp and head, one exchange
//            through shared memory), p, and w = p sv 2^(8 - E), 2^E >= the tile's largest sv.
//   output   O^T[D x heads] = V-tile^T (A, read "transposed" as stored: D contiguous) . w.
//            w is split into four E4M3 pieces w = c0 + c1/16 + c2/256 + c3/4096: off by at
//            most 2^-17 relative, or 2^-30 of the tile's largest possible w.  Each tile's
//            product lands in fresh tensor-memory columns and is folded into fp32 registers
//            (one channel d per thread) with the running maximum's factors.
// A CTA (one per SM): warp 0 loads pages (TMA; one lane per box of gcd(page, 128) rows, its
// scales by bulk copies), warp 1 issues MMAs, warps 2-5 do softmax and accumulation.
//
// Split: the batch's tiles, row after row (a row is a sequence, kv head and chunk of GT query
// heads), form one list that is cut into equal ranges, one per CTA, whatever the lengths.
// A row inside one range is finished there; a row cut by a border leaves partial sums (o, m, l)
// in the workspace, which k_attn_join adds up in the order of the tiles, so results do not
// depend on timing.
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

#include "ptx.cuh"
#include "quant.cuh"

namespace fp8lin {

constexpr int kAttnThreads = 192;
constexpr int kAttnTile = 128;

struct AttnArgs {
  const uint16_t* q;       // bf16 [B][Hq][D], strides below
  const float* ks;         // [pages][H][P]
  const float* vs;
  const int32_t* table;    // [B][max_pages], row stride table_stride
  const int32_t* lens;     // [B]
  uint16_t* out;           // bf16 [B][Hq][D]
  float* lse;              // [B][Hq] or nullptr
  float* ws_o;             // [2 * CTAs][GT][D]
  float* ws_ml;            // [2 * CTAs][2][GT]
  int2* ws_row;            // [rows]: (slot of the first partial, CTA of the last one), or (-1, -1)
  int64_t q_row, q_head, table_stride;
  int64_t window, cap;     // tokens; window 0 = none; cap = max_pages * P
  int64_t pages;
  float scale;
  int B, H, G, HC, D, P, BR;   // HC chunks of query heads per kv head; BR rows per box
};

template <int GT_, int DCH_>
struct AttnCfg {
  static constexpr int GT = GT_, DCH = DCH_;
  static constexpr int STAGES = DCH == 1 ? 6 : 3;
  static constexpr uint32_t KV_BYTES = kAttnTile * 128 * DCH;
  static constexpr uint32_t Q_BYTES = 2 * GT * 128 * DCH;
  static constexpr uint32_t P_ROW = 4 * GT;                  // bytes per token of the split weights
  static constexpr uint32_t P_BYTES = kAttnTile * P_ROW;
  static constexpr uint32_t OFF_Q = STAGES * 2 * KV_BYTES;
  static constexpr uint32_t OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr uint32_t OFF_S = OFF_P + P_BYTES;         // scales: [STAGES][2][128] fp32
  static constexpr uint32_t OFF_STATE = OFF_S + STAGES * 1024;
  static constexpr uint32_t S_COLS = 2 * GT, O_COLS = 4 * GT;
  static constexpr uint32_t TMEM_USED = 2 * S_COLS + DCH * O_COLS;
  static constexpr uint32_t TMEM_COLS = TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : 256;
};

template <int GT, int STAGES>
struct alignas(16) AttnState {
  float red[2][4][GT];     // per-warp maxima, double-buffered by tile
  float redsv[2][4];
  float lsum[4][GT];
  float cq[2][GT];         // per-head factor of the staged queries
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t sfull[2], qfull[2];
  uint64_t pfull, ofull, drain;
  uint32_t boxes[STAGES];  // which boxes of the stage hold a valid page
  uint32_t tmem_base;
  int abort;
  int total, first_b, first_off;
};

template <class C>
constexpr size_t attn_smem_bytes() {
  return 1024 + C::OFF_STATE + sizeof(AttnState<C::GT, C::STAGES>);
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

// The walk over a CTA's range of tiles, segment by segment (a segment: the part of one row
// inside the range).  Every role walks the same sequence.
struct AttnWalk {
  int b, rr, t0, t1, left;
  AttnSeq s;
  __device__ __forceinline__ void start(const AttnArgs& a, int first_b, int off, int count) {
    b = first_b;
    s = attn_seq(a, b);
    rr = off / s.n;
    t0 = off - rr * s.n;
    t1 = min(s.n, t0 + count);
    left = count - (t1 - t0);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    if (left <= 0) return false;
    if (++rr == a.H * a.HC) {
      rr = 0;
      s = attn_seq(a, ++b);
    }
    t0 = 0;
    t1 = min(s.n, left);
    left -= t1;
    return true;
  }
};

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
// Barrier of the 128 softmax threads that also tells whether any of them has failed.
__device__ __forceinline__ bool attn_barrier_or(bool p) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(int(p))
      : "memory");
  return r != 0;
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

// Shared-memory descriptor of an MN-major operand (rows along K, `row` bytes of the M or N
// axis each, written with the swizzle of that width): 8-row groups `row * 8` bytes apart in
// the stride offset; the leading offset is unused because one row spans the whole M or N.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t row) {
  const uint64_t layout = row == 128 ? 2u : row == 64 ? 4u : 6u;    // 128-, 64-, 32-byte swizzle
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)((row * 8) >> 4) << 32) |
         ((uint64_t)1 << 46) | (layout << 61);
}
// Instruction descriptor with A in the cache's format (0 E4M3, 1 E5M2), B E4M3; `mn`: both
// operands MN-major.
__device__ __forceinline__ constexpr uint32_t attn_idesc(int fmt, uint32_t n, bool mn) {
  return idesc_f8_e4m3_f32(128, n) | (uint32_t(fmt) << 7) | (mn ? (3u << 15) : 0u);
}

// fp32 pair -> two E4M3 codes and what they leave, times 16.
__device__ __forceinline__ uint32_t split16(float& a, float& b) {
  const uint32_t c = cvt2<kE4M3>(a, b);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(c)));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  a = (a - f.x) * 16.0f;
  b = (b - f.y) * 16.0f;
  return c;
}

// Scan of the batch by one warp: the number of tiles of all rows, then the sequence and the
// offset in its rows at which this CTA's range begins.
__device__ __forceinline__ void attn_scan(const AttnArgs& a, int lane, int* total, int* first_b, int* first_off) {
  const int rows = a.H * a.HC;
  int sum = 0;
  for (int i = 0; i < a.B; i += 32)
    sum += __reduce_add_sync(~0u, i + lane < a.B ? attn_seq(a, i + lane).n * rows : 0);
  const int ctas = min(int(gridDim.x), sum);
  const int x0 = int(int64_t(sum) * blockIdx.x / ctas);
  int run = 0;
  for (int i = 0; i < a.B; i += 32) {
    const int v = i + lane < a.B ? attn_seq(a, i + lane).n * rows : 0;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += y;
    }
    if (x0 >= run + inc - v && x0 < run + inc) {
      *first_b = i + lane;
      *first_off = x0 - (run + inc - v);
    }
    run += __shfl_sync(~0u, inc, 31);
    if (run > x0) break;
  }
  if (lane == 0) *total = sum;
}

// Queries of a segment -> two E4M3 pieces as K-major rows (hi: head g, lo: head GT + g) in
// shared memory, and the factor that turns their products into base-2 exponents.
template <class C>
__device__ __forceinline__ void attn_stage_q(const AttnArgs& a, const AttnWalk& w, uint8_t* sq, float* cq, int tid) {
  constexpr int UPH = 8 * C::DCH;            // 16-channel units per head
  const int c = w.rr / a.HC, g0 = (w.rr % a.HC) * C::GT;
#pragma unroll
  for (int u0 = 0; u0 < C::GT * UPH; u0 += 128) {
    const int u = u0 + tid;
    const bool on = u < C::GT * UPH;         // uniform over a warp: units come in multiples of 64
    if (!on) break;
    const int head = u / UPH, ch = u % UPH;
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (g0 + head < a.G && ch * 16 < a.D) {
      const uint4* p = reinterpret_cast<const uint4*>(a.q + int64_t(w.b) * a.q_row +
                                                      int64_t(c * a.G + g0 + head) * a.q_head + ch * 16);
      v[0] = __ldg(p);
      v[1] = __ldg(p + 1);
    }
    const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t mx = 0;                         // largest |q| as bf16 bits: NaN and Inf sort above all
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int d = 1; d < UPH; d <<= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, d));
    const bool bad = mx >= 0x7F80u;          // a NaN or infinity: the head's output is NaN
    const int e = min(7 - (int(mx >> 7) - 127), 126);       // q 2^e in [128, 256)
    const float up = __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p0 = bf16_lo(x[2 * i]) * up, p1 = bf16_hi(x[2 * i]) * up;
      float p2 = bf16_lo(x[2 * i + 1]) * up, p3 = bf16_hi(x[2 * i + 1]) * up;
      const uint32_t h0 = split16(p0, p1), h1 = split16(p2, p3);
      hi[i] = bad ? 0x7F7F7F7Fu : h0 | (h1 << 16);
      lo[i] = bad ? 0x7F7F7F7Fu : cvt2<kE4M3>(p0, p1) | (cvt2<kE4M3>(p2, p3) << 16);
    }
    uint8_t* base = sq + (ch / 8) * (2 * C::GT * 128);
    *reinterpret_cast<uint4*>(base + head * 128 + (((ch & 7) ^ (head & 7)) * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(base + (C::GT + head) * 128 + (((ch & 7) ^ (head & 7)) * 16)) =
        make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (ch == 0) cq[head] = a.scale * 1.44269504088896340736f / up;
  }
}

template <int FMT, class C>
__global__ void __launch_bounds__(kAttnThreads, 1)
    k_paged_attention(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const AttnArgs a) {
  constexpr int GT = C::GT, DCH = C::DCH, STAGES = C::STAGES;
  using State = AttnState<GT, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  State* ps = reinterpret_cast<State*>(gbase + C::OFF_STATE);
  volatile int* abort = &ps->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&ps->full[s]), 1);
      mbar_init(smem_u32(&ps->empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ps->sfull[i]), 1);
      mbar_init(smem_u32(&ps->qfull[i]), 4);
    }
    mbar_init(smem_u32(&ps->pfull), 4);
    mbar_init(smem_u32(&ps->ofull), 1);
    mbar_init(smem_u32(&ps->drain), 1);
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
  if (warp == 2) attn_scan(a, lane, &ps->total, &ps->first_b, &ps->first_off);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ps->tmem_base;
  const uint32_t tmem_o = tmem + 2 * C::S_COLS;
  const int total = ps->total;
  const int ctas = min(int(gridDim.x), total);
  const int cta = blockIdx.x;
  const int count = cta < ctas ? int(int64_t(total) * (cta + 1) / ctas) - int(int64_t(total) * cta / ctas) : 0;

  if (count > 0) {
    AttnWalk w;
    w.start(a, ps->first_b, ps->first_off, count);
    if (warp == 0) {
      // ------------------------------------------------ pages -> shared memory
      const int nb = kAttnTile / a.BR;
      int t = w.t0;
      // this lane's box of tile t: its page if it holds a token, and the row inside it
      auto lookup = [&](int& page, int& row) {
        const int tok = (w.s.ft + t) * kAttnTile + lane * a.BR;
        page = -1;
        row = 0;
        if (lane < nb && tok < w.s.len && tok + a.BR > w.s.st) {
          const int p = tok / a.P;
          row = tok - p * a.P;
          page = __ldg(a.table + int64_t(w.b) * a.table_stride + p);
        }
      };
      int page, row;
      lookup(page, row);
      int it = 0;
      for (; it < count; ++it) {
        const int h = w.rr / a.HC;
        const int pg = page, rw = row;
        if (++t == w.t1 && w.next(a)) t = 0;
        if (it + 1 < count) lookup(page, row);
        const int s = it % STAGES;
        if (!__all_sync(~0u, mbar_wait(smem_u32(&ps->empty[s]), ((it / STAGES) & 1u) ^ 1u, abort))) break;
        const bool ok = pg >= 0 && pg < a.pages;
        const uint32_t bar = smem_u32(&ps->full[s]);
        const uint32_t boxes = __ballot_sync(~0u, ok);
        if (lane == 0) {
          ps->boxes[s] = boxes;
          mbar_arrive_expect_tx(bar, 2 * C::KV_BYTES + __popc(boxes) * uint32_t(a.BR) * 8u);
        }
        __syncwarp();
        if (lane < nb) {
          const uint32_t off = base + uint32_t(s) * (2 * C::KV_BYTES) + uint32_t(lane * a.BR) * 128u;
          const int pc = ok ? pg : int(a.pages);
#pragma unroll
          for (int c = 0; c < DCH; ++c) {
            tma_load_4d(off + c * (kAttnTile * 128), &tmK, bar, c * 128, rw, h, pc);
            tma_load_4d(off + C::KV_BYTES + c * (kAttnTile * 128), &tmV, bar, c * 128, rw, h, pc);
          }
          if (ok) {
            const int64_t at = (int64_t(pg) * a.H + h) * a.P + rw;
            const uint32_t sc = base + C::OFF_S + s * 1024 + lane * a.BR * 4;
            bulk_load(sc, a.ks + at, uint32_t(a.BR) * 4u, bar);
            bulk_load(sc + 512, a.vs + at, uint32_t(a.BR) * 4u, bar);
          }
        }
      }
      if (*abort) {                      // every load already issued lands before the CTA exits
        for (int j = max(0, it - STAGES); j < it; ++j)
          mbar_drain(smem_u32(&ps->full[j % STAGES]), (j / STAGES) & 1u);
      }
      pdl_trigger();
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------------------------------------- MMA issuer
        constexpr uint32_t id_s = attn_idesc(FMT, 2 * GT, false), id_o = attn_idesc(FMT, 4 * GT, true);
        int t = w.t0, seg = 0;
        bool fresh = true;                 // the next tile is the first of its segment
        auto scores = [&](int i) {         // S of tile i; tiles come in order
          const int s = i % STAGES;
          if (fresh && !mbar_wait(smem_u32(&ps->qfull[seg & 1]), (seg >> 1) & 1u, abort)) return false;
          if (!mbar_wait(smem_u32(&ps->full[s]), (i / STAGES) & 1u, abort)) return false;
          tc_fence_after();
          const uint32_t k0 = base + uint32_t(s) * (2 * C::KV_BYTES);
          const uint32_t q0 = base + C::OFF_Q + (seg & 1) * C::Q_BYTES;
#pragma unroll
          for (int k = 0; k < 4 * DCH; ++k)
            mma_f8(tmem + (i & 1) * C::S_COLS, sw128_kmajor_desc(k0 + (k / 4) * (kAttnTile * 128) + (k % 4) * 32),
                   sw128_kmajor_desc(q0 + (k / 4) * (2 * GT * 128) + (k % 4) * 32), id_s, k > 0 ? 1u : 0u);
          mma_commit(smem_u32(&ps->sfull[i & 1]));
          fresh = false;
          if (++t == w.t1 && w.next(a)) {
            t = 0;
            ++seg;
            fresh = true;
          }
          return true;
        };
        bool ok = scores(0) && (count < 2 || scores(1));
        for (int i = 0; ok && i < count; ++i) {
          if (!mbar_wait(smem_u32(&ps->pfull), i & 1u, abort)) break;
          tc_fence_after();
          const int s = i % STAGES;
          const uint32_t v0 = base + uint32_t(s) * (2 * C::KV_BYTES) + C::KV_BYTES;
#pragma unroll
          for (int c = 0; c < DCH; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8(tmem_o + c * C::O_COLS, mn_desc(v0 + c * (kAttnTile * 128) + k * 32 * 128, 128),
                     mn_desc(base + C::OFF_P + k * 32 * C::P_ROW, C::P_ROW), id_o, k > 0 ? 1u : 0u);
          mma_commit(smem_u32(&ps->ofull));
          mma_commit(smem_u32(&ps->empty[s]));
          if (i + 2 < count) ok = scores(i + 2);
        }
        if (*abort) {                      // the MMAs already issued finish before tensor memory is freed
          mma_commit(smem_u32(&ps->drain));
          mbar_drain(smem_u32(&ps->drain), 0u);
        }
      }
    } else {
      // ------------------------------------------------ softmax and accumulation
      const int tid = threadIdx.x - 64;            // staging unit and barrier index
      const int quad = warp & 3;                   // tensor-memory lanes of this warp
      const int tok = quad * 32 + lane;            // token of the tile; channel of the output
      const uint32_t tlane = uint32_t(quad * 32) << 16;
      uint8_t* sq = gbase + C::OFF_Q;
      auto stage = [&](const AttnWalk& x, int buf) {
        attn_stage_q<C>(a, x, sq + buf * C::Q_BYTES, ps->cq[buf], tid);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ps->qfull[buf]));
      };
      AttnWalk ahead = w;                          // the segment whose queries are staged next
      stage(ahead, 0);
      bool more = ahead.next(a);
      bool ok = true;
      attn_barrier_or(false);                      // the first segment's factors are visible
      int it = 0;
      for (int seg = 0;; ++seg) {
        if (more) {                                // the buffer's last reader, segment seg - 1, is done
          stage(ahead, (seg + 1) & 1);
          more = ahead.next(a);
        }
        float cq[GT], m[GT], l[GT], o[DCH][GT], fa[GT], fb[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          cq[g] = ps->cq[seg & 1][g];
          m[g] = -INFINITY;
          l[g] = 0.0f;
          fa[g] = fb[g] = 0.0f;
#pragma unroll
          for (int c = 0; c < DCH; ++c) o[c][g] = 0.0f;
        }
        // o = o * fa + (product of the last tile) * fb
        auto accumulate = [&](int i) {
          ok &= mbar_wait(smem_u32(&ps->ofull), i & 1u, abort);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < DCH; ++c) {
            uint32_t r[2][2 * GT];
            if constexpr (GT == 8) {
              tmem_ld16(tmem_o + tlane + c * C::O_COLS, r[0]);
              tmem_ld16(tmem_o + tlane + c * C::O_COLS + 16, r[1]);
            } else {
              tmem_ld32(tmem_o + tlane + c * C::O_COLS, r[0]);
              tmem_ld32(tmem_o + tlane + c * C::O_COLS + 32, r[1]);
            }
            tmem_ld_wait();
            tmem_regs_ready(r[0]);
            tmem_regs_ready(r[1]);
#pragma unroll
            for (int g = 0; g < GT; ++g) {
              const float x = __uint_as_float(r[0][g]) + __uint_as_float(r[0][GT + g]) * 0.0625f;
              const float y = __uint_as_float(r[1][g]) + __uint_as_float(r[1][GT + g]) * 0.0625f;
              o[c][g] = fmaf(o[c][g], fa[g], fmaf(y, 0.00390625f, x) * fb[g]);
            }
          }
        };
        bool failed = false;
        for (int t = w.t0; t < w.t1; ++t, ++it) {
          const int s = it % STAGES, sb = it & 1;
          ok &= mbar_wait(smem_u32(&ps->full[s]), (it / STAGES) & 1u, abort);
          const float* sc = reinterpret_cast<const float*>(gbase + C::OFF_S + s * 1024);
          const int t0 = (w.s.ft + t) * kAttnTile;
          const uint32_t boxes = ps->boxes[s];
          const bool live = t0 + tok >= w.s.st && t0 + tok < w.s.len && ((boxes >> (tok / a.BR)) & 1u);
          const float sk = live ? sc[tok] : 0.0f, sv = live ? sc[128 + tok] : 0.0f;
          ok &= mbar_wait(smem_u32(&ps->sfull[sb]), (it >> 1) & 1u, abort);
          tc_fence_after();
          uint32_t r[2 * GT];
          if constexpr (GT == 8) tmem_ld16(tmem + tlane + sb * C::S_COLS, r);
          else tmem_ld32(tmem + tlane + sb * C::S_COLS, r);
          tmem_ld_wait();
          tmem_regs_ready(r);
          float x[GT];
#pragma unroll
          for (int g = 0; g < GT; ++g) {
            const float v = fmaf(__uint_as_float(r[GT + g]), 0.0625f, __uint_as_float(r[g])) * (cq[g] * sk);
            x[g] = live ? v : -INFINITY;
            const float wm = warp_max(x[g]);
            if (lane == 0) ps->red[sb][quad][g] = wm;
          }
          {
            const float wm = warp_max(sv);
            if (lane == 0) ps->redsv[sb][quad] = wm;
          }
          if (attn_barrier_or(!ok)) {
            failed = true;
            break;
          }
          const float4 vm = *reinterpret_cast<const float4*>(ps->redsv[sb]);
          // 2^E >= the largest sv (E >= -110: below that, values are tiny against any other)
          const int E = max(int(__float_as_uint(fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w))) >> 23) - 126, -110);
          const float rsv = sv * __uint_as_float(uint32_t(8 - E + 127) << 23);
          const float down = __uint_as_float(uint32_t(E - 8 + 127) << 23);
          float na[GT], nb[GT];
#pragma unroll
          for (int g = 0; g < GT; ++g) {
            const float tm = fmaxf(fmaxf(ps->red[sb][0][g], ps->red[sb][1][g]),
                                   fmaxf(ps->red[sb][2][g], ps->red[sb][3][g]));
            const float mn = fmaxf(m[g], tm);
            const float ref = mn == -INFINITY ? 0.0f : mn;      // nothing valid so far: every factor is 0
            na[g] = ex2(m[g] - ref);
            const float be = ex2(tm - ref);
            const float p = ex2(x[g] - (tm == -INFINITY ? 0.0f : tm));
            m[g] = mn;
            l[g] = fmaf(l[g], na[g], p * be);
            nb[g] = be * down;
            x[g] = p * rsv;
          }
          uint32_t pk[GT];                                      // [piece][heads], 4 codes a word
#pragma unroll
          for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int g = 0; g < GT; g += 4)
              pk[j * (GT / 4) + g / 4] = split16(x[g], x[g + 1]) | (split16(x[g + 2], x[g + 3]) << 16);
#pragma unroll
          for (int g = 0; g < GT; g += 4)
            pk[3 * (GT / 4) + g / 4] = cvt2<kE4M3>(x[g], x[g + 1]) | (cvt2<kE4M3>(x[g + 2], x[g + 3]) << 16);
          if (t > w.t0) accumulate(it - 1);
#pragma unroll
          for (int g = 0; g < GT; ++g) {
            fa[g] = na[g];
            fb[g] = nb[g];
          }
          uint8_t* pr = gbase + C::OFF_P + tok * C::P_ROW;
          const int sw = GT == 8 ? (tok >> 2) & 1 : (tok >> 1) & 3;
#pragma unroll
          for (int j = 0; j < GT / 4; ++j)
            *reinterpret_cast<uint4*>(pr + ((j ^ sw) * 16)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          if (!live) {                                          // whatever the cache holds there times 0 is 0
            uint4* vr = reinterpret_cast<uint4*>(gbase + uint32_t(s) * (2 * C::KV_BYTES) + C::KV_BYTES + tok * 128);
#pragma unroll
            for (int c = 0; c < DCH; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j) vr[c * (kAttnTile * 8) + j] = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ps->pfull));
        }
        if (failed) break;
        accumulate(it - 1);
        // sums of p over the tile's tokens
#pragma unroll
        for (int g = 0; g < GT; ++g) {
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) l[g] += __shfl_xor_sync(~0u, l[g], d);
          if (lane == 0) ps->lsum[quad][g] = l[g];
        }
        if (attn_barrier_or(!ok)) break;
        const int c = w.rr / a.HC, g0 = (w.rr % a.HC) * GT;
        const int64_t row = int64_t(w.b) * (a.H * a.HC) + w.rr;
        const bool whole = w.t0 == 0 && w.t1 == w.s.n;
        const int slot = 2 * cta + (seg > 0 ? 1 : 0);
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          const float sum = ps->lsum[0][g] + ps->lsum[1][g] + ps->lsum[2][g] + ps->lsum[3][g];
          if (g0 + g < a.G) {
            if (whole) {
              const int64_t head = int64_t(w.b) * (int64_t(a.H) * a.G) + int64_t(c) * a.G + g0 + g;
              const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;      // no valid token: zeros, lse -inf
#pragma unroll
              for (int ch = 0; ch < DCH; ++ch)
                if (ch * 128 + tok < a.D)
                  reinterpret_cast<__nv_bfloat16*>(a.out)[head * a.D + ch * 128 + tok] =
                      __float2bfloat16_rn(sum == 0.0f ? 0.0f : o[ch][g] * inv);
              if (a.lse != nullptr && tok == g)
                a.lse[head] = sum == 0.0f ? -INFINITY : (m[g] + __log2f(sum)) * 0.69314718055994530942f;
            } else {
#pragma unroll
              for (int ch = 0; ch < DCH; ++ch)
                if (ch * 128 + tok < a.D)
                  a.ws_o[(int64_t(slot) * GT + g) * a.D + ch * 128 + tok] = o[ch][g];
              if (tok == g) {
                a.ws_ml[(int64_t(slot) * 2) * GT + g] = m[g];
                a.ws_ml[(int64_t(slot) * 2 + 1) * GT + g] = sum;
              }
            }
          }
        }
        if (w.t0 == 0 && tok == 0) {
          // the row's last tile in the list of all tiles, and the CTA whose range holds it
          const int64_t last = int64_t(total) * cta / ctas + (it - (w.t1 - w.t0)) + w.s.n - 1;
          const int lc = int(((last + 1) * ctas + total - 1) / total) - 1;
          a.ws_row[row] = whole ? make_int2(-1, -1) : make_int2(slot, lc);
        }
        if (!w.next(a)) break;
      }
    }
  } else {
    if (warp == 0) pdl_trigger();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Rows that more than one CTA worked on: their partial sums added up in the order of the
// tiles.  One block per row and head; its warps take the partials in turn.
template <int GT>
__global__ void __launch_bounds__(128) k_attn_join(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float so[4][256];
  __shared__ float sl[4];
  const int64_t row = blockIdx.x;
  const int2 info = a.ws_row[row];
  if (info.x < 0) return;
  const int g = blockIdx.y, rr = int(row % (a.H * a.HC));
  const int c = rr / a.HC, g0 = (rr % a.HC) * GT;
  if (g0 + g >= a.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = info.y - info.x / 2 + 1;
  auto slot_of = [&](int i) { return i == 0 ? info.x : 2 * (info.x / 2 + i); };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, a.ws_ml[int64_t(slot_of(i)) * 2 * GT + g]);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.0f : m;
  float o[8], l = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 0.0f;
  for (int i = warp; i < n; i += 4) {
    const int64_t s = slot_of(i);
    const float f = ex2(a.ws_ml[s * 2 * GT + g] - ref);
    l = fmaf(f, a.ws_ml[(s * 2 + 1) * GT + g], l);
    const float* p = a.ws_o + (s * GT + g) * a.D;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * 32 + lane < a.D) o[j] = fmaf(f, p[j * 32 + lane], o[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) so[warp][j * 32 + lane] = o[j];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const int64_t head = (row / (a.H * a.HC)) * (int64_t(a.H) * a.G) + int64_t(c) * a.G + g0 + g;
  for (int d = threadIdx.x; d < a.D; d += 128) {
    const float v = (so[0][d] + so[1][d]) + (so[2][d] + so[3][d]);
    reinterpret_cast<__nv_bfloat16*>(a.out)[head * a.D + d] = __float2bfloat16_rn(l == 0.0f ? 0.0f : v / l);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[head] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
}

}  // namespace fp8lin
