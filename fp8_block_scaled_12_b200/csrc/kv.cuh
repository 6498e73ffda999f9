// kv.cuh -- what goes into and comes out of the paged FP8 key-value cache (sm_100a).
//
//  k_norm_rope_write  per token and head: RMS norm, position rotation, and the store: q (and
//                     k without a cache) as bf16, k and v of the cache as FP8 codes and one
//                     scale per token and head.  Every part may be left out, so the same
//                     kernel serves fp8_qk_norm_rope, fp8_kv_write and the fused call.
//  k_kv_read          pages of a batch of sequences back as bf16 rows.
//
// Mathematics of one head x[0..D) of a token at position p:
//   n_i = x_i / sqrt(mean(x^2) + eps) * w_i
//   y_a = n_a cos(p f_i) - n_b sin(p f_i),  y_b = n_b cos(p f_i) + n_a sin(p f_i)
// for the R / 2 pairs (a, b) = (i, R/2 + i), or (2i, 2i + 1) interleaved; channels from R on
// keep n.  The cosines and sines come from a table.  All of it stays in fp32 registers, so
// a value is rounded once, where it is stored: to bf16, or by the FP8 rule of quant.cuh.
// Bound by memory: 2 bytes read and 2 (bf16) or 1 (FP8) written per channel.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace fp8lin {

enum : int { kRopeNone = 0, kRopeInterleaved = 1, kRopeHalves = 2 };

// The cache as the kernels see it; strides in bytes (codes).
struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t page_stride, head_stride, token_stride;
  int64_t pages;
  int P, H, D;
};

// One of q, k and v on its way through a call.
struct KvPart {
  const uint16_t* src;      // bf16 [T][heads][D], token and head strides in elements
  int64_t tok, head;
  uint16_t* out;            // bf16 output (may be src), or nullptr: into the cache
  int64_t out_tok, out_head;
  const uint16_t* w;        // norm weights bf16 [D]; nullptr: no norm
  uint8_t* codes;           // the cache's codes and scales
  float* scales;
  int heads;
  int turn;                 // whether it is rotated
  int begin, blocks;        // its blocks of the grid
};

struct KvWriteArgs {
  KvPart part[3];
  const float* cos_sin;     // [max_pos][R]
  const int64_t* pos;       // [T]
  const int64_t* slots;     // [T]
  int64_t page_stride, head_stride, token_stride, slot_count;   // of the cache
  int64_t max_pos;
  float eps, inv_d;         // inv_d = 1 / D
  int T, D, R, P, H;        // P, H: the cache's page size and heads
  int parts;
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// LPH lanes own one head of one token, 16 channels each as two runs of 8 (a, b): for pairs
// (i, R/2 + i) the two runs that rotate into each other, so that the rotation never leaves a
// thread, else run j of each half of the head.  Loads and bf16 stores are 16 bytes a lane and
// adjacent over the lanes.  A group of lanes keeps U heads (two, or one while one token a group
// is all there is: the heads' latencies add up then) and goes from token to token: the norm's
// weights are loaded once, position, slot, cosines and sines serve all of its heads, nothing is
// divided but the slot, and the channels of the next kWriteAhead tokens are on their way through
// shared memory meanwhile.  A block works on one of q, k and v, so
// pointers and strides stay in constant memory and what one of them does not need is not there.
// Issue slots bound it next to memory, hence packed fp32 pairs throughout.  16384 tokens of
// 32 + 8 + 8 heads of 128 in one pass: 66 us, 5.6 TB/s (with q, k and v mixed in a block 87 us,
// one head a group 93 us, 8 channels a lane, scalar arithmetic and no loads ahead 133 us); the
// same k and v alone: 21 us (19 us with ue8m0 scales, which need no division); norm and rotation
// of 4096 tokens of 32 + 8 heads: 16.3 us.  Three blocks an SM leave 80 registers: 36 of the 48
// variants that write the cache and rotate spill 4 to 12 bytes a thread, the one measured 12.
constexpr int kWriteAhead = 2;

template <int LPH, int U, int ROPE, int FMT, int SF, bool CACHE>
__device__ __forceinline__ void write_part(const KvWriteArgs& a, const KvPart& c,
                                           uint4 (&ring)[kWriteAhead + 1][U][2][256]) {
  const int units = (c.heads + U - 1) / U;
  const int j = threadIdx.x & (LPH - 1);
  const int group = ((int(blockIdx.x) - c.begin) * 256 + int(threadIdx.x)) / LPH;
  const int step = c.blocks * (256 / LPH) / units;         // tokens at a time; at least one (host)
  const int t0 = group / units;
  const int h0 = (group - t0 * units) * U;
  const int left = c.heads - h0;                           // heads of the unit: U, or fewer at the end
  const bool on = t0 < step && j * 16 < a.D;
  // the runs, and whether and by which pairs they turn
  int ca = 8 * j, cb = a.D / 2 + 8 * j, pa = 0, pb = 0;
  bool ta = false, tb = false;
  if (ROPE == kRopeHalves) {
    ta = tb = 16 * j < a.R;
    pa = 8 * j;
    pb = 8 * j + 4;
    ca = ta ? 8 * j : 16 * j;
    cb = ta ? a.R / 2 + 8 * j : 16 * j + 8;
  } else if (ROPE == kRopeInterleaved) {
    ta = ca < a.R;
    tb = cb < a.R;
    pa = ca / 2;
    pb = cb / 2;
  }
  const bool norm = c.w != nullptr;
  uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
  if (norm && on) {
    wa = __ldg(reinterpret_cast<const uint4*>(c.w + ca));
    wb = __ldg(reinterpret_cast<const uint4*>(c.w + cb));
  }
  // tokens ahead, in shared memory: every thread reads only what it copied itself
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (!on || u >= left)
      for (int i = 0; i <= kWriteAhead; ++i)
        ring[i][u][0][threadIdx.x] = ring[i][u][1][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  auto fetch = [&](int t, int s) {
    if (on && t < a.T) {
      const uint16_t* p = c.src + t * c.tok + h0 * c.head;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < left) {
          cp_async16(smem_u32(&ring[s][u][0][threadIdx.x]), p + u * c.head + ca);
          cp_async16(smem_u32(&ring[s][u][1][threadIdx.x]), p + u * c.head + cb);
        }
      }
    }
    cp_async_commit();
  };
  int64_t pos = 0, slot = -1;
  auto fetch_index = [&](int t) {
    if (on && t < a.T) {
      if (ROPE != kRopeNone && (ta || tb)) pos = __ldg(a.pos + t);
      if (CACHE) slot = __ldg(a.slots + t);
    }
  };
  fetch_index(t0);
#pragma unroll
  for (int i = 0; i < kWriteAhead; ++i) fetch(t0 + i * step, i);
  int s = 0;
  // every lane of a warp walks the same number of steps (the shuffles below need them all)
  for (int tb0 = 0; tb0 < a.T; tb0 += step) {
    const int t = tb0 + t0;
    const bool live = on && t < a.T;
    fetch(t + kWriteAhead * step, s == 0 ? kWriteAhead : s - 1);
    // HALVES: the eight pairs' cosines and sines; INTERLEAVED: four of run a, four of run b
    float4 cs[2], sn[2];
    if (ROPE != kRopeNone) {
      const int64_t p = min(max(pos, int64_t(0)), a.max_pos - 1);
      const float* row = a.cos_sin + p * a.R;
      if (ta && live) {
        cs[0] = __ldg(reinterpret_cast<const float4*>(row + pa));
        sn[0] = __ldg(reinterpret_cast<const float4*>(row + a.R / 2 + pa));
      }
      if (tb && live) {
        cs[1] = __ldg(reinterpret_cast<const float4*>(row + pb));
        sn[1] = __ldg(reinterpret_cast<const float4*>(row + a.R / 2 + pb));
      }
    }
    // where the token goes in the cache
    uint8_t* code_at = nullptr;
    float* scale_at = nullptr;
    if (CACHE && live && slot >= 0 && slot < a.slot_count) {       // under 2^31 (host)
      const int page = int(slot) / a.P, row = int(slot) - page * a.P;
      code_at = c.codes + page * a.page_stride + row * a.token_stride + h0 * a.head_stride;
      scale_at = c.scales + (int64_t(page) * a.H + h0) * a.P + row;
    }
    fetch_index(t + step);
    cp_async_wait<kWriteAhead>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 xa = ring[s][u][0][threadIdx.x], xb = ring[s][u][1][threadIdx.x];
      const uint32_t w8[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
      uint64_t y[8];                                       // pairs of channels: run a, run b
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = pack2(bf16_lo(w8[i]), bf16_hi(w8[i]));
      if (norm) {
        uint64_t s0 = mul2(y[0], y[0]), s1 = mul2(y[4], y[4]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s0 = fma2(y[i], y[i], s0);
          s1 = fma2(y[4 + i], y[4 + i], s1);
        }
        const float2 f0 = unpack2(s0), f1 = unpack2(s1);
        float ss = (f0.x + f0.y) + (f1.x + f1.y);
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
        const uint32_t g8[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = mul2(mul2(y[i], pack2(r, r)), pack2(bf16_lo(g8[i]), bf16_hi(g8[i])));
      }
      if (ROPE != kRopeNone) {
        const float c8[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
        const float s8[8] = {sn[0].x, sn[0].y, sn[0].z, sn[0].w, sn[1].x, sn[1].y, sn[1].z, sn[1].w};
        if (ROPE == kRopeHalves) {
          if (ta) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t cp = pack2(c8[2 * i], c8[2 * i + 1]), sp = pack2(s8[2 * i], s8[2 * i + 1]);
              const uint64_t sm = pack2(-s8[2 * i], -s8[2 * i + 1]), m0 = y[i], m1 = y[4 + i];
              y[i] = fma2(m1, sm, mul2(m0, cp));
              y[4 + i] = fma2(m0, sp, mul2(m1, cp));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i < 4 ? ta : tb) {
              const float2 m = unpack2(y[i]);
              y[i] = fma2(pack2(m.y, m.x), pack2(-s8[i], s8[i]), mul2(y[i], pack2(c8[i], c8[i])));
            }
          }
        }
      }
      if (CACHE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = unpack2(y[i]);
          m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (code_at != nullptr && u < left) {
          const GroupScale<FMT, SF> sc(m);
          uint32_t q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 v = unpack2(sc.apply2(y[i]));
            q[i] = cvt2<FMT>(v.x, v.y);
          }
          uint8_t* at = code_at + u * a.head_stride;
          *reinterpret_cast<uint2*>(at + ca) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
          *reinterpret_cast<uint2*>(at + cb) = make_uint2(q[4] | (q[5] << 16), q[6] | (q[7] << 16));
          if (j == 0) scale_at[u * a.P] = sc.s;
        }
      } else if (live && u < left) {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = unpack2(y[i]);
          r[i] = bf16x2(v.x, v.y);
        }
        uint16_t* at = c.out + t * c.out_tok + (h0 + u) * c.out_head;
        *reinterpret_cast<uint4*>(at + ca) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(at + cb) = make_uint4(r[4], r[5], r[6], r[7]);
      }
    }
    s = s == kWriteAhead ? 0 : s + 1;
  }
}

// CACHE: whether any part goes into the cache.
template <int LPH, int U, int ROPE, int FMT, int SF, bool CACHE>
__global__ void __launch_bounds__(256, 3) k_norm_rope_write(const __grid_constant__ KvWriteArgs a) {
  __shared__ uint4 ring[kWriteAhead + 1][U][2][256];
  pdl_wait();
  pdl_trigger();
  int i = 0;
  while (i + 1 < a.parts && int(blockIdx.x) >= a.part[i + 1].begin) ++i;
  const KvPart& c = a.part[i];
  if (!CACHE || c.out != nullptr) {
    write_part<LPH, U, ROPE, FMT, SF, false>(a, c, ring);
  } else if constexpr (CACHE) {
    if (ROPE == kRopeNone || c.turn) write_part<LPH, U, ROPE, FMT, SF, true>(a, c, ring);
    else write_part<LPH, U, kRopeNone, FMT, SF, true>(a, c, ring);
  }
}

// ------------------------------------------------------------------- read back
// Row r of the outputs is token r - offsets[b] of the sequence b whose range holds r.  A block
// takes a run of rows, its warps in turns, so that what it reads and writes at a time lies
// together; a warp searches the offsets once and reads the table once a page.  Its steps are
// slices of 128 16-channel chunks of a row (k's heads, then v's), four chunks a lane, and the next
// step's codes are loaded before this one's are converted.  Rows whose page is not in the cache
// are zeros; rows outside every range are not written.
// Bound by memory, two thirds of it the bf16 stores: 32 contexts of up to 4096 tokens, 8 heads
// of 128: 74 us, 5.5 TB/s (92 us with two 16-byte stores in place of one of 32 bytes, 79 us with
// runs of rows per warp).
struct KvReadArgs {
  KvCache c;
  const int32_t* table;     // [B][max_pages]
  const int32_t* offsets;   // [B + 1]
  uint16_t* ko;             // bf16 [rows][H][D]
  uint16_t* vo;
  int64_t table_stride, max_pages, rows;
  int B;
  uint32_t cph_magic;       // ceil(2^32 / (D / 16)): quotients by multiplication; 0 for D = 16
  int run;                  // rows per block
};

// 4 codes -> 4 fp32 values times s, as two bf16 pairs.
template <int FMT>
__device__ __forceinline__ uint2 dec4(uint32_t w, float s) {
  uint32_t h0, h1;
  if (FMT == kE4M3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(uint16_t(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(uint16_t(w >> 16)));
  } else {
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h0) : "h"(uint16_t(w)));
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h1) : "h"(uint16_t(w >> 16)));
  }
  const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&h0));
  const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&h1));
  return make_uint2(bf16x2(f0.x * s, f0.y * s), bf16x2(f1.x * s, f1.y * s));
}

// 32 bytes in one store (two 16-byte stores would each write half of every sector).
__device__ __forceinline__ void store32(void* p, uint2 a, uint2 b, uint2 c, uint2 d) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(b.x),
               "r"(b.y), "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y)
               : "memory");
}

template <int FMT>
__global__ void __launch_bounds__(256, 2) k_kv_read(const KvReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int cph = a.c.D / 16;                 // chunks per head
  const int chunks = a.c.H * cph;             // of k, and as many of v
  const int64_t first_row = max(int64_t(blockIdx.x) * a.run, int64_t(__ldg(a.offsets)));
  const int64_t end = min(min((int64_t(blockIdx.x) + 1) * a.run, a.rows), int64_t(__ldg(a.offsets + a.B)));
  int64_t r = first_row + (threadIdx.x >> 5);
  if (r >= end) return;
  int b = 0;                                  // offsets[b] <= r < offsets[b + 1]
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (__ldg(a.offsets + mid) <= r) b = mid;
    else hi = mid;
  }
  int64_t next_b = __ldg(a.offsets + b + 1);
  auto token = [&]() { return int(min(r - int64_t(__ldg(a.offsets + b)), int64_t(INT32_MAX))); };
  int tok = token();
  int pi = tok / a.c.P, row = tok - pi * a.c.P;
  int64_t page;
  auto turn = [&]() {                         // the page of the current token
    page = pi < a.max_pages ? __ldg(a.table + b * a.table_stride + pi) : -1;
    if (page >= a.c.pages) page = -1;
  };
  turn();
  int first = 0;                              // the step's first chunk
  uint4 q[4];
  float s[4];
  auto load = [&]() {
    const int64_t src = page * a.c.page_stride + row * a.c.token_stride;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = first + u * 32 + lane;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      s[u] = 0.0f;
      if (page >= 0 && i < 2 * chunks) {
        const bool is_v = i >= chunks;
        const int c = is_v ? i - chunks : i;
        const int h = a.cph_magic != 0u ? int(__umulhi(uint32_t(c), a.cph_magic)) : c;
        q[u] = ldg_stream(reinterpret_cast<const uint4*>((is_v ? a.c.v : a.c.k) + src + h * a.c.head_stride +
                                                         (c - h * cph) * 16));
        s[u] = __ldg((is_v ? a.c.vs : a.c.ks) + (page * a.c.H + h) * a.c.P + row);
      }
    }
  };
  load();
  while (true) {
    uint4 v[4];
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = q[u];
      f[u] = s[u];
    }
    const int64_t at = r;
    const int from = first;
    first += 128;
    if (first >= 2 * chunks) {                // the next row
      first = 0;
      r += 8;
      row += 8;
      if (r < end) {
        if (r >= next_b) {                    // the sequence that has this row
          do next_b = __ldg(a.offsets + ++b + 1);
          while (r >= next_b);
          tok = token();
          pi = tok / a.c.P;
          row = tok - pi * a.c.P;
          turn();
        } else if (row >= a.c.P) {            // pages hold at least eight rows
          row -= a.c.P;
          ++pi;
          turn();
        }
      }
    }
    const bool more = r < end;
    if (more) load();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = from + u * 32 + lane;
      if (i < 2 * chunks) {
        const bool is_v = i >= chunks;
        uint16_t* dst = (is_v ? a.vo : a.ko) + (at * chunks + (is_v ? i - chunks : i)) * 16;
        const uint2 y0 = dec4<FMT>(v[u].x, f[u]), y1 = dec4<FMT>(v[u].y, f[u]);
        const uint2 y2 = dec4<FMT>(v[u].z, f[u]), y3 = dec4<FMT>(v[u].w, f[u]);
        store32(dst, y0, y1, y2, y3);
      }
    }
    if (!more) break;
  }
}

}  // namespace fp8lin
