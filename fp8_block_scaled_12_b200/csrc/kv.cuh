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

struct KvWriteArgs {
  const uint16_t* q;        // [T][Hq][D], token and head strides in elements
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
  uint16_t* qo;             // bf16 outputs (qo may be q, ko may be k)
  uint16_t* ko;
  int64_t qo_tok, qo_head, ko_tok, ko_head;
  const uint16_t* wq;       // norm weights bf16 [D]; nullptr: no norm
  const uint16_t* wk;
  const float* cos_sin;     // [max_pos][R]
  const int64_t* pos;       // [T]
  const int64_t* slots;     // [T]
  KvCache c;
  int64_t T, max_pos;
  float eps;
  int Hq, Hk, Hv, D, R;     // heads of q, k and v that this call handles
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// LPH lanes own one head of one token, 8 channels each as two runs of 4 (a, b): adjacent
// runs, or, for pairs (i, R/2 + i), the two runs that rotate into each other, so that the
// rotation never leaves a thread.  A group of lanes takes U consecutive heads of a token:
// their loads are in flight together and share the token's cosines and sines.
template <int LPH, int U, int ROPE, int FMT, int SF, bool CACHE>
__global__ void __launch_bounds__(256) k_norm_rope_write(const KvWriteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int heads = a.Hq + a.Hk + a.Hv;
  const int hb = (heads + U - 1) / U;
  const int j = threadIdx.x & (LPH - 1);
  const int64_t total = a.T * hb;
  const int64_t stride = int64_t(gridDim.x) * (256 / LPH);
  const bool lane_on = j * 8 < a.D;
  int ca = 8 * j, cb = 8 * j + 4;
  const bool turned = ROPE != kRopeNone && 8 * j < a.R;
  if (ROPE == kRopeHalves && turned) {
    ca = 4 * j;
    cb = a.R / 2 + 4 * j;
  }
  // every lane of a warp walks the same number of steps (the shuffles below need them all)
  for (int64_t i0 = int64_t(blockIdx.x) * (256 / LPH); i0 < total; i0 += stride) {
    const int64_t item = i0 + threadIdx.x / LPH;
    const bool item_on = item < total;
    const int64_t t = item_on ? item / hb : 0;
    const int h0 = item_on ? int(item - t * hb) * U : heads;
    int64_t slot = -1;
    if (CACHE && item_on) slot = __ldg(a.slots + t);
    uint2 x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u;
      x[u][0] = x[u][1] = make_uint2(0u, 0u);
      if (h < heads && lane_on) {
        const uint16_t* p = h < a.Hq ? a.q + t * a.q_tok + h * a.q_head
                            : h < a.Hq + a.Hk ? a.k + t * a.k_tok + (h - a.Hq) * a.k_head
                                              : a.v + t * a.v_tok + (h - a.Hq - a.Hk) * a.v_head;
        if (ROPE == kRopeHalves) {
          x[u][0] = *reinterpret_cast<const uint2*>(p + ca);
          x[u][1] = *reinterpret_cast<const uint2*>(p + cb);
        } else {
          const uint4 y = *reinterpret_cast<const uint4*>(p + ca);
          x[u][0] = make_uint2(y.x, y.y);
          x[u][1] = make_uint2(y.z, y.w);
        }
      }
    }
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ROPE != kRopeNone && turned && item_on && h0 < a.Hq + a.Hk) {
      const int64_t p = min(max(__ldg(a.pos + t), int64_t(0)), a.max_pos - 1);
      const float* row = a.cos_sin + p * a.R + 4 * j;
      cs = __ldg(reinterpret_cast<const float4*>(row));
      sn = __ldg(reinterpret_cast<const float4*>(row + a.R / 2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u;
      const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk, is_v = !is_q && !is_k && h < heads;
      const uint32_t w4[4] = {x[u][0].x, x[u][0].y, x[u][1].x, x[u][1].y};
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(w4[i]);
        y[2 * i + 1] = bf16_hi(w4[i]);
      }
      const uint16_t* wn = is_q ? a.wq : is_k ? a.wk : nullptr;
      // the norm's sum needs every lane of the group, so the whole warp takes part
      if (__any_sync(0xffffffffu, wn != nullptr)) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (wn != nullptr && lane_on) {
          const float r = 1.0f / sqrtf(ss / float(a.D) + a.eps);
          const uint2 wa = __ldg(reinterpret_cast<const uint2*>(wn + ca));
          const uint2 wb = __ldg(reinterpret_cast<const uint2*>(wn + cb));
          const uint32_t v4[4] = {wa.x, wa.y, wb.x, wb.y};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = y[2 * i] * r * bf16_lo(v4[i]);
            y[2 * i + 1] = y[2 * i + 1] * r * bf16_hi(v4[i]);
          }
        }
      }
      if (ROPE != kRopeNone && turned && (is_q || is_k)) {
        const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ia = ROPE == kRopeInterleaved ? 2 * i : i, ib = ROPE == kRopeInterleaved ? 2 * i + 1 : 4 + i;
          const float n0 = y[ia], n1 = y[ib];
          y[ia] = n0 * c[i] - n1 * s[i];
          y[ib] = n1 * c[i] + n0 * s[i];
        }
      }
      if (CACHE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if ((is_k || is_v) && slot >= 0 && slot < a.c.pages * a.c.P) {
          const GroupScale<FMT, SF> sc(m);
          uint32_t c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = cvt2<FMT>(sc.apply(y[2 * i]), sc.apply(y[2 * i + 1]));
          const uint2 code = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
          const int64_t page = slot / a.c.P, row = slot - page * a.c.P;
          const int hc = is_k ? h - a.Hq : h - a.Hq - a.Hk;
          uint8_t* dst = (is_k ? a.c.k : a.c.v) + page * a.c.page_stride + hc * a.c.head_stride + row * a.c.token_stride;
          if (lane_on) {
            if (ROPE == kRopeHalves) {
              *reinterpret_cast<uint32_t*>(dst + ca) = code.x;
              *reinterpret_cast<uint32_t*>(dst + cb) = code.y;
            } else {
              *reinterpret_cast<uint2*>(dst + ca) = code;
            }
          }
          if (j == 0) (is_k ? a.c.ks : a.c.vs)[(page * a.c.H + hc) * a.c.P + row] = sc.s;
        }
      }
      if ((is_q || (!CACHE && is_k)) && lane_on) {
        uint16_t* p = is_q ? a.qo + t * a.qo_tok + h * a.qo_head : a.ko + t * a.ko_tok + (h - a.Hq) * a.ko_head;
        const uint2 oa = make_uint2(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]));
        const uint2 ob = make_uint2(bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
        if (ROPE == kRopeHalves) {
          *reinterpret_cast<uint2*>(p + ca) = oa;
          *reinterpret_cast<uint2*>(p + cb) = ob;
        } else {
          *reinterpret_cast<uint4*>(p + ca) = make_uint4(oa.x, oa.y, ob.x, ob.y);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- read back
// Row r of the outputs is token r - offsets[b] of the sequence b whose range holds r.  One
// warp per row: a binary search of the offsets, then 16 channels per lane and step of its
// k and v heads.  Rows whose page is not in the cache are zeros; rows outside every range
// are not written.
struct KvReadArgs {
  KvCache c;
  const int32_t* table;     // [B][max_pages]
  const int32_t* offsets;   // [B + 1]
  uint16_t* ko;             // bf16 [rows][H][D]
  uint16_t* vo;
  int64_t table_stride, max_pages, rows;
  int B;
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

template <int FMT>
__global__ void __launch_bounds__(256) k_kv_read(const KvReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int cph = a.c.D / 16;                 // 16-channel chunks per head
  const int chunks = a.c.H * cph;             // of k, and as many of v
  const int64_t nwarp = int64_t(gridDim.x) * 8;
  for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < a.rows; r += nwarp) {
    if (r < __ldg(a.offsets) || r >= __ldg(a.offsets + a.B)) continue;
    int lo = 0, hi = a.B;                     // offsets[lo] <= r < offsets[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.offsets + mid) <= r) lo = mid;
      else hi = mid;
    }
    const int64_t tok = r - __ldg(a.offsets + lo);
    const int64_t pi = tok / a.c.P, row = tok - pi * a.c.P;
    int64_t page = tok >= 0 && pi < a.max_pages ? __ldg(a.table + lo * a.table_stride + pi) : -1;
    const bool ok = page >= 0 && page < a.c.pages;
    const int64_t src = page * a.c.page_stride + row * a.c.token_stride;
    for (int i0 = 0; i0 < 2 * chunks; i0 += 128) {
      uint4 q[4];
      float s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 32 + lane;
        q[u] = make_uint4(0u, 0u, 0u, 0u);
        s[u] = 0.0f;
        if (ok && i < 2 * chunks) {
          const bool is_v = i >= chunks;
          const int c = is_v ? i - chunks : i;
          const int h = c / cph;
          q[u] = ldg_stream(reinterpret_cast<const uint4*>((is_v ? a.c.v : a.c.k) + src + h * a.c.head_stride +
                                                           (c - h * cph) * 16));
          s[u] = __ldg((is_v ? a.c.vs : a.c.ks) + (page * a.c.H + h) * a.c.P + row);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 32 + lane;
        if (i < 2 * chunks) {
          const bool is_v = i >= chunks;
          uint4* dst = reinterpret_cast<uint4*>((is_v ? a.vo : a.ko) + (r * chunks + (is_v ? i - chunks : i)) * 16);
          const uint2 y0 = dec4<FMT>(q[u].x, s[u]), y1 = dec4<FMT>(q[u].y, s[u]);
          const uint2 y2 = dec4<FMT>(q[u].z, s[u]), y3 = dec4<FMT>(q[u].w, s[u]);
          dst[0] = make_uint4(y0.x, y0.y, y1.x, y1.y);
          dst[1] = make_uint4(y2.x, y2.y, y3.x, y3.y);
        }
      }
    }
  }
}

}  // namespace fp8lin
