// Per-head RMSNorm and rotation of query and key rows, and their store into cache pages
// (include/dg_paged.h: dg_qk_norm_rope, dg_paged_append).
//
// A head row x of h channels becomes y = x * rsqrt(mean(x^2) + eps) * gain, then pair
// (i, i + h/2) turns by position * base^(-2i/h).  The angle is kept in turns: position
// times the pair's 64-bit fraction of a turn, modulo 2^64, is exact, and its top 32 bits go
// through sincospif, so position 2^30 costs no more precision than position 1.  sincospif
// takes a float: the angle is cut to 24 bits, at most 2^-25 half turns (9e-8 radians), below
// what 16-bit rows resolve and on a level with the rounding of f32 ones.
//
// Bound by memory: each element is read once and written once, with ~10 operations on it.
// A head is held by h/16 lanes (rounded up to a power of two), each with channels
// 8l .. 8l + 7 of both halves, so that a pair's two channels meet in one thread, every
// access is 16 bytes, and the sum of squares needs log2(h/16) shuffles.  The sines are
// computed once per (token, warp) and used for all of the warp's heads.
#pragma once

#include <cuda_fp16.h>

#include "../../include/dg_paged.h"
#include "k_common.cuh"

namespace dg {

struct HeadsDev {
  char* p;              // element (t, j, 0) at p + t * ts + j * hs (bytes)
  long long ts, hs;
};

struct RowsParams {
  int n;                // rows
  int hq, hkv;          // query heads, key heads (value heads: hkv, append only)
  int h, lg;            // channels; log2 of the lanes that hold a head
  int iters;            // groups of 32 >> lg heads a warp takes
  int parts;            // warps per row
  HeadsDev q, k, v, qo, ko;  // ko: dg_qk_norm_rope only
  const void *qg, *kg;
  float eps, inv_h;     // eps < 0: no norm; 1 / h
  int rotate;
  const int32_t* positions;  // dg_qk_norm_rope
  // append
  char *kc, *vc;        // pages
  long long ps, ts, hs; // page, token and head strides in bytes
  int page_log2, n_pages, max_pages, B, max_q;
  const int32_t *q_start, *kv_len, *table;
  int32_t* err;
};

__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ __half narrow<__half>(float x) {
  return __float2half_rn(x);
}

// Two fp32 values in a register pair, for the packed instructions.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight consecutive elements as four fp32 pairs, and back.
template <class T> __device__ __forceinline__ void widen8(const T (&x)[8], uint64_t (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = f2(widen(x[2 * i]), widen(x[2 * i + 1]));
}
__device__ __forceinline__ void narrow8(const uint64_t (&y)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unf2(y[i], &x[2 * i], &x[2 * i + 1]);
}
__device__ __forceinline__ void narrow8(const uint64_t (&y)[4], bf16 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unf2(y[i], &a, &b);
    reinterpret_cast<__nv_bfloat162*>(x)[i] = __floats2bfloat162_rn(a, b);
  }
}
__device__ __forceinline__ void narrow8(const uint64_t (&y)[4], __half (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unf2(y[i], &a, &b);
    reinterpret_cast<__half2*>(x)[i] = __floats2half2_rn(a, b);
  }
}

// The sequence of row t: how many of q_start[1 .. B] are <= t, by a 32-way search of the
// whole warp (two dependent loads up to 1,024 sequences).  B if t lies behind the last.
__device__ __forceinline__ int find_seq(const int32_t* q_start, int B, int t, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + (lane + 1) * step;
    const unsigned below = __ballot_sync(0xffffffffu, i <= hi && q_start[i] <= t);
    lo += __popc(below) * step;
    hi = min(hi, lo + step);
  }
  const int i = lo + lane + 1;
  return lo + __popc(__ballot_sync(0xffffffffu, i <= hi && q_start[i] <= t));
}

// 64 registers, so that 32 warps an SM hide the loads: loading the next heads ahead took 72 to
// 80 and was slower (23,487 rows appended: 81 to 126 us), more warps with spills as well.
// Blocks of two warps, which make room as soon as their own rows are done (76 us; eight warps
// a block 78).
constexpr int HEAD_ROWS_WARPS = 2;

template <class T, bool APPEND>
__global__ void __launch_bounds__(HEAD_ROWS_WARPS * 32, 32 / HEAD_ROWS_WARPS)
    head_rows_kernel(const RowsParams p, const __grid_constant__ dg_rope rope) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * HEAD_ROWS_WARPS + (threadIdx.x >> 5);  // < 2^32
  const unsigned row_warps = (unsigned)p.n * (unsigned)p.parts;
  if (w >= row_warps) {  // warp-uniform
    // The warps behind the rows' look at the batch, a sequence a lane: rows find their sequence
    // by a search, which passes by chunks that are empty or out of order.
    const unsigned b = (w - row_warps) * 32 + lane;
    if (APPEND && p.err && b < (unsigned)p.B) {
      const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
      if (q0 < 0 || q1 < q0 || q1 > p.n || q1 - q0 > p.max_q || kv < 0 ||
          kv > (long long)p.max_pages << p.page_log2)
        atomicOr(p.err, DG_PAGED_BAD_BATCH);
    }
    return;
  }
  const int t = (int)(w / (unsigned)p.parts), part = (int)(w % (unsigned)p.parts);
  const int l = lane & ((1 << p.lg) - 1), hl = lane >> p.lg, per = 32 >> p.lg;
  const int half = p.h >> 1;
  const bool on = 8 * l < half;  // lanes of a head beyond h/16 idle

  // Groups of `per` heads: the queries', then the keys', then the values' (a group holds one
  // kind, so what depends on it is worked out once a kind).
  const int gq = (p.hq + per - 1) >> (5 - p.lg), gk = (p.hkv + per - 1) >> (5 - p.lg);
  const int g0 = part * p.iters, g1 = min(g0 + p.iters, gq + (APPEND ? 2 : 1) * gk);
  int kind = g0 < gq ? 0 : g0 < gq + gk ? 1 : 2;
  int j = (g0 - (kind == 0 ? 0 : kind == 1 ? gq : gq + gk)) * per + hl;  // this lane's head
  const char* src;  // this lane's first channels of it
  auto source = [&] {
    const HeadsDev& x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    src = x.p + t * x.ts + j * x.hs + 8 * l * (int)sizeof(T);
  };
  auto load = [&](T(&a)[8], T(&c)[8]) {
    if (on && j < (kind == 0 ? p.hq : p.hkv)) {
      ld8(reinterpret_cast<const T*>(src), a);
      ld8(reinterpret_cast<const T*>(src) + half, c);
    }
  };
  // the row is on its way while its place and its sines are worked out
  T a[8], c[8];
  source();
  load(a, c);

  long long pos;
  long long slot = -1;  // byte offset of the row's slot, -1: not stored
  if (APPEND) {
    const int b = find_seq(p.q_start, p.B, t, lane);
    if (b >= p.B) return;
    const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
    if (t < q0) return;
    if (q0 < 0 || q1 > p.n || q1 <= t || q1 - q0 > p.max_q || kv < 0 ||
        kv > (long long)p.max_pages << p.page_log2)
      return;
    pos = (long long)kv - (q1 - q0) + (t - q0);
    if (pos >= 0) {
      const int page = p.table[(long long)b * p.max_pages + (pos >> p.page_log2)];
      if (page >= 0 && page < p.n_pages)
        slot = page * p.ps + (pos & ((1 << p.page_log2) - 1)) * p.ts;
      else if (lane == 0 && p.err)
        atomicOr(p.err, DG_PAGED_BAD_PAGE);
    }
  } else {
    pos = p.rotate ? p.positions[t] : 0;
  }

  // Sines of this lane's eight pairs.  The lanes at the same place of the warp's heads need
  // the same eight: each works out 8 / per of them (one at least), and they exchange.
  uint64_t cs[4], sn[4];
  if (p.rotate && g0 < gq + gk) {
    const int each = max(8 / per, 1);  // 1, 2 or 4
    float c4[4], s4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= each) break;
      const int pair = 8 * l + (hl * each + i & 7);
      // through memory: a constant-bank read of 32 different words would be 32 reads
      unsigned long long f;
      asm("ld.u64 %0, [%1];" : "=l"(f) : "l"(&rope.turns[on ? pair : 0]));
      const unsigned long long turn = (unsigned long long)pos * f;
      sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f /* 2^-31 */, &s4[i], &c4[i]);
    }
    float c8[8], s8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = (i / each << p.lg) | l;
      const float s0 = each == 1 ? s4[0] : each == 2 ? s4[i & 1] : s4[i & 3];
      const float c0 = each == 1 ? c4[0] : each == 2 ? c4[i & 1] : c4[i & 3];
      s8[i] = __shfl_sync(0xffffffffu, s0, from);
      c8[i] = __shfl_sync(0xffffffffu, c0, from);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = f2(c8[2 * i], c8[2 * i + 1]);
      sn[i] = f2(s8[2 * i], s8[2 * i + 1]);
    }
  }

  for (int g = g0; g < g1; ++kind, j = hl) {
    if (g > g0) {
      source();
      load(a, c);
    }
    const int heads = kind == 0 ? p.hq : p.hkv;
    const int end = min(g1, kind == 0 ? gq : kind == 1 ? gq + gk : gq + 2 * gk);
    if (APPEND && kind > 0 && slot < 0) return;  // keys and values have nowhere to go
    long long src_step, dst_step;
    char* dst;
    if (kind == 0) {
      dst = p.qo.p + t * p.qo.ts;
      dst_step = p.qo.hs;
      src_step = p.q.hs;
    } else if (APPEND) {
      dst = (kind == 1 ? p.kc : p.vc) + slot;
      dst_step = p.hs;
      src_step = kind == 1 ? p.k.hs : p.v.hs;
    } else {
      dst = p.ko.p + t * p.ko.ts;
      dst_step = p.ko.hs;
      src_step = p.k.hs;
    }
    dst += j * dst_step + 8 * l * (int)sizeof(T);
    src_step *= per;
    dst_step *= per;
    const T* gain = reinterpret_cast<const T*>(kind == 0 ? p.qg : p.kg) + (on ? 8 * l : 0);
    const bool gained = kind < 2 && (kind == 0 ? p.qg : p.kg) != nullptr;
#pragma unroll 1
    while (true) {
      if (kind < 2) {
        uint64_t u[4], v[4];  // the two halves' channels
        widen8(a, u);
        widen8(c, v);
        if (p.eps >= 0.f) {
          uint64_t s2 = mul2(u[0], u[0]), s3 = mul2(v[0], v[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            s2 = fma2(u[i], u[i], s2);
            s3 = fma2(v[i], v[i], s3);
          }
          float x, y;
          unf2(add2(s2, s3), &x, &y);
          float ss = on ? x + y : 0.f;  // idle lanes hold nothing
          for (int o = 1 << p.lg >> 1; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * p.inv_h + p.eps);
          const uint64_t r2 = f2(r, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = mul2(u[i], r2);
            v[i] = mul2(v[i], r2);
          }
          if (gained) {  // from L1 each time: registers held through the loop cost more
            T g8[8];
            uint64_t e[4];
            ld8(gain, g8);
            widen8(g8, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = mul2(u[i], e[i]);
            ld8(gain + half, g8);
            widen8(g8, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], e[i]);
          }
        }
        if (p.rotate) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t x = u[i];
            u[i] = sub2(mul2(x, cs[i]), mul2(v[i], sn[i]));
            v[i] = fma2(v[i], cs[i], mul2(x, sn[i]));
          }
        }
        narrow8(u, a);
        narrow8(v, c);
      }
      if (on && j < heads) {
        st8(reinterpret_cast<T*>(dst), a);
        st8(reinterpret_cast<T*>(dst) + half, c);
      }
      if (++g >= end) break;
      j += per;
      src += src_step;
      dst += dst_step;
      load(a, c);
    }
  }
}

}  // namespace dg
