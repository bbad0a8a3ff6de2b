// Per-head RMSNorm and rotation of query and key rows, and their store into cache pages
// (include/dg_paged.h: dg_qk_norm_rope, dg_paged_append).
//
// A head row x of h channels becomes y = x * rsqrt(mean(x^2) + eps) * gain, then pair
// (i, i + h/2) turns by position * base^(-2i/h).  The angle is kept in turns: position
// times the pair's 64-bit fraction of a turn, modulo 2^64, is exact, and its top 32 bits go
// through sincospif, so position 2^30 costs no more precision than position 1.
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
  float eps;            // < 0: no norm
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

template <class T, bool APPEND>
__global__ void __launch_bounds__(256)
    head_rows_kernel(const RowsParams p, const __grid_constant__ dg_rope rope) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(w / p.parts), part = (int)(w % p.parts);
  if (t >= p.n) return;  // warp-uniform
  const int l = lane & ((1 << p.lg) - 1);
  const int half = p.h >> 1;
  const bool on = 8 * l < half;  // lanes of a head beyond h/16 idle

  long long pos;
  long long slot = -1;  // byte offset of the row's slot, -1: not stored
  if (APPEND) {
    const int b = find_seq(p.q_start, p.B, t, lane);
    if (b >= p.B) return;
    const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
    if (t < q0) return;
    if (q0 < 0 || q1 > p.n || q1 <= t || q1 - q0 > p.max_q || kv < 0 ||
        kv > (long long)p.max_pages << p.page_log2) {
      if (lane == 0 && p.err) atomicOr(p.err, DG_PAGED_BAD_BATCH);
      return;
    }
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

  float cs[8], sn[8];
  if (p.rotate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned long long turn =
          on ? (unsigned long long)pos * rope.turns[8 * l + i] : 0ull;
      sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f /* 2^-31 */, &sn[i], &cs[i]);
    }
  }

  const int per = 32 >> p.lg;
  const int heads = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int hl = lane >> p.lg;
  for (int it = 0; it < p.iters; ++it) {
    const int j0 = (part * p.iters + it) * per;
    if (j0 >= heads) break;
    const int j = j0 + hl;
    // which of q, k, v this head is (0, 1, 2) and its index there
    const int kind = j < p.hq ? 0 : (!APPEND || j < p.hq + p.hkv) ? 1 : 2;
    const int jj = kind == 0 ? j : kind == 1 ? j - p.hq : j - p.hq - p.hkv;
    const bool act = on && j < heads && (!APPEND || kind == 0 || slot >= 0);
    const HeadsDev& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    T a[8], c[8];
    if (act) {
      const T* x = reinterpret_cast<const T*>(src.p + t * src.ts + jj * src.hs);
      ld8(x + 8 * l, a);
      ld8(x + half + 8 * l, c);
    }
    T* dst = nullptr;
    if (act) {
      char* base;
      if (kind == 0)
        base = p.qo.p + t * p.qo.ts + jj * p.qo.hs;
      else if (!APPEND)
        base = p.ko.p + t * p.ko.ts + jj * p.ko.hs;
      else
        base = (kind == 1 ? p.kc : p.vc) + slot + jj * p.hs;
      dst = reinterpret_cast<T*>(base);
    }
    if (kind != 2) {
      float u[8], w2[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = act ? widen(a[i]) : 0.f;
        w2[i] = act ? widen(c[i]) : 0.f;
      }
      if (p.eps >= 0.f) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += u[i] * u[i] + w2[i] * w2[i];
        // a warp's heads may be of different kinds, so each reduces within its own lanes
        // (at most 16: h <= 256)
        const unsigned m = ((1u << (1 << p.lg)) - 1u) << (hl << p.lg);
        for (int o = 1 << p.lg >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(m, ss, o);
        const float r = 1.0f / sqrtf(ss / (float)p.h + p.eps);
        const T* gain = reinterpret_cast<const T*>(kind == 0 ? p.qg : p.kg);
        if (gain && act) {
          T g0[8], g1[8];
          ld8(gain + 8 * l, g0);
          ld8(gain + half + 8 * l, g1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] *= r * widen(g0[i]);
            w2[i] *= r * widen(g1[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] *= r;
            w2[i] *= r;
          }
        }
      }
      if (p.rotate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x0 = u[i], x1 = w2[i];
          u[i] = x0 * cs[i] - x1 * sn[i];
          w2[i] = x1 * cs[i] + x0 * sn[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = narrow<T>(u[i]);
        c[i] = narrow<T>(w2[i]);
      }
    }
    if (act) {
      st8(dst + 8 * l, a);
      st8(dst + half + 8 * l, c);
    }
  }
}

}  // namespace dg
