// Attention of chunks of new tokens over a cache in pages (include/dg_paged.h:
// dg_paged_attention).
//
// One warp per (row, query head): a pass over the visible keys with the running maximum m
// and sum l of the softmax, o = o 2^(m_old - m) + 2^(s - m) v.  Simple and right for every
// shape; each key is read again by every row.
#pragma once

#include "k_paged_rows.cuh"

namespace dg {

struct PagedAttnParams {
  const char *k, *v;
  long long ps, ts, hs;  // page, token and head strides in bytes
  int page_log2, n_pages, max_pages, B, n, max_q;
  const int32_t *q_start, *kv_len, *table;
  HeadsDev q;
  int hq, hkv;
  int causal;
  const uint8_t* causal_seq;
  int window;
  float scale_log2;
  void* out;
  float* lse;
  int32_t* err;
};

template <class T, int H>
__global__ void __launch_bounds__(256) paged_attn_rows_kernel(const PagedAttnParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(w / p.hq), j = (int)(w % p.hq);
  if (t >= p.n) return;
  const int b = find_seq(p.q_start, p.B, t, lane);
  if (b >= p.B) return;
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
  if (t < q0) return;
  if (q0 < 0 || q1 > p.n || q1 <= t || q1 - q0 > p.max_q || kv < 0 ||
      kv > (long long)p.max_pages << p.page_log2) {
    if (lane == 0 && p.err) atomicOr(p.err, DG_PAGED_BAD_BATCH);
    return;
  }
  const int past = kv - (q1 - q0), pos = past + (t - q0);
  const bool causal = p.causal_seq ? p.causal_seq[b] != 0 : p.causal != 0;
  const int hi = causal ? min(kv, pos + 1) : kv;
  const int lo = p.window ? max(0, (causal ? pos + 1 : past) - p.window) : 0;
  constexpr int D = H / 32;
  const int g = j / (p.hq / p.hkv);
  float q[D], o[D];
  const T* qp = reinterpret_cast<const T*>(p.q.p + t * p.q.ts + j * p.q.hs) + D * lane;
#pragma unroll
  for (int i = 0; i < D; ++i) {
    q[i] = widen(qp[i]) * p.scale_log2;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int s = lo; s < hi; ++s) {
    const int page = p.table[(long long)b * p.max_pages + (s >> p.page_log2)];
    if (page < 0 || page >= p.n_pages) {
      bad = true;
      break;
    }
    const long long at =
        page * p.ps + (s & ((1 << p.page_log2) - 1)) * p.ts + g * p.hs + D * lane * sizeof(T);
    const T* kp = reinterpret_cast<const T*>(p.k + at);
    const T* vp = reinterpret_cast<const T*>(p.v + at);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < D; ++i) x += q[i] * widen(kp[i]);
    x = warp_sum(x);
    const float mn = fmaxf(m, x), a = exp2f(m - mn), e = exp2f(x - mn);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < D; ++i) o[i] = o[i] * a + e * widen(vp[i]);
    m = mn;
  }
  if (bad && lane == 0 && p.err) atomicOr(p.err, DG_PAGED_BAD_PAGE);
  const float nan = __int_as_float(0x7fc00000);
  const float inv = bad ? nan : l == 0.f ? 0.f : 1.f / l;
  T* op = reinterpret_cast<T*>(p.out) + ((long long)t * p.hq + j) * H + D * lane;
#pragma unroll
  for (int i = 0; i < D; ++i) op[i] = narrow<T>(o[i] * inv);
  if (p.lse && lane == 0)
    p.lse[(long long)t * p.hq + j] =
        bad ? nan : l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace dg
