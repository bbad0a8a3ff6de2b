// Attention of chunks of new tokens over a cache in pages (include/dg_paged.h:
// dg_paged_attention) on tcgen05.
//
//   out = softmax(scale Q K^T) V, one pass over the keys with the running maximum m and sum
//   l of each row; P = 2^(s - m) is unnormalised and the division comes last.
//
// Rows.  The G = Hq / Hkv query heads of a key head share its keys, so a tile's 128 rows are
// T = 128 / G tokens times G heads, and a single token fills G rows.  An ITEM is a sequence,
// a key head and up to 2 T tokens, with the key tiles (128 keys) that any of its rows sees.
// With more than T tokens its two row tiles take every key tile (a PAIR); with fewer its one
// row tile is computed as two streams, the even and the odd key tiles (SOLO), and the two
// meet at the end.  Either way two softmax warpgroups work while the tensor cores fill the
// other's scores.
//
// Split.  All items form one line, each as long as its key tiles plus PA_ITEM (what filling
// and emptying the pipeline for it costs, in tiles); 148 CTAs take equal contiguous parts of
// it, so no length mix leaves SMs idle.  (Items that are all alike stay whole where that costs
// less than cutting them: eight canvases' 128 items of 10 tiles, 47 -> 38 us.)  A CTA's part
// is a run of whole items with a cut one at either end; cut pieces leave (m, l, O) in the
// workspace and paged_merge_kernel adds an item's pieces in the order of the line (the same
// bits every time).  Each CTA finds its part from the lengths on the device: no host plan, and
// a captured graph follows them.
//
// CTA.  Warps 0-3 and 4-7: the streams' softmax, a thread a row (TMEM lane = row).  Warp 8:
// MMA issue for both streams in turn, which keeps one's softmax under the other's products
// (with a warp for each the streams fell into step, 5,100 cycles a pair of tiles).  Warps 9
// and 11: TMA of keys and rows, and of values.  Warp 10: waits for tiles on the MMA warp's
// behalf.  S (128 columns) and O of both
// streams fill TMEM; P takes S's place as the A operand of O += P V.  K and V tiles pass
// through one ring of slots in the order of their first use.  O is rescaled only when a row's
// maximum has grown by 2^8, by its own warp; until then P's exponents are taken against the
// older maximum, which the final division cancels.  P is rounded to the cache's type, as the
// tensor cores take it, while l adds the fp32 weights: half a step of each weight (normal
// rows: 0.0023 of the output's norm away from 64 bits in bf16, 0.00028 in f16; 0.0017 and
// 0.00021 with fp32 weights, the output's own rounding).
//
// Bound.  Single tokens and drafts read each visible key and value once: memory (64 sequences
// of up to 16,384 keys: 203 us for 1.24 GB, 6.1 TB/s, 0.93 of the measured copy rate, from
// pages of 16 tokens, 2 KB a box; 237 us, 5.2 TB/s, 0.80 in a loop of a second, in which the
// power cap takes the SMs to 1,480 MHz).  Long chunks: a pair of tiles (128 keys of 2 x 128
// rows) takes the tensor cores 2,050 cycles and the SFU's exponentials as long; here it takes
// about 3,200, since a stream's next scores need the columns its weights stand in, so that
// softmax and products of one stream follow each other (8,192 causal tokens, 16 heads of 128:
// 240 to 250 us, 1,100 to 1,150 TFLOP/s, 0.66 to 0.69 of the measured cuBLAS burst rate; 276 us,
// 996 TFLOP/s, 0.60 in a loop of a second, at 1,640 MHz).  Short work: the first scores come
// 9,500 cycles after the start (lengths, plan, page table, keys, and instructions that no one
// has run yet), the last rows leave 4,000 after theirs.
#pragma once

#include "k_paged_rows.cuh"
#include "tc_ptx.cuh"

namespace dg {

constexpr int PA_CTAS = 148;
constexpr int PA_THREADS = 384;  // 12 warps: 8 softmax, MMA, keys, tile watch, values
constexpr int PA_KT = 128;                 // keys a tile
constexpr int PA_ITEM = 2;                 // an item's fixed cost in tiles
constexpr int PA_CUT = 2;                  // no cut leaves fewer tiles on a side
constexpr int PA_PART = 2;                 // shortest part of the line
constexpr int PA_MERGE = 5;                // what cutting items costs a call, in tiles
constexpr uint32_t PA_CHUNK = 128 * 128;   // 128 rows of 64 channels

template <int H> struct PagedCfg {
  static constexpr int CH = H / 64;                 // 64-channel chunks
  static constexpr uint32_t TILE = CH * PA_CHUNK;   // a Q, K or V tile
  static constexpr int SLOTS = H == 128 ? 4 : 8;
  static constexpr size_t SMEM =
      1024 + (2 + SLOTS) * TILE + 768 /* barriers, plan */ + 2 * 128 * 8 /* m, l */ +
      8 * 2048 /* output staging */;
};

struct PagedAttnParams {
  int page_log2, n_pages, max_pages, B, n, max_q;
  const int32_t *q_start, *kv_len, *table;
  int hq, hkv, G, T;
  int causal;
  const uint8_t* causal_seq;
  int window;
  float scale_log2;
  void* out;
  float* lse;
  int32_t* err;
  uint64_t wait_ns;  // limit of every wait
  int stall;         // != 0 (tests of the way out only): no values are loaded
  // workspace
  int part_rows;  // rows of a piece
  float4* part_o;   // [PA_CTAS][2][H / 4][part_rows]: a warp's rows are contiguous
  float2* part_ml;  // [PA_CTAS][2][part_rows]
  struct PagedRec* rec;  // [PA_CTAS]
};

// An item whose first piece is CTA c's second slot; the others are the first slots of
// c + 1 .. last.
struct PagedRec {
  int valid, last, row0, ntok, g, pad_[3];
};

struct PagedSeq {
  int b, q0, ql, past, kv, causal;
};

// Sequence b, with ql = 0 where its numbers are out of range: bit 0 then, and bit 1 where
// q_start decreases (paged_plan then leaves the whole batch out).
__device__ __forceinline__ int paged_seq(const PagedAttnParams& p, int b, PagedSeq* s) {
  const int q0 = p.q_start[b], q1 = p.q_start[b + 1], kv = p.kv_len[b];
  s->b = b;
  s->q0 = q0;
  s->kv = kv;
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.n || q1 - q0 > p.max_q || kv < 0 ||
                   kv > (long long)p.max_pages << p.page_log2;
  s->ql = bad ? 0 : q1 - q0;
  s->past = bad ? 0 : kv - s->ql;
  s->causal = p.causal_seq ? p.causal_seq[b] != 0 : p.causal != 0;
  return (int)bad | (q1 < q0) << 1;
}

// Keys [lo, hi) that tokens i0 .. i0 + nt - 1 of the sequence see between them, and the tile
// range [t0, t0 + n) that holds them (one tile, seen by nobody, if there are none).
struct PagedKeys {
  int lo, hi, t0, n;
};
__device__ __forceinline__ PagedKeys paged_keys(const PagedAttnParams& p, const PagedSeq& s,
                                                int i0, int nt) {
  PagedKeys k;
  k.hi = s.causal ? min(s.kv, s.past + i0 + nt) : s.kv;
  k.lo = 0;
  if (p.window) {
    const long long lo = (long long)(s.causal ? s.past + i0 + 1 : s.past) - p.window;
    k.lo = lo > 0 ? (int)lo : 0;
  }
  if (k.hi <= k.lo) {
    k.lo = k.hi = k.t0 = 0;
    k.n = 1;
  } else {
    k.t0 = k.lo / PA_KT;
    k.n = (k.hi - 1) / PA_KT + 1 - k.t0;
  }
  return k;
}

// Line length of the sequence of each lane (0 items: 0), and the extremes of its items'
// tiles.  A lane adds up its own items when they are few or alike; longer causal chunks are
// added up by the whole warp, one at a time.
__device__ __forceinline__ int paged_work(const PagedAttnParams& p, const PagedSeq& s, int lane,
                                          int* n_min, int* n_max) {
  const int step = 2 * p.T, items = (s.ql + step - 1) / step;
  int w = 0;
  const bool many = items > 4 && s.causal;
  const int alone = many ? 0 : s.causal ? items : min(items, 1);
#pragma unroll 1
  for (int i = 0; i < alone; ++i) {
    const int n = paged_keys(p, s, i * step, min(step, s.ql - i * step)).n;
    *n_min = min(*n_min, n);
    *n_max = max(*n_max, n);
    w += n + PA_ITEM;
  }
  if (!s.causal) w *= items;  // all its items see the same keys
#pragma unroll 1
  for (unsigned m = __ballot_sync(0xffffffffu, many); m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    PagedSeq x;
    x.ql = __shfl_sync(0xffffffffu, s.ql, src);
    x.past = __shfl_sync(0xffffffffu, s.past, src);
    x.kv = __shfl_sync(0xffffffffu, s.kv, src);
    x.causal = 1;
    const int items_x = (x.ql + step - 1) / step;
    int v = 0;
#pragma unroll 1
    for (int i = lane; i < items_x; i += 32) {
      const int n = paged_keys(p, x, i * step, min(step, x.ql - i * step)).n;
      *n_min = min(*n_min, n);
      *n_max = max(*n_max, n);
      v += n + PA_ITEM;
    }
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == src) w = v;
  }
  return w * p.hkv;
}

// The line's division: `parts` parts in whole multiples of `unit` tiles, the first `rem` of
// them one multiple longer.  (The host refuses calls whose line could reach 2^31, counting
// each row once: chunks that do not overlap.)
struct PagedSplit {
  unsigned q, rem, unit;
  int parts;
  // total 0: no parts.  n_min, n_max: the extremes of the items' tiles.
  __device__ __forceinline__ PagedSplit(unsigned total, int n_min, int n_max) {
    unsigned count = total;
    unit = 1;
    parts = (int)min((unsigned)PA_CTAS, (total + PA_PART - 1) / PA_PART);
    if (n_min == n_max && total > 0) {
      const unsigned len = n_min + PA_ITEM, items = total / len;
      if ((items + PA_CTAS - 1) / PA_CTAS * len <= total / parts + PA_MERGE) {
        unit = len;
        count = items;
        parts = (int)min((unsigned)PA_CTAS, items);
      }
    }
    q = count / max(parts, 1);
    rem = count - q * parts;
  }
  __device__ __forceinline__ int start(unsigned c) const {
    return (int)((c * q + min(c, rem)) * unit);
  }
  __device__ __forceinline__ int owner(unsigned at) const {  // the part that holds it
    at /= unit;
    const unsigned cut = rem * (q + 1);
    return (int)(at < cut ? at / (q + 1) : rem + (at - cut) / q);
  }
};

// Tiles of an item of n that lie before line unit u of it.
__device__ __forceinline__ int paged_cut(int u, int n) {
  const int x = u - PA_ITEM;
  return x >= n ? n : x < PA_CUT ? 0 : x > n - PA_CUT ? n : x;
}

// Walks the pieces of a CTA's part of the line.
struct PagedWalk {
  PagedSeq s;
  PagedKeys k;
  int i0, nt;    // the item's tokens
  int g;         // its key head
  int off;       // line units of it that lie before
  int left;      // line units of the part still to come
  // the current piece: key tiles first .. first + count - 1 of the item
  int first, count;

  __device__ __forceinline__ void item(const PagedAttnParams& p) {
    nt = min(2 * p.T, s.ql - i0);
    k = paged_keys(p, s, i0, nt);
  }
  // `count` units from unit `skip` of sequence `seq` on (a whole warp: 32 items at a time).
  __device__ __forceinline__ void start(const PagedAttnParams& p, const PagedSeq& seq, int skip,
                                        int count_, int lane) {
    left = count_;
    if (left <= 0) return;
    s = seq;
    const int step = 2 * p.T, items = (s.ql + step - 1) / step;
    int at = 0;
#pragma unroll 1
    for (int i = 0; i < items; i += 32) {
      const int mine = i + lane;
      int incl = 0;
      if (mine < items)
        incl = (paged_keys(p, s, mine * step, min(step, s.ql - mine * step)).n + PA_ITEM) * p.hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int n = __popc(__ballot_sync(0xffffffffu, mine < items && incl <= skip));
      at = min(i + n, items - 1);
      if (n > 0) skip -= __shfl_sync(0xffffffffu, incl, n - 1);
      if (n < 32) break;
    }
    i0 = at * step;
    item(p);
    const int len = k.n + PA_ITEM;
    g = min((int)((unsigned)skip / (unsigned)len), p.hkv - 1);
    off = min(skip - g * len, len - 1);
  }
  // Prepares the next piece; false at the end of the part.
  __device__ __forceinline__ bool next(const PagedAttnParams& p) {
#pragma unroll 1
    while (left > 0) {
      if (off == k.n + PA_ITEM) {  // the item is done: next head, tokens, sequence
        off = 0;
        if (++g == p.hkv) {
          g = 0;
          i0 += 2 * p.T;
#pragma unroll 1
          while (i0 >= s.ql) {
            if (s.b + 1 >= p.B) {  // only if the lengths change under the call
              left = 0;
              return false;
            }
            paged_seq(p, s.b + 1, &s);
            i0 = 0;
          }
          item(p);
        }
      }
      const int take = min(k.n + PA_ITEM - off, left);
      first = paged_cut(off, k.n);
      off += take;
      left -= take;
      count = paged_cut(off, k.n) - first;
      if (count > 0) return true;  // else the part has none of the item's tiles
    }
    return false;
  }
  __device__ __forceinline__ bool pair(const PagedAttnParams& p) const { return nt > p.T; }
};

namespace tc {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// mbar_wait that also gives up once another role has (and says so to the others).  A role
// that has given up arrives nowhere any more: arrivals for tiles that were not waited for
// would let the MMA warp run on and release slots whose copies never came, and the wait for
// the copies in flight at the end of the kernel counts on each slot's phases.
__device__ __forceinline__ bool mbar_wait_or(uint64_t* bar, uint32_t parity,
                                             volatile int32_t* gave_up, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*gave_up) return false;
    if (global_ns() - t0 > limit_ns) {
      *gave_up = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Descriptor of an operand whose contiguous axis is not the contraction (V: 64 channels of
// one key per 128-byte row, swizzled): groups of 8 keys are 1024 B apart, chunks of 64
// channels PA_CHUNK.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(PA_CHUNK >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// kind::f16 with both operands of type T (fp32 result); bt: B's contiguous axis is N.
template <class T> __device__ constexpr uint32_t idesc16(int M, int N, bool bt);
template <> __device__ constexpr uint32_t idesc16<bf16>(int M, int N, bool bt) {
  return idesc_bf16(M, N) | (bt ? 1u << 16 : 0u);
}
template <> __device__ constexpr uint32_t idesc16<__half>(int M, int N, bool bt) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24) |
         (bt ? 1u << 16 : 0u);
}

// One thread of a converged warp, the same one every time.  The MMA warp runs its loop
// converged and branches on this for each batch: 64 cycles an MMA here, which is what the
// tensor core takes; with the issue predicated on lane 0 instead it was 73 alone and 85
// beside busy warps.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]: A holds two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#define DG_R32(r)                                                                                \
  "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "   \
  "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
#define DG_OUT32(c, r)                                                                            \
  c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7]), c(r[8]), c(r[9]),      \
      c(r[10]), c(r[11]), c(r[12]), c(r[13]), c(r[14]), c(r[15]), c(r[16]), c(r[17]), c(r[18]),  \
      c(r[19]), c(r[20]), c(r[21]), c(r[22]), c(r[23]), c(r[24]), c(r[25]), c(r[26]), c(r[27]),  \
      c(r[28]), c(r[29]), c(r[30]), c(r[31])

// 32 columns of this warp's lanes; the registers hold them after tmem_wait32.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {" DG_R32() "}, [%32];"
               : DG_OUT32("=f", r)
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DG_OUT32("+f", r)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" DG_R32() "};" ::DG_OUT32("r", r),
               "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
#undef DG_R32
#undef DG_OUT32

}  // namespace tc

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// x << n, 0 for n of 32 or more.
__device__ __forceinline__ unsigned shl(unsigned x, unsigned n) {
  unsigned y;
  asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(n));
  return y;
}

// A row's reference m is set PA_LIFT below its maximum and may lag it by 8 more: the weights
// 2^(s - m) reach 2^8 in bf16, whose exponents have room below 1, and 2^15 in f16, whose
// largest number is 65,504 and whose steps below 2^-14 stay at 2^-24.  Lifted by 2^7, f16
// keeps its 11 bits down to 2^-21 of the largest weight (2^-14 else), and what it rounds off
// of smaller ones is at most 2^-32 of the largest.  l and O carry the factor alike.
template <class T> constexpr float PA_LIFT = 0.f;
template <> constexpr float PA_LIFT<__half> = 7.f;

template <class T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<bf16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct PagedPlan {
  unsigned sums[16];                 // of each warp's sequences
  int mins[16], maxs[16];
  PagedSeq seq;                      // where this CTA's part begins,
  int skip;                          // and the line units of it that lie before
  int32_t gave_up;
  int32_t bad[16];  // a page out of range, of keys and of values, by piece modulo 8
  uint32_t issued[8], issued_q;  // loads so far into each ring slot (place + 1), of rows
};

struct PagedBars {
  uint64_t q_full, q_empty, done;
  uint64_t s_full[2], p_full[4] /* [stream][keys 0-63, 64-127] */, o_full[2], half_done[2];
  uint64_t full[8], empty[8];
};
static_assert(sizeof(PagedPlan) + sizeof(PagedBars) <= 768, "fits the tail of shared memory");

// The line's division, and plan.seq / plan.skip, where the part of CTA c begins (if it has
// one).  Every thread of the CTA calls it; a barrier must follow.  Short on purpose: each CTA
// runs it once, and its instructions arrive as it goes.  Where q_start decreases chunks may
// overlap, their rows would have no one owner and the line could outgrow 32 bits: no parts.
__device__ __forceinline__ PagedSplit paged_plan(const PagedAttnParams& p, PagedPlan* plan,
                                                 int c) {
  constexpr int WARPS = PA_THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (p.B + PA_THREADS - 1) / PA_THREADS;
  PagedSeq s = {};
  int low = 0x7fffffff, high = 0, back = 0;
  unsigned total = 0, start = 0, mine = 0, incl = 0;
  PagedSplit split(0, 0, 0);
  // once to add up, once to find the part: up to a sequence a thread, the first pass's sums
  // serve the second
#pragma unroll 1
  for (int i = 0; i < 2 * chunks; ++i) {
    if (i == chunks) {
      split = PagedSplit(back ? 0 : total, low, high);
      if (c >= split.parts) break;
      start = split.start(c);
      total = 0;
    }
    if (i == 0 || chunks > 1) {
      const int b = (i < chunks ? i : i - chunks) * PA_THREADS + tid;
      s.ql = 0;
      s.causal = 0;
      const int bad = b < p.B ? paged_seq(p, b, &s) : 0;
      if (bad && i < chunks && c == 0 && p.err) atomicOr(p.err, DG_PAGED_BAD_BATCH);
      int n_min = 0x7fffffff, n_max = 0;
      incl = mine = paged_work(p, s, lane, &n_min, &n_max);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      n_min = __reduce_min_sync(0xffffffffu, n_min);
      n_max = __reduce_max_sync(0xffffffffu, n_max);
      if (i > 0) __syncthreads();  // the last chunk's sums have been read
      if (lane == 31) {
        plan->sums[warp] = incl;
        plan->mins[warp] = n_min;
        plan->maxs[warp] = n_max;
      }
      back |= __syncthreads_or(bad & 2);
    }
    const bool in = lane < WARPS;
    unsigned before = in ? plan->sums[lane] : 0;
    low = min(low, __reduce_min_sync(0xffffffffu, in ? plan->mins[lane] : 0x7fffffff));
    high = max(high, __reduce_max_sync(0xffffffffu, in ? plan->maxs[lane] : 0));
    const unsigned all = __reduce_add_sync(0xffffffffu, before);
    before = __reduce_add_sync(0xffffffffu, lane < warp ? before : 0);
    const unsigned at = total + before + incl - mine;
    if (i >= chunks && start >= at && start < at + mine) {
      plan->seq = s;
      plan->skip = (int)(start - at);
    }
    total += all;
  }
  return split;
}

// Ring places, from a piece's first, of step u's keys and values (see the MMA warp): the ring
// holds K0 V0 K1 V1 .. for a pair, whose steps 2 i and 2 i + 1 share tile i, and
// K0 K1 V0 K2 V1 K3 .. else.
__device__ __forceinline__ uint32_t paged_k_at(uint32_t base, bool pair, int u) {
  return base + (pair ? u & ~1 : u < 2 ? u : 2 * u - 1);
}
__device__ __forceinline__ uint32_t paged_v_at(uint32_t base, bool pair, int u, int steps) {
  return base + (pair ? u | 1 : min(steps, 2) + u + min(u, max(steps - 2, 0)));
}

template <int N> __device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

constexpr int PA_REGS_HIGH = 192, PA_REGS_LOW = 120;

// Registers: 12 warps launch with 168 a thread (64,512 in all); the softmax warpgroups take
// 192 and leave the other four warps 120 (256 x 192 + 128 x 120 = 64,512): no spills.
template <class T, int H>
__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const PagedAttnParams p) {
  typedef PagedCfg<H> Cfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sq = smem;                       // 2 row tiles
  uint8_t* ring = sq + 2 * Cfg::TILE;       // SLOTS key or value tiles
  PagedBars* bar = reinterpret_cast<PagedBars*>(ring + Cfg::SLOTS * Cfg::TILE);
  PagedPlan* plan = reinterpret_cast<PagedPlan*>(bar + 1);
  float2* xml = reinterpret_cast<float2*>(ring + Cfg::SLOTS * Cfg::TILE + 768);  // [2][128]
  uint4* stage = reinterpret_cast<uint4*>(xml + 256) + (threadIdx.x >> 5) * 128;  // 2 KB a warp
  __shared__ uint32_t tslot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tc::mbar_init(&bar->q_full, 1);
    tc::mbar_init(&bar->q_empty, 1);
    tc::mbar_init(&bar->done, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar->s_full + i, 1);
      tc::mbar_init(bar->p_full + 2 * i, 5);  // 4 softmax warps, and the tiles are there
      tc::mbar_init(bar->p_full + 2 * i + 1, 4);
      tc::mbar_init(bar->o_full + i, 1);
      tc::mbar_init(bar->half_done + i, 1);
    }
    for (int i = 0; i < Cfg::SLOTS; ++i) {
      tc::mbar_init(bar->full + i, 1);
      tc::mbar_init(bar->empty + i, 1);
    }
    tc::fence_mbar_init();
    plan->seq = {p.B, 0, 0, 0, 0, 0};  // no sequence, should lengths that change hide the part's
    plan->skip = 0;
    plan->gave_up = 0;
    for (int i = 0; i < 16; ++i) plan->bad[i] = 0;
    for (int i = 0; i < 8; ++i) plan->issued[i] = 0;
    plan->issued_q = 0;
  }
  if (warp == 8) tc::tmem_alloc(&tslot, 512);
  if (tid == PA_THREADS - 32) {
    tc::prefetch_tmap(&mq);
    tc::prefetch_tmap(&mk);
    tc::prefetch_tmap(&mv);
  }
  pdl_enter();
  const int c = blockIdx.x;
  const PagedSplit split = paged_plan(p, plan, c);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tslot;
  volatile int32_t* gave_up = &plan->gave_up;

  if (tid == 0) p.rec[c].valid = 0;
  const bool idle = c >= split.parts;
  PagedWalk w;
  w.start(p, plan->seq, plan->skip, idle ? 0 : split.start(c + 1) - split.start(c), lane);
  bool ok = true;

  if (warp >= 8) {
  reg_dec<PA_REGS_LOW>();
  if (warp == 9 || warp == 11) {
    // ------------------------------------------------------------------ TMA, keys and values
    // A warp each: with pages of 16 tokens a tile is 16 boxes, and one warp's bookkeeping and
    // issue took as long as the copies (64 caches of up to 16,384 keys: 251 us, 204 with a warp
    // for each).
    const bool values = warp == 11;
    ok = !values || !p.stall;
    const CUtensorMap* map = values ? &mv : &mk;
    int32_t* bad_page = plan->bad + (values ? 8 : 0);
    uint32_t base = 0, piece = 0;  // ring tiles of earlier pieces, pieces
    const int rows = min(1 << p.page_log2, PA_KT), npg = PA_KT / rows;
    const int pg = lane & (npg - 1), ch = lane / npg;  // this lane's page of a tile, and chunk
    // Page numbers: a lane holds one of 32 consecutive ones, of two such blocks, so the table
    // is read a block ahead of its use.
    int e0 = -1, e1 = -1, blk = 0;
    auto entries = [&](int k) {
      const long long key = ((long long)k * 32 + lane) << p.page_log2;
      return key < w.k.hi && key + (1LL << p.page_log2) > w.k.lo
                 ? p.table[(long long)w.s.b * p.max_pages + k * 32 + lane]
                 : -1;
    };
    auto load = [&](int tile, uint32_t n) {  // into ring place n
      const int key = tile * PA_KT + pg * rows, page = key >> p.page_log2;
      const int first = (tile * PA_KT) >> (p.page_log2 + 5);  // a tile's pages share a block
      if (first > blk) {
        e0 = e1;
        e1 = entries(++blk + 1);
      }
      const int id = __shfl_sync(0xffffffffu, e0, page & 31);
      const bool need = ch < Cfg::CH && key < w.k.hi && key + rows > w.k.lo;
      const bool good = need && id >= 0 && id < p.n_pages;
      const unsigned mask = __ballot_sync(0xffffffffu, good);
      const bool bad = __any_sync(0xffffffffu, need && !good);
      const int s = n % Cfg::SLOTS;
      ok = ok && tc::mbar_wait_or(bar->empty + s, ((n / Cfg::SLOTS) & 1) ^ 1, gave_up, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        if (bad) {
          bad_page[piece & 7] = 1;
          if (p.err) atomicOr(p.err, DG_PAGED_BAD_PAGE);
        }
        plan->issued[s] = n + 1;
        tc::mbar_expect_tx(bar->full + s, __popc(mask) * rows * 128);
      }
      __syncwarp();
      if (good)
        tc::tma_load_4d(ring + s * Cfg::TILE + ch * PA_CHUNK + pg * rows * 128, map, bar->full + s,
                        ch * 64, key & ((1 << p.page_log2) - 1), w.g, id);
    };
    for (; w.next(p); ++piece) {
      const bool pair = w.pair(p);
      const int t0 = w.k.t0 + w.first, steps = pair ? 2 * w.count : w.count;
      blk = (t0 * PA_KT) >> (p.page_log2 + 5);
      e0 = entries(blk);
      e1 = entries(blk + 1);
      if (lane == 0) bad_page[piece & 7] = 0;
#pragma unroll 1
      for (int i = 0; i < w.count; ++i) {
        // the rows: at once in the first piece, later after the piece's first two key tiles,
        // since the last piece may still hold their buffer
        if (!values && i == (piece == 0 ? 0 : min(w.count - 1, 2))) {
          if (piece > 0 && w.count <= 2) load(t0 + i, paged_k_at(base, pair, pair ? 2 * i : i));
          ok = ok && tc::mbar_wait_or(&bar->q_empty, (piece & 1) ^ 1, gave_up, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            const int tiles = pair ? 2 : 1;
            if (lane == 0) {
              plan->issued_q = piece + 1;
              tc::mbar_expect_tx(&bar->q_full, tiles * Cfg::CH * p.G * p.T * 128);
            }
            __syncwarp();
            if (lane < tiles * Cfg::CH) {
              const int t = lane / Cfg::CH, qc = lane % Cfg::CH;
              tc::tma_load_3d(sq + t * Cfg::TILE + qc * PA_CHUNK, &mq, &bar->q_full, qc * 64,
                              w.g * p.G, w.s.q0 + w.i0 + t * p.T);
            }
          }
          if (piece > 0 && w.count <= 2) continue;
        }
        const int u = pair ? 2 * i : i;
        load(t0 + i, values ? paged_v_at(base, pair, u, steps) : paged_k_at(base, pair, u));
      }
      base += 2 * w.count;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    uint32_t base = 0, piece = 0;  // ring tiles of earlier pieces, pieces
    uint32_t pc = 0;               // parity of each stream's P tiles
    constexpr uint32_t idS = tc::idesc16<T>(128, 128, false);
    constexpr uint32_t idO = tc::idesc16<T>(128, H, true);
    const uint64_t q_desc = tc::sdesc_k128(tc::smem_addr(sq));
    const uint64_t k_desc = tc::sdesc_k128(tc::smem_addr(ring));
    const uint64_t v_desc = tc::sdesc_mn128(tc::smem_addr(ring));
    // Only the elected thread's `ok` counts, so the lanes need no vote.
    auto wait = [&](uint64_t* b, uint32_t parity) {
      ok = ok && tc::mbar_wait_or(b, parity, gave_up, p.wait_ns);
    };
    for (; w.next(p); ++piece) {
      // through a reduction, whose result the compiler knows to be the same in every lane
      const bool pair = __reduce_max_sync(0xffffffffu, (unsigned)w.pair(p)) != 0;
      const int count = __reduce_max_sync(0xffffffffu, w.count);
      const int steps = pair ? 2 * count : count;
      wait(&bar->q_full, piece & 1);
      // Step u adds P V of stream u & 1 and issues the same stream's next scores, two steps
      // ahead.  Solo: step u is key tile u.  Pair: steps 2 i and 2 i + 1 are key tile i.
      // The first half of P comes with the step's tiles (the next warp's doing).
#pragma unroll 1
      for (int u = -2; u < steps; ++u) {
        const int t = u & 1;
        const bool more = u + 2 < steps;
        const uint32_t vs = paged_v_at(base, pair, u, steps), ks = paged_k_at(base, pair, u + 2);
        const uint64_t vd = v_desc + (uint64_t)((vs % Cfg::SLOTS) * (Cfg::TILE >> 4));
        const uint64_t kd = k_desc + (uint64_t)((ks % Cfg::SLOTS) * (Cfg::TILE >> 4));
        if (u < 0 && more) wait(bar->full + ks % Cfg::SLOTS, (ks / Cfg::SLOTS) & 1);
        if (u >= 0) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // O_t += P_t V, 64 keys at a time
            wait(bar->p_full + 2 * t + hf, (pc >> t) & 1);
            tc::fence_after_sync();
            if (tc::elect() && ok) {
#pragma unroll
              for (int k = 4 * hf; k < 4 * hf + 4; ++k)
                tc::mma_ts(tmem + 256 + t * H, tmem + t * 128 + k * 8, vd + k * (2048 >> 4), idO,
                           u >= 2 || k != 0);
              if (hf == 0) tc::mma_commit(bar->half_done + t);
            }
            __syncwarp();
          }
          pc ^= 1u << t;
        }
        if (tc::elect() && ok) {
          if (more) {
            tc::fence_after_sync();
            const uint64_t qd = q_desc + (uint64_t)(pair && t ? Cfg::TILE >> 4 : 0);
#pragma unroll
            for (int k = 0; k < 4 * Cfg::CH; ++k) {  // S_t = Q K^T
              const uint32_t o = ((k >> 2) * PA_CHUNK + (k & 3) * 32) >> 4;
              tc::mma_bf16(tmem + t * 128, qd + o, kd + o, idS, k != 0);
            }
            tc::mma_commit(bar->s_full + t);
          }
          // The ring's places are released in their order, values (place vs) before keys (a
          // later one).  Consecutive places of one loader lie at most 3 apart (at a piece's
          // end), so the release that let it load place n - 3 is that of n - 7, and n - 8 is
          // free as well: its wait for place n - 4 (4 slots) never meets the parity of n - 8.
          if (u >= 0) {
            if (!more) tc::mma_commit(bar->o_full + t);
            if (!pair || t == 1) tc::mma_commit(bar->empty + vs % Cfg::SLOTS);
          }
          if (more) {
            if (!pair || t == 1) tc::mma_commit(bar->empty + ks % Cfg::SLOTS);
            if (u + 3 == steps) tc::mma_commit(&bar->q_empty);
          }
        }
        __syncwarp();
      }
      base += 2 * count;
    }
    // nothing of the tensor cores' may be in flight when TMEM is freed
    if (tc::elect()) {
      tc::mma_commit(&bar->done);
      if (!tc::mbar_wait(&bar->done, 0)) *gave_up = 1;
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------------ tiles for the MMA
    // Waits for the tiles of each step on the MMA warp's behalf, whose own waits would keep
    // the tensor cores idle (650 of 3,600 cycles a pair of tiles), and clears what no row
    // sees in them.  A slot's two latest tiles differ in parity, so a wait for a tile is sound
    // only once the slot's previous tile has landed, and copies land in any order.  It waits
    // for all tiles itself but a piece's first keys, which the MMA warp waits for; that those
    // have landed it learns from the scores made of them, before any wait for the tiles that
    // follow them in their slots.
    uint32_t base = 0, said = 0;  // ring tiles of earlier pieces, parity of each stream's steps
    auto wait = [&](uint64_t* b, uint32_t parity) {
      ok = ok && tc::mbar_wait_or(b, parity, gave_up, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
    };
    // values nobody sees become 0, so that 0 * value is 0 whatever the slot held
    auto clear_v = [&](uint32_t i, int lo, int hi) {
      uint8_t* v = ring + (i % Cfg::SLOTS) * Cfg::TILE;
#pragma unroll 1
      for (int ch = 0; ch < Cfg::CH; ++ch) {
        uint8_t* vc = v + ch * PA_CHUNK;
#pragma unroll 1
        for (int x = lane; x < lo * 8; x += 32)
          *reinterpret_cast<uint4*>(vc + x * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int x = hi * 8 + lane; x < PA_KT * 8; x += 32)
          *reinterpret_cast<uint4*>(vc + x * 16) = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    while (w.next(p)) {
      const bool pair = w.pair(p);
      const int count = w.count, steps = pair ? 2 * count : count;
      const int key0 = (w.k.t0 + w.first) * PA_KT;
      // keys nobody sees are in the piece's first tile, its last or none
      const int cut_lo = w.k.lo > key0 ? 0 : -1;
      const int cut_hi = w.k.hi < key0 + count * PA_KT ? count - 1 : -1;
#pragma unroll 1
      for (int u = 0; u < steps; ++u) {
        const int t = u & 1;
        const bool tiles = !pair || t == 0;
        if (tiles) {
          const uint32_t vs = paged_v_at(base, pair, u, steps);
          const int tile = pair ? u >> 1 : u;
          wait(bar->full + vs % Cfg::SLOTS, (vs / Cfg::SLOTS) & 1);
          if (ok && (tile == cut_lo || tile == cut_hi)) {
            const int lo = min(max(w.k.lo - key0 - tile * PA_KT, 0), PA_KT);
            clear_v(vs, lo, min(max(w.k.hi - key0 - tile * PA_KT, lo), PA_KT));
          }
        }
        // (this also keeps the arrival below out of the stream's last phase, which is over)
        wait(bar->s_full + t, said >> t & 1);
        if (tiles && u + 2 < steps) {
          const uint32_t ks = paged_k_at(base, pair, u + 2);
          wait(bar->full + ks % Cfg::SLOTS, (ks / Cfg::SLOTS) & 1);
        }
        said ^= 1u << t;
        if (ok && lane == 0) tc::mbar_arrive(bar->p_full + 2 * t);
      }
      base += 2 * count;
    }
  }
  } else {
    // ------------------------------------------------------------------ softmax
    reg_inc<PA_REGS_HIGH>();
    const int t = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane;
    const int tok = r / p.G, head = r - tok * p.G;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * H + lanes;
    const float sl = p.scale_log2;
    uint32_t sc = 0, oc = 0, piece = 0;
    for (; w.next(p); ++piece) {
      const bool pair = w.pair(p);
      const int i0 = pair ? t * p.T : 0;  // first token of this row tile within the item
      const int cnt = pair ? w.count : (w.count + 1 - t) >> 1;
      const bool live = tok < p.T && i0 + tok < w.nt;
      // keys this row sees; a row of no token takes any
      int lo = 0, hi = 0x7fffffff;
      if (live) {
        const PagedKeys k1 = paged_keys(p, w.s, w.i0 + i0 + tok, 1);
        lo = k1.lo;
        hi = k1.hi;
      }
      const int lo_max = __reduce_max_sync(0xffffffffu, lo);
      const int hi_min = __reduce_min_sync(0xffffffffu, hi);
      const bool work = __any_sync(0xffffffffu, live);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < cnt; ++i) {
        const int key0 = (w.k.t0 + w.first + (pair ? i : 2 * i + t)) * PA_KT;
        ok = ok && tc::mbar_wait_or(bar->s_full + t, sc & 1, gave_up, p.wait_ns);
        ++sc;
        ok = __all_sync(0xffffffffu, ok);
        if (work && ok) {
          tc::fence_after_sync();
          // A tile with keys that not every row sees is first rewritten with -inf there, by
          // its own loop: in the loops below the selections would cost every tile their room
          // in the instruction cache.
          if (key0 < lo_max || key0 + PA_KT > hi_min) {
#pragma unroll 1
            for (int q = 0; q < PA_KT; q += 32) {
              float x[32];
              uint32_t y[32];
              tc::tmem_ld32_async(ts + q, x);
              // bits lo .. hi - 1 of this chunk (a shift by 32 or more gives 0)
              const unsigned seen = shl(0xffffffffu, max(lo - key0 - q, 0)) &
                                    ~shl(0xffffffffu, max(hi - key0 - q, 0));
              tc::tmem_wait32(x);
#pragma unroll
              for (int i2 = 0; i2 < 32; ++i2)
                y[i2] = seen >> i2 & 1 ? __float_as_uint(x[i2]) : 0xff800000u;
              tc::tmem_st32(ts + q, y);
            }
            tc::tmem_wait_st();
          }
          // 64 keys at a time, P V of the first half under the softmax of the second.  The
          // weights are taken against the row's old reference m at once, while the half's
          // maximum comes out of the same pass; only where it exceeds m by far (the first tile,
          // seldom later) does the reference move, O and l follow, and the half is done
          // again.  A pass for the maximum first would lie on the way from the scores to the
          // products (450 of 3,450 cycles a pair of tiles).
          const uint64_t sl2 = f2(sl, sl);
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t pk[32];
            float sum;
#pragma unroll 1
            while (true) {
              const float neg = m == -INFINITY ? 0.f : -m;
              const uint64_t neg2 = f2(neg, neg);
              uint64_t sum2[2] = {0, 0};
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              auto weights = [&](const float* x, uint32_t* w16) {
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  float e0, e1;
                  mx[y & 3] = max3(mx[y & 3], x[2 * y], x[2 * y + 1]);
                  unf2(fma2(f2(x[2 * y], x[2 * y + 1]), sl2, neg2), &e0, &e1);
                  e0 = ex2(e0);
                  e1 = ex2(e1);
                  sum2[y & 1] = add2(sum2[y & 1], f2(e0, e1));
                  w16[y] = pack2<T>(e0, e1);
                }
              };
              float sa[32], sb[32];
              tc::tmem_ld32_async(ts + 64 * hf, sa);
              tc::tmem_wait32(sa);
              tc::tmem_ld32_async(ts + 64 * hf + 32, sb);
              weights(sa, pk);
              tc::tmem_wait32(sb);
              weights(sb, pk + 16);
              float x, y;
              unf2(add2(sum2[0], sum2[1]), &x, &y);
              sum = x + y;
              const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sl;
              const bool grow = mt - m > 8.f + PA_LIFT<T>;  // (a difference: exact where it counts)
              if (!__any_sync(0xffffffffu, grow)) break;
              const float a = grow ? ex2(m - (mt - PA_LIFT<T>)) : 1.f;
              // rows that have seen nothing yet have nothing to scale
              const bool scale = __any_sync(0xffffffffu, grow && m != -INFINITY);
              l *= a;
              m = grow ? mt - PA_LIFT<T> : m;
              if (scale) {
                if (hf == 1) {  // O must have the first half's products before it is scaled
                  ok = ok && tc::mbar_wait_or(bar->half_done + t, (sc & 1) ^ 1, gave_up, p.wait_ns);
                  ok = __all_sync(0xffffffffu, ok);
                  tc::fence_after_sync();
                }
#pragma unroll 1
                for (int q = 0; q < H; q += 32) {
                  float o[32];
                  tc::tmem_ld32_async(to + q, o);
                  tc::tmem_wait32(o);
                  uint32_t ou[32];
#pragma unroll
                  for (int z = 0; z < 32; ++z) ou[z] = __float_as_uint(o[z] * a);
                  tc::tmem_st32(to + q, ou);
                }
              }
            }
            l += sum;
            // P over scores that have been read: columns 0-31, then 32-63
            tc::tmem_st32(ts + 32 * hf, pk);
            tc::tmem_wait_st();
            if (hf == 0) {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(bar->p_full + 2 * t);
            }
          }
        } else {
          tc::fence_before_sync();
          if (ok && lane == 0) tc::mbar_arrive(bar->p_full + 2 * t);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (ok && lane == 0) tc::mbar_arrive(bar->p_full + 2 * t + 1);
      }
      if (cnt > 0) {
        ok = ok && tc::mbar_wait_or(bar->o_full + t, oc & 1, gave_up, p.wait_ns);
        ++oc;
        ok = __all_sync(0xffffffffu, ok);
      }
      // ---- the piece's rows: whole items to out, cut ones to the workspace
      const bool begins = w.first == 0, ends = w.first + w.count == w.k.n;
      // this row within the item's rows of out (-1: none), and in the workspace
      const int row_at = live ? (i0 + tok) * p.hq + w.g * p.G + head : -1;
      const long long piece_at = (long long)c * 2 + (begins ? 1 : 0);
      const int piece_row = (pair ? t * 128 : 0) + r;
      float w0 = 1.f, w1 = 0.f;  // weights of this stream's and the other's O
      float M = m, L = l;
      if (!pair) {
        xml[t * 128 + r] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 a = xml[r], b = xml[128 + r];
        M = fmaxf(a.x, b.x);
        w0 = a.x == -INFINITY ? 0.f : ex2(a.x - M);
        w1 = b.x == -INFINITY ? 0.f : ex2(b.x - M);
        L = w0 * a.y + w1 * b.y;
      }
      // Read only here: the loaders have looked at all of the piece's pages once each stream's
      // products are done, and a stream without a tile of its own has waited for none but at
      // the barrier above.
      const bool bad = (plan->bad[piece & 7] | plan->bad[8 + (piece & 7)]) != 0;
      if (bad) L = __int_as_float(0x7fc00000);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const bool whole = begins && ends;
      if (work && ok) {
        tc::fence_after_sync();
        const bool two = !pair && w.count > 1;
        const uint32_t o_a = pair ? to : tmem + 256 + lanes, o_b = tmem + 256 + H + lanes;
        const float f0 = whole ? w0 * inv : w0, f1 = whole ? w1 * inv : w1;
        T* out = static_cast<T*>(p.out) + ((long long)w.s.q0 + w.i0) * p.hq * H;
        // one short loop: the code of a piece's end runs once a piece, and what of it the
        // instruction cache has lost costs more than its latencies
        const int q_end = pair ? H : (t + 1) * (H / 2);
#pragma unroll 1
        for (int q = pair ? 0 : t * (H / 2); q < q_end; q += 32) {
          float o[32];
          tc::tmem_ld32_async(o_a + q, o);
          tc::tmem_wait32(o);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] *= f0;
          if (two) {
            float o2[32];
            tc::tmem_ld32_async(o_b + q, o2);
            tc::tmem_wait32(o2);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = fmaf(o2[x], f1, o[x]);
          }
          if (whole) {
            // through this warp's 2 KB of shared memory, so that a store instruction
            // writes 64 contiguous bytes of 8 rows (chunks of 16 bytes, swizzled by row)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              stage[lane * 4 + (x ^ ((lane >> 1) & 3))] =
                  make_uint4(pack2<T>(o[8 * x], o[8 * x + 1]), pack2<T>(o[8 * x + 2], o[8 * x + 3]),
                             pack2<T>(o[8 * x + 4], o[8 * x + 5]),
                             pack2<T>(o[8 * x + 6], o[8 * x + 7]));
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int rr = 8 * x + (lane >> 2);
              const uint4 y = stage[rr * 4 + ((lane & 3) ^ ((rr >> 1) & 3))];
              const int at = __shfl_sync(0xffffffffu, row_at, rr);
              if (at >= 0) reinterpret_cast<uint4*>(out + (long long)at * H + q)[lane & 3] = y;
            }
            __syncwarp();
          } else if (live) {
            float4* dst = p.part_o + (piece_at * (H / 4) + q / 4) * p.part_rows + piece_row;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              dst[x * (long long)p.part_rows] =
                  make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
      }
      if (live && (pair || t == 0)) {
        if (!whole)
          p.part_ml[piece_at * p.part_rows + piece_row] = make_float2(M, L);
        else if (p.lse)
          p.lse[((long long)w.s.q0 + w.i0) * p.hq + row_at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
      if (!pair) {
        // both warpgroups have read both accumulators and xml
        tc::fence_before_sync();
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      if (tid == 0 && begins && !ends) {
        // the line's position of the item's end gives the last CTA that holds a piece
        const int begin = split.start(c + 1) - w.left - w.off;
        const int len = w.k.n + PA_ITEM;
        int last = split.owner(begin + len - 1);
        while (last > c && paged_cut(split.start(last) - begin, w.k.n) == w.k.n) --last;
        PagedRec rec;
        rec.valid = 1;
        rec.last = last;
        rec.row0 = w.s.q0 + w.i0;
        rec.ntok = w.nt;
        rec.g = w.g;
        p.rec[c] = rec;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0) {
    // no copy may land after the CTA has gone: normally all have been waited for already
    bool landed = true;
    for (int i = 0; i < Cfg::SLOTS; ++i)
      if (plan->issued[i])
        landed = tc::mbar_wait(bar->full + i, ((plan->issued[i] - 1) / Cfg::SLOTS) & 1) && landed;
    if (plan->issued_q) landed = tc::mbar_wait(&bar->q_full, (plan->issued_q - 1) & 1) && landed;
    if ((plan->gave_up || !landed) && p.err) atomicOr(p.err, DG_PAGED_TIMEOUT);
  }
  if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// Adds the pieces of cut items: block (c, y) takes rows 8 R y .. of the item that starts and
// does not end in CTA c.  Thread (row, 4 channels) with 8 rows fastest, so that a piece's
// channels of 8 rows are one 128-byte line, and R such rows a thread.  Every thread keeps its
// rows' running maximum and sum itself: (m, l) and O of several pieces are on their way
// together and nothing waits for another thread (weights by a first pass through shared memory
// took 10.0 us for drafted tokens, this takes 7.2).  R = 3 for items of two row tiles, mostly
// two pieces each (8,192-token prompt, 38 MB of pieces: 11.7 us; 13.6 with R = 4); R = 1 for
// one, many pieces and few blocks.
template <class T, int H, int R>
__global__ void __launch_bounds__(2 * H) paged_merge_kernel(const PagedAttnParams p) {
  pdl_enter();
  const int c = blockIdx.x, i = threadIdx.x & 7, q = threadIdx.x >> 3;
  const PagedRec rec = p.rec[c];
  if (!rec.valid) return;
  const int n = min(rec.last, PA_CTAS - 1) - c + 1;
  const int row0 = blockIdx.y * 8 * R + i;
  constexpr int AHEAD = R > 1 ? 2 : 8;  // pieces on their way together
  float M[R], L[R];
  float4 o[R];
#pragma unroll
  for (int x = 0; x < R; ++x) {
    M[x] = -INFINITY;
    L[x] = 0.f;
    o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += AHEAD) {
    float2 ml[AHEAD][R];
    float4 v[AHEAD][R];
#pragma unroll
    for (int y = 0; y < AHEAD; ++y) {
      // k-th piece: slot 1 of CTA c, then slot 0 of c + k.  Past the last piece or row the
      // last again, unused: loads without branches go out together.
      const int k = min(k0 + y, n - 1);
      const long long at = ((long long)(c + k) * 2 + (k == 0)) * p.part_rows;
#pragma unroll
      for (int x = 0; x < R; ++x) {
        const int row = min(row0 + 8 * x, p.part_rows - 1);
        ml[y][x] = p.part_ml[at + row];
        v[y][x] = p.part_o[at * (H / 4) + (long long)q * p.part_rows + row];
      }
    }
#pragma unroll
    for (int y = 0; y < AHEAD; ++y)
#pragma unroll
      for (int x = 0; x < R; ++x) {
        if (k0 + y >= n) break;
        const float m = ml[y][x].x, Mn = fmaxf(M[x], m);
        const float a = M[x] == -INFINITY ? 0.f : ex2(M[x] - Mn);
        const float b = m == -INFINITY ? 0.f : ex2(m - Mn);
        M[x] = Mn;
        L[x] = L[x] * a + ml[y][x].y * b;  // NaN stays NaN: a page out of range
        o[x].x = o[x].x * a + v[y][x].x * b;
        o[x].y = o[x].y * a + v[y][x].y * b;
        o[x].z = o[x].z * a + v[y][x].z * b;
        o[x].w = o[x].w * a + v[y][x].w * b;
      }
  }
#pragma unroll
  for (int x = 0; x < R; ++x) {
    const int row = row0 + 8 * x, r = row & 127, tk = r / p.G, tok = (row >> 7) * p.T + tk;
    if (row >= p.part_rows || tk >= p.T || tok >= rec.ntok) continue;
    const long long at = (long long)(rec.row0 + tok) * p.hq + rec.g * p.G + (r - tk * p.G);
    const float inv = L[x] == 0.f ? 0.f : 1.f / L[x];
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at * H + 4 * q) =
        make_uint2(pack2<T>(o[x].x * inv, o[x].y * inv), pack2<T>(o[x].z * inv, o[x].w * inv));
    if (p.lse && q == 0)
      p.lse[at] = L[x] == 0.f ? -INFINITY : (M[x] + log2f(L[x])) * 0.6931471805599453f;
  }
}

}  // namespace dg
