// distill.cu -- distillation from a teacher's top logits.
//
// A row holds the student's V logits x and K teacher logits t at the
// vocabulary entries idx.  With temperature T,
//   p      = softmax(t / T) over the row's valid entries,
//   log q  = x / T - log sum_j exp(x_j / T),
//   loss   = sum_k p_k (log p_k - log q[idx_k]),
//   dx_j   = g / T * (q_j - sum over {k : idx_k = j} of p_k).
// An entry with t = -inf or idx outside [0, V) is not valid; a row without
// valid entries has loss 0 and gradient 0.
//
// The row's online pair is (m, s): m = max x, s = sum 2^((x - m) c) with
// c = log2(e) / T.  The difference is taken before the product, so a row
// filled with the type's lowest value is a uniform row and not an overflow.
#include <climits>
#include <cstdio>

#include "rr.h"
#include "rr_internal.h"
#include "rowwise.cuh"
#include "token.cuh"

namespace rr {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct MaxPlain {
  using T = float;
  static __device__ __forceinline__ T f(T a, T b) { return fmaxf(a, b); }
};

// The (m, s) monoid.  A side whose maximum is -inf has s = 0, or NaN when it
// holds a NaN.
// Over a warp: the maximum, then the sums brought to it.
__device__ __forceinline__ void ms2_warp(float &m, float &s, float c) {
  const float M = warp_allreduce<MaxPlain, 32>(m);
  if (m != -INFINITY) s *= ex2_approx((m - M) * c);
  s = warp_allreduce<SumF32, 32>(s);
  m = M;
}

// A run of N elements folded into the thread's pair.
template <int N>
__device__ __forceinline__ void ms2_fold(float &m, float &s, const float (&e)[N], float c) {
  float v = e[0];
#pragma unroll
  for (int j = 1; j < N; ++j) v = fmaxf(v, e[j]);
  if (v > m) {
    s = (m == -INFINITY) ? s : s * ex2_approx((m - v) * c);
    m = v;
  }
  // before the first finite element the reference is 0: -inf terms add 0,
  // NaN stays
  const float ref = (m == -INFINITY) ? 0.0f : m;
#pragma unroll
  for (int j = 0; j < N; ++j) s += ex2_approx((e[j] - ref) * c);
}

template <class E> __device__ __forceinline__ float value(const E *p) {
  if constexpr (sizeof(E) == 2) return bf16_f(*p);
  else return *p;
}
template <class E> __device__ __forceinline__ void put(E *p, float v) {
  if constexpr (sizeof(E) == 2) *p = f_bf16(v);
  else *p = v;
}

// ---- the kernel ----------------------------------------------------------------
// A persistent CTA takes a row at a time (a cluster of C CTAs, each a slice of
// it, where there are fewer rows than SMs or rows so long that those in
// flight would not fit the L2).  The slice passes through a ring of pieces in
// shared memory, filled by bulk copies:
//
//   the producer warp   waits for a free piece and starts its copy, as far
//                       ahead as the ring allows; a slice twice for its two
//                       passes, the second time out of the L2 (the rows in
//                       flight are held to 75 MiB of it), so DRAM is read
//                       once;
//   T consumer threads  pass 1 folds the pieces as they land into (M, s);
//                       pass 2 writes dx;
//   the exchange warp   joins the warps' pairs, sends the CTA's to its peers
//                       and joins theirs; writes the loss;
//   the teacher warp    turns the next row's teacher logits into
//                       probabilities and gathers the student's logits at
//                       their entries;
//   the finisher warp   rewrites dx at the entries, behind pass 2.
//
// (kLoss: pass 1 alone; kGrad: pass 2 alone, with a given lse; a CTA then
// takes one slice of a row at a time.)  The row is seen in 16-byte units:
// unit u holds elements u N - off + j; the partial units at a row's ends are
// loaded by element and filled up with -inf, which adds nothing.
//
// DRAM bounds it.  Measured, 8192 x 131072 bf16 with K = 64, loss and gradient:
// 654 us, 0.97 of the copy bandwidth.  Slices kept in shared memory between
// the passes (clusters of 2, 4 and 8 CTAs, the pairs' exchange before or
// behind the next row's pass 1) took 735, 831 and 872 us: CTAs of a cluster
// wait for one another twice a row, which costs more than the L2's second
// read.  One warp in place of teacher and finisher took 10 % longer on rows
// of 64 KiB, whose lists are then the longest chain.
//
// Arithmetic.  Pass 1 takes y = x c as fma(x, c, -M), M the rounded product of
// the thread's largest x and c, so its rounding drops out of s and of every
// term; one packed instruction a pair.  The rounding is at most 64 octaves
// while |M| < 2^31, which a sum of 2^31 terms has room for.  M starts at -2^31,
// so what lies below (masks) adds 0.  Where the row's M is not between
// those (a row of nothing but mask, +inf) the row is folded again, differences
// first, and pass 2 does the same.
// kGrad's q = exp(x / T - lse) is off by the roundings of numbers of the lse's
// size, up to six of them: 2^-13 of q at |lse| = 256, all of it at 10^7 (a row of
// nothing but mask).  Past 256 the pair is taken from the row, by the consumers
// of the CTA that has its first slice; it then writes the whole row and the
// others nothing of it, since dx may be x.
//
// Every wait is bounded.  The pairs go to two places in turn: a CTA writes
// place A again only after every peer's next pair has reached it in place B,
// which each sent after its reads of A.  Lists, statistics and warps' pairs
// have two places in the same way, an item's freed by the item after next.
enum { kLoss = 0, kBoth = 1, kGrad = 2 };

constexpr int kRingMaxPieces = 16;
constexpr size_t kRingSmem = 224 * 1024;       // a CTA's most; two of 112 KiB fit, and so on
constexpr int kRingUnits = 4;                  // units of a piece a thread has in hand

struct RingShape {
  int64_t items;     // rows, or (kGrad) slices of rows
  int slices;        // kGrad: slices a row
  int slice_units;   // units of a CTA's slice
  int np;            // pieces of a slice
  int P;             // pieces of the ring
  int lg_tab;        // log2 of the places of the finisher warp's table
};

// A row by n threads, this one t: f(element, value) for the elements outside
// its whole 16-byte units, g(first element, unit) for those, four at a time.
template <class E, class F, class G>
__device__ __forceinline__ void each_of_row(const E *x, int64_t V, int t, int n, F f, G g) {
  constexpr int N = 16 / (int)sizeof(E);
  const int64_t head = min(V, (int64_t)((-(uintptr_t)x & 15) / sizeof(E)));
  const int64_t units = (V - head) / N, rest = V - head - units * N;
  const uint4 *u = reinterpret_cast<const uint4 *>(x + head);
  for (int64_t b = t; b < units; b += 4 * n) {
    uint4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (b + k * n < units) w[k] = u[b + k * n];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (b + k * n < units) g(head + (b + k * n) * N, w[k]);
  }
  if (t < head + rest) {   // at most 2 N - 2 of them
    const int64_t j = t < head ? t : units * N + t;
    f(j, value(x + j));
  }
}

// A CTA's part of an item.
template <class E>
struct Part {
  static constexpr int N = 16 / (int)sizeof(E);
  int64_t row, first;   // row; element at the part's first place
  int nu;               // units
  int ub, ue;           // whole units among them: [ub, ue)
  __device__ __forceinline__ Part(const DistillArgs &a, const RingShape &g, int64_t item, int slice,
                                  bool sliced) {
    row = sliced ? item / g.slices : item;
    if (sliced) slice = (int)(item - row * g.slices);
    const E *x = reinterpret_cast<const E *>(a.x) + row * a.ldx;
    const int off = (int)(((uintptr_t)x & 15) / sizeof(E));
    const int64_t units = (a.V + off + N - 1) / N;
    const int64_t u0 = min((int64_t)slice * g.slice_units, units);
    nu = (int)min((int64_t)g.slice_units, units - u0);
    first = u0 * N - off;
    ub = nu > 0 && first < 0 ? 1 : 0;
    ue = nu > 0 && first + (int64_t)nu * N > a.V ? max(ub, nu - 1) : nu;
  }
};

// Which piece comes next, and the parity of its barriers.
struct Cursor {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int P) {
    if (++slot == P) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void st_dsmem_f2(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
// bulk_g2s with an L2 eviction policy.
__device__ __forceinline__ void bulk_g2s_hint(void *dst, const void *src, uint32_t bytes,
                                              uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest of a unit's elements (NaN ones passed over) and its pairs.
template <class E>
__device__ __forceinline__ float unit_max(const uint4 &w) {
  if constexpr (sizeof(E) == 2) {
    const uint32_t h = max_bf16x2(max_bf16x2(w.x, w.y), max_bf16x2(w.z, w.w));
    return fmaxf(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
  } else {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                 fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
}
template <class E>
__device__ __forceinline__ void unit_pairs(const uint4 &w, uint64_t (&p)[8 / sizeof(E)]) {
  if constexpr (sizeof(E) == 2) {
    p[0] = bf16x2_to_f2(w.x);
    p[1] = bf16x2_to_f2(w.y);
    p[2] = bf16x2_to_f2(w.z);
    p[3] = bf16x2_to_f2(w.w);
  } else {
    p[0] = f2_pack(__uint_as_float(w.x), __uint_as_float(w.y));
    p[1] = f2_pack(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

constexpr float kFar = 2147483648.0f;   // 2^31 octaves: see Arithmetic
// Whether q has to come from the row instead of its lse (NaN: the row's q are
// NaN either way).
__device__ __forceinline__ bool lse_coarse(float lse) { return fabsf(lse) > 256.0f; }
enum { kSlice = 0, kWhole = 1, kNothing = 2 };   // kGrad: what of a row an item writes

// A thread's pair in base 2: M = max(x c, -kFar), s in two halves.
struct Fold2 {
  float M = -kFar;
  uint64_t ref = f2_pack(kFar, kFar), s = 0;   // ref: (-M, -M)
  __device__ __forceinline__ void raise(float vmax, float c) {
    const float v = vmax * c;
    if (v > M) {
      const float f = ex2_approx(M - v);
      s = f2_mul(s, f2_pack(f, f));
      M = v;
      ref = f2_pack(-v, -v);
    }
  }
  __device__ __forceinline__ void pair(uint64_t x2, uint64_t c2) {
    float lo, hi;
    f2_unpack(f2_fma(x2, c2, ref), lo, hi);
    s = f2_add(s, f2_pack(ex2_approx(lo), ex2_approx(hi)));
  }
};

// The teacher warp's part of a row: probabilities (0 for what is not valid),
// their natural logarithms, the student's logits.  Returns whether there is
// an entry.  Entries outside [b0, b1) need no logit unless `all`.
template <class E>
__device__ __forceinline__ bool teacher_warp(const DistillArgs &a, int64_t row, int lane, int *sidx,
                                             float *sp, float *slp, float *sx, bool all, int64_t b0,
                                             int64_t b1) {
  const E *x = reinterpret_cast<const E *>(a.x) + row * a.ldx;
  float m = -INFINITY, s = 0.0f;
  for (int k = lane; k < a.K; k += 32) {
    int64_t j = load_token(a.idx, a.idx_wide, row * a.K + k, a.V);
    const float y =
        a.t_bf16 ? bf16_f(__ldg(reinterpret_cast<const unsigned short *>(a.t) + row * a.K + k))
                 : __ldg(reinterpret_cast<const float *>(a.t) + row * a.K + k);
    if (y == -INFINITY) j = -1;
    if (j >= 0) {
      const float e[1] = {y};
      ms2_fold<1>(m, s, e, a.c);
    }
    sidx[k] = (int)j;
    slp[k] = y;
    sx[k] = j >= 0 && (all || (j >= b0 && j < b1)) ? value(x + j) : 0.0f;
  }
  ms2_warp(m, s, a.c);
  const float ls = logf(s), inv = 1.0f / s;
  for (int k = lane; k < a.K; k += 32) {
    const float d = slp[k] - m;
    sp[k] = sidx[k] >= 0 ? ex2_approx(d * a.c) * inv : 0.0f;
    slp[k] = d * a.inv_T - ls;
  }
  return !(m == -INFINITY && s == 0.0f);
}

// Sums the probabilities of equal entries, in list order, by one warp: place
// of each distinct entry's sum in `tab` for its first entry of the list, -1
// for the others and for what is outside [b0, b1).
__device__ __forceinline__ void merge_entries(const int *sidx, const float *sp, int K, int64_t b0,
                                              int64_t b1, int *key, float *sum, int *place, int lg,
                                              int lane) {
  const int places = 1 << lg;
  for (int i = lane; i < places; i += 32) {
    key[i] = -1;
    sum[i] = 0.0f;
  }
  __syncwarp();
  for (int b = 0; b < K; b += 32) {
    const int k = b + lane;
    const int j = k < K && sidx[k] >= b0 && sidx[k] < b1 ? sidx[k] : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, j);
    const int lead = __ffs(peers) - 1;
    int at = 0;
    bool fresh = false;
    if (j >= 0 && lane == lead) {
      at = (int)(((uint32_t)j * 2654435761u) >> (32 - lg));
      int old;
      while ((old = atomicCAS(key + at, -1, j)) != -1 && old != j) at = (at + 1) & (places - 1);
      fresh = old == -1;
      float p = sum[at];
      for (uint32_t rest = peers; rest; rest &= rest - 1) p += sp[b + __ffs(rest) - 1];
      sum[at] = p;
    }
    if (k < K) place[k] = fresh ? at : -1;
    __syncwarp();
  }
}

template <class E, int MODE, int T>
__global__ void __launch_bounds__(T + 128)
k_distill_ring(DistillArgs a, RingShape g, int *err) {
  pdl_begin();
  constexpr int N = 16 / (int)sizeof(E), W = T / 32, PU = kRingUnits * T;
  constexpr uint32_t kNone = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;   // -inf
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kRingMaxPieces], empty[kRingMaxPieces];
  // two places each, taken in turn by the items: lists ready, lists read,
  // warps' pairs ready, row's pair ready, dx written; pairs of the peers
  __shared__ __align__(8) uint64_t tfull[2], tfree[2], rfull[2], sfull[2], done[2], xbar[2];
  __shared__ __align__(8) float2 xpair[2][16];
  __shared__ float2 red[2][W];
  __shared__ struct { float m, s; int careful; } stat[2];          // the row's pair
  // grad_out, kGrad's lse, no gradient, what is written
  __shared__ struct { float g, lse; int none, what; } given[2];
  __shared__ int dead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.K;
  const uint32_t C = cluster_nctarank(), r = cluster_ctarank();
  const int64_t item0 = cluster_id_x(), step = cluster_nid_x();
  constexpr size_t piece_bytes = (size_t)PU * 16;
  unsigned char *p = smem + (size_t)g.P * piece_bytes;
  auto carve = [&](size_t n) {
    unsigned char *q = p;
    p += n;
    return q;
  };
  int *const sidx = reinterpret_cast<int *>(carve((size_t)K * 8));
  float *const sp = reinterpret_cast<float *>(carve((size_t)K * 8));
  float *const slp = reinterpret_cast<float *>(carve((size_t)K * 8));
  float *const sx = reinterpret_cast<float *>(carve((size_t)K * 8));
  int *const place = reinterpret_cast<int *>(carve((size_t)K * 4));
  int *const tkey = reinterpret_cast<int *>(carve((size_t)4 << g.lg_tab));
  float *const tsum = reinterpret_cast<float *>(carve((size_t)4 << g.lg_tab));

  if (tid == 0) {
    dead = 0;
    for (int i = 0; i < g.P; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], W);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&rfull[i], W);
      mbar_init(&sfull[i], 1);
      mbar_init(&tfree[i], MODE == kBoth ? 2 : 1);
      mbar_init(&done[i], W);
      mbar_init(&xbar[i], C);
    }
    fence_mbar_init();
  }
  cluster_sync();   // the peers' barriers are ready too
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!mbar_wait_or_die(bar, parity, kWaitBudget, &dead, false)) set_error(err, kErrTimeout);
  };
  auto turn = [](int i) { return (uint32_t)(i >> 1) & 1; };   // parity of item i's place i & 1
  auto arrive = [&](uint64_t *bar) {   // by a warp, when all its lanes are there
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == W) {
    // ---- producer ----
    Cursor q;
    bool laps = false;   // of the ring
    const uint64_t keep = l2_evict_last_policy(), once = l2_evict_first_policy();
    for (int64_t item = item0; item < g.items; item += step) {
      const Part<E> part(a, g, item, (int)r, MODE == kGrad);
      const E *x = reinterpret_cast<const E *>(a.x) + part.row * a.ldx;
      bool unread = false;
      if constexpr (MODE == kGrad) {
        const float gr = a.g[part.row], lse = a.lse[part.row];
        unread = gr == 0.0f || lse_coarse(lse);
      }
      if (unread) {   // zeros, or what the consumers read themselves
        for (int k = 0; k < g.np; ++k, q.next(g.P), laps |= q.slot == 0) {
          wait(&empty[q.slot], q.phase ^ 1);
          if (lane == 0) mbar_arrive(&full[q.slot]);
        }
        continue;
      }
      const int loads = MODE == kBoth ? 2 * g.np : g.np;   // both passes'
      for (int n = 0; n < loads; ++n, q.next(g.P), laps |= q.slot == 0) {
        const int k = n < g.np ? n : n - g.np;
        const int pa = k * PU, pb = min(pa + PU, part.nu);
        unsigned char *dst = smem + (size_t)q.slot * piece_bytes;
        wait(&empty[q.slot], q.phase ^ 1);
        const int wa = max(pa, part.ub), wb = min(pb, part.ue);
        const uint32_t bytes = wb > wa ? (uint32_t)(wb - wa) * 16 : 0;
        for (int e = 0; e < 2; ++e) {   // the partial units
          const int u = e == 0 ? 0 : part.nu - 1;
          const bool mine = (e == 0 ? part.ub == 1 : part.ue < part.nu) && u >= pa && u < pb;
          if (mine && lane < N) {
            const int64_t i = part.first + (int64_t)u * N + lane;
            E *el = reinterpret_cast<E *>(dst) + (u - pa) * N + lane;
            if constexpr (sizeof(E) == 2) *el = (i >= 0 && i < a.V) ? x[i] : (E)0xff80;
            else *el = (i >= 0 && i < a.V) ? x[i] : -INFINITY;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (bytes) {
            mbar_arrive_expect_tx(&full[q.slot], bytes);
            bulk_g2s_hint(dst + (size_t)(wa - pa) * 16,
                          reinterpret_cast<const unsigned char *>(x + part.first) + (size_t)wa * 16,
                          bytes, &full[q.slot], n + g.np < loads ? keep : once);
          } else {
            mbar_arrive(&full[q.slot]);
          }
        }
      }
    }
    // should a wait have given up, no copy is left in flight behind the CTA:
    // the last one into each place that was used
    for (int k = 0; k < g.P; ++k)
      if (k < q.slot) mbar_wait_bounded(&full[k], q.phase, kWaitBudget);
      else if (laps) mbar_wait_bounded(&full[k], q.phase ^ 1, kWaitBudget);
  } else if (warp == W + 1) {
    // ---- teacher ----
    int i = 0;
    for (int64_t item = item0; item < g.items; item += step, ++i) {
      const int h = i & 1;
      const Part<E> part(a, g, item, (int)r, MODE == kGrad);
      int64_t b0 = max(part.first, (int64_t)0), b1 = min(part.first + (int64_t)part.nu * N, a.V);
      if (item + 2 * step < g.items) {   // the lists after the next: from DRAM by then
        const int64_t row = MODE == kGrad ? (item + 2 * step) / g.slices : item + 2 * step;
        const size_t ni = (size_t)K * (a.idx_wide ? 8 : 4), nt = (size_t)K * (a.t_bf16 ? 2 : 4);
        for (size_t o = (size_t)lane * 128; o < ni; o += 4096)
          prefetch_l2(reinterpret_cast<const char *>(a.idx) + row * ni + o);
        for (size_t o = (size_t)lane * 128; o < nt; o += 4096)
          prefetch_l2(reinterpret_cast<const char *>(a.t) + row * nt + o);
      }
      float gr = 0.0f, lse = 0.0f;
      if constexpr (MODE != kLoss) gr = __ldg(a.g + part.row);
      int what = kSlice;
      if constexpr (MODE == kGrad) {
        lse = __ldg(a.lse + part.row);
        if (lse_coarse(lse)) {
          what = item % g.slices == 0 ? kWhole : kNothing;
          b0 = 0;
          b1 = what == kWhole ? a.V : 0;
        }
      }
      if (i >= 2) wait(&tfree[h], turn(i - 2));
      const bool any = teacher_warp<E>(a, part.row, lane, sidx + h * K, sp + h * K, slp + h * K,
                                       sx + h * K, MODE != kGrad && r == 0, b0, b1);
      if (lane == 0) {
        given[h].g = gr;
        given[h].lse = lse;
        given[h].none = !any || (MODE != kLoss && gr == 0.0f);
        given[h].what = what;
      }
      arrive(&tfull[h]);
    }
  } else if (warp == W + 3) {
    // ---- finisher: dx at the entries, behind the dense part ----
    if constexpr (MODE != kLoss) {
      int i = 0;
      for (int64_t item = item0; item < g.items; item += step, ++i) {
        const int h = i & 1;
        const Part<E> part(a, g, item, (int)r, MODE == kGrad);
        int64_t b0 = max(part.first, (int64_t)0), b1 = min(part.first + (int64_t)part.nu * N, a.V);
        wait(&tfull[h], turn(i));
        const bool on = !given[h].none;
        const int what = MODE == kGrad ? given[h].what : kSlice;
        if (what != kSlice) {
          b0 = 0;
          b1 = what == kWhole ? a.V : 0;
        }
        if (on) merge_entries(sidx + h * K, sp + h * K, K, b0, b1, tkey, tsum, place, g.lg_tab, lane);
        wait(&done[h], turn(i));
        if (on) {
          // q from the row's statistics, as pass 2 has it
          const float gt = given[h].g * a.inv_T;
          E *dx = reinterpret_cast<E *>(a.dx) + part.row * a.lddx;
          float gq = 0.0f;
          if (MODE == kBoth || what == kWhole) gq = gt / stat[h].s;
          for (int k = lane; k < K; k += 32) {
            if (place[k] < 0) continue;
            const float v = sx[h * K + k], P = tsum[place[k]];
            float q;
            if (MODE == kGrad && what == kSlice)
              q = ex2_approx(fmaf(v, a.inv_T, -given[h].lse) * kLog2e) * gt;
            else q = (stat[h].careful ? ex2_approx((v - stat[h].m) * a.c)
                                      : ex2_approx(fmaf(v, a.c, -stat[h].m))) * gq;
            put(dx + sidx[h * K + k], q - gt * P);
          }
        }
        arrive(&tfree[h]);
      }
    }
  } else if (warp == W + 2) {
    // ---- exchange ----
    if constexpr (MODE != kGrad) {
      int exchanges = 0;
      // the cluster's pair from the CTAs'; scale as ms2_warp's c
      auto join_pairs = [&](float &m, float &s, float scale) {
        const int e = exchanges & 1;
        if (C == 1) return;
        if (lane < (int)C) {
          st_dsmem_f2(map_peer(smem_u32(&xpair[e][r]), (uint32_t)lane), m, s);
          mbar_arrive_remote(&xbar[e], (uint32_t)lane);
        }
        if (!mbar_wait_or_die(&xbar[e], turn(exchanges), kWaitBudget, &dead, true))
          set_error(err, kErrTimeout);
        m = lane < (int)C ? xpair[e][lane].x : -INFINITY;
        s = lane < (int)C ? xpair[e][lane].y : 0.0f;
        ms2_warp(m, s, scale);
        ++exchanges;
      };
      int i = 0;
      for (int64_t item = item0; item < g.items; item += step, ++i) {
        const int h = i & 1;
        const Part<E> part(a, g, item, (int)r, false);
        wait(&rfull[h], turn(i));
        float m = lane < W ? red[h][lane].x : -INFINITY;
        float s = lane < W ? red[h][lane].y : 0.0f;
        ms2_warp(m, s, 1.0f);
        wait(&tfull[h], turn(i));   // the logits at the entries have been read
        join_pairs(m, s, 1.0f);
        const bool careful = !(fabsf(m) < kFar);
        if (careful) {
          m = -INFINITY;
          s = 0.0f;
          const E *x = reinterpret_cast<const E *>(a.x) + part.row * a.ldx;
          const int64_t b1 = min(part.first + (int64_t)part.nu * N, a.V);
          for (int64_t j = max(part.first, (int64_t)0) + lane; j < b1; j += 32) {
            const float e[1] = {value(x + j)};
            ms2_fold<1>(m, s, e, a.c);
          }
          ms2_warp(m, s, a.c);
          join_pairs(m, s, a.c);
        }
        if (lane == 0) {
          stat[h].m = m;
          stat[h].s = s;
          stat[h].careful = careful;
        }
        arrive(&sfull[h]);
        if (r == 0) {
          const float ls = log2f(s);
          const float lse = careful ? fmaf(m, a.inv_T, ls * kLn2) : (m + ls) * kLn2;
          float sum = 0.0f, any = 0.0f;
          for (int k = lane; k < K; k += 32) {
            const float pk = sp[h * K + k], v = sx[h * K + k];
            any += sidx[h * K + k] >= 0 ? 1.0f : 0.0f;
            if (pk != 0.0f) {
              // past the range of x c, the natural units still hold
              float lq = careful ? (v - m) * a.inv_T - ls * kLn2 : (fmaf(v, a.c, -m) - ls) * kLn2;
              if (lq == -INFINITY && v > -INFINITY) lq = fmaf(v, a.inv_T, -lse);
              sum += pk * (slp[h * K + k] - lq);
            }
          }
          sum = warp_allreduce<SumF32, 32>(sum);
          any = warp_allreduce<SumF32, 32>(any);
          if (lane == 0) {
            a.loss[part.row] = any > 0.0f ? sum : 0.0f;
            a.lse[part.row] = lse;
          }
        }
        arrive(&tfree[h]);
      }
    }
  } else {
    // ---- consumers ----
    const uint4 *ring = reinterpret_cast<const uint4 *>(smem);
    const uint64_t c2 = f2_pack(a.c, a.c), t2 = f2_pack(a.inv_T, a.inv_T), e2 = f2_pack(kLog2e, kLog2e);
    Cursor q;
    // a slice piece by piece: f(first unit, units, its place in the ring)
    auto walk = [&](int nu, auto f) {
      for (int k = 0; k < g.np; ++k, q.next(g.P)) {
        const int pa = k * PU;
        wait(&full[q.slot], q.phase);
        f(pa, min(PU, nu - pa), ring + q.slot * PU);
        arrive(&empty[q.slot]);
      }
    };
    auto pass1 = [&](int64_t item, int i) {
      const int h = i & 1;
      const Part<E> part(a, g, item, (int)r, false);
      Fold2 fold;
      walk(part.nu, [&](int, int n, const uint4 *base) {
        uint4 w[kRingUnits];
#pragma unroll
        for (int j = 0; j < kRingUnits; ++j)
          w[j] = tid + j * T < n ? base[tid + j * T] : make_uint4(kNone, kNone, kNone, kNone);
        float v = unit_max<E>(w[0]);
#pragma unroll
        for (int j = 1; j < kRingUnits; ++j) v = fmaxf(v, unit_max<E>(w[j]));
        fold.raise(v, a.c);
#pragma unroll
        for (int j = 0; j < kRingUnits; ++j) {
          uint64_t pr[N / 2];
          unit_pairs<E>(w[j], pr);
#pragma unroll
          for (int k = 0; k < N / 2; ++k) fold.pair(pr[k], c2);
        }
      });
      float m = fold.M, s, s2;
      f2_unpack(fold.s, s, s2);
      s += s2;
      ms2_warp(m, s, 1.0f);
      if (i >= 2) wait(&sfull[h], turn(i - 2));   // the place has been read
      if (lane == 0) red[h][warp] = make_float2(m, s);
      arrive(&rfull[h]);
    };
    auto pass2 = [&](int64_t item, int i) {
      const int h = i & 1;
      const Part<E> part(a, g, item, (int)r, MODE == kGrad);
      wait(MODE == kGrad ? &tfull[h] : &sfull[h], turn(i));
      const bool none = given[h].none, careful = MODE == kBoth && stat[h].careful;
      const float gt = none ? 0.0f : given[h].g * a.inv_T, lse = given[h].lse;
      float gq = gt, m = 0.0f;
      if constexpr (MODE == kBoth) {
        m = stat[h].m;
        gq = gt / stat[h].s;
      }
      E *dx = reinterpret_cast<E *>(a.dx) + part.row * a.lddx;
      const bool same = ((uintptr_t)(dx + part.first) & 15) == 0;
      const uint64_t g2 = f2_pack(gq, gq), m2 = f2_pack(-m, -m), l2 = f2_pack(-lse, -lse);
      auto one = [&](float v) {
        if constexpr (MODE == kGrad) return ex2_approx(fmaf(v, a.inv_T, -lse) * kLog2e) * gq;
        else return (careful ? ex2_approx((v - m) * a.c) : ex2_approx(fmaf(v, a.c, -m))) * gq;
      };
      // dx of a unit
      auto rewrite = [&](const uint4 &w) {
        float e[N];
        uint64_t pr[N / 2];
        unit_pairs<E>(w, pr);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const uint64_t y = MODE == kGrad ? f2_mul(f2_fma(pr[k], t2, l2), e2) : f2_fma(pr[k], c2, m2);
          float lo, hi;
          f2_unpack(y, lo, hi);
          f2_unpack(f2_mul(f2_pack(ex2_approx(lo), ex2_approx(hi)), g2), e[2 * k], e[2 * k + 1]);
        }
        if constexpr (sizeof(E) == 2)
          return make_uint4(bf16x2_bits(e[0], e[1]), bf16x2_bits(e[2], e[3]), bf16x2_bits(e[4], e[5]),
                            bf16x2_bits(e[6], e[7]));
        else
          return join<E, N>(e);
      };
      const int what = MODE == kGrad && !none ? given[h].what : kSlice;
      if (what != kSlice) {
        walk(part.nu, [](int, int, const uint4 *) {});
        if (what == kWhole) {
          const E *x = reinterpret_cast<const E *>(a.x) + part.row * a.ldx;
          float M = -INFINITY, s = 0.0f;
          each_of_row(
              x, a.V, tid, T,
              [&](int64_t, float v) {
                const float e[1] = {v};
                ms2_fold<1>(M, s, e, a.c);
              },
              [&](int64_t, const uint4 &w) {
                float e[N];
                split<E, 16>(w, e);
                ms2_fold<N>(M, s, e, a.c);
              });
          ms2_warp(M, s, a.c);
          if (lane == 0) red[h][warp] = make_float2(M, s);
          named_sync(1, T);   // and the row has been read
          M = lane < W ? red[h][lane].x : -INFINITY;
          s = lane < W ? red[h][lane].y : 0.0f;
          ms2_warp(M, s, a.c);
          if (tid == 0) {
            stat[h].m = M;
            stat[h].s = s;
            stat[h].careful = 1;
          }
          const float f = gt / s;
          each_of_row(
              x, a.V, tid, T, [&](int64_t j, float v) { put(dx + j, ex2_approx((v - M) * a.c) * f); },
              [&](int64_t j, const uint4 &w) {
                float e[N];
                split<E, 16>(w, e);
#pragma unroll
                for (int k = 0; k < N; ++k) e[k] = ex2_approx((e[k] - M) * a.c) * f;
                if (same) {
                  *reinterpret_cast<uint4 *>(dx + j) = join<E, N>(e);
                } else {
#pragma unroll
                  for (int k = 0; k < N; ++k) put(dx + j + k, e[k]);
                }
              });
          named_sync(1, T);   // red is free
        }
        arrive(&done[h]);
        return;
      }
      const bool plain = same && !none && !careful;
      walk(part.nu, [&](int pa, int n, const uint4 *base) {
        uint4 *dv = reinterpret_cast<uint4 *>(dx + part.first) + pa + tid;
        if (plain && n == PU && pa >= part.ub && pa + PU <= part.ue) {
          uint4 w[kRingUnits];
#pragma unroll
          for (int j = 0; j < kRingUnits; ++j) w[j] = base[tid + j * T];
#pragma unroll
          for (int j = 0; j < kRingUnits; ++j) __stcs(dv + j * T, rewrite(w[j]));
          return;
        }
        if (same) {
          for (int t = tid; t < n; t += T) {
            const int u = pa + t;
            if (u >= part.ub && u < part.ue) {
              uint4 out = make_uint4(0, 0, 0, 0);
              if (plain) {
                out = rewrite(base[t]);
              } else if (!none) {
                float e[N];
                split<E, 16>(base[t], e);
#pragma unroll
                for (int j = 0; j < N; ++j) e[j] = one(e[j]);
                out = join<E, N>(e);
              }
              __stcs(dv + (t - tid), out);
            } else {
              const E *el = reinterpret_cast<const E *>(base + t);
              const int64_t k0 = part.first + (int64_t)u * N;
              for (int j = 0; j < N; ++j)
                if (k0 + j >= 0 && k0 + j < a.V) put(dx + k0 + j, none ? 0.0f : one(value(el + j)));
            }
          }
          return;
        }
        // dx starts elsewhere in a unit: element by element
        const E *el = reinterpret_cast<const E *>(base);
        for (int t = tid; t < n * N; t += T) {
          const int64_t k = part.first + (int64_t)pa * N + t;
          if (k >= 0 && k < a.V) put(dx + k, none ? 0.0f : one(value(el + t)));
        }
      });
      arrive(&done[h]);   // dx's dense part is written
    };
    int i = 0;
    for (int64_t item = item0; item < g.items; item += step, ++i) {
      if constexpr (MODE != kGrad) pass1(item, i);
      if constexpr (MODE != kLoss) pass2(item, i);
    }
  }
  __syncwarp();
  cluster_sync();   // no CTA leaves while a peer may send to it
}

template <class E, int MODE, int T>
int ring_launch(const DistillArgs &a, RingShape g, int C, size_t room, int64_t rows, cudaStream_t s,
                const DevInfo &d) {
  auto kern = k_distill_ring<E, MODE, T>;
  constexpr int PU = kRingUnits * T;
  constexpr size_t piece = (size_t)PU * 16;
  g.np = (g.slice_units + PU - 1) / PU;
  g.lg_tab = 5;
  while ((1 << g.lg_tab) < 2 * a.K) ++g.lg_tab;
  const size_t lists = (size_t)a.K * 36 + ((size_t)8 << g.lg_tab);
  while (room < kRingSmem && room < lists + 3 * piece) room *= 2;   // long lists
  if (room > kRingSmem) room = kRingSmem;
  g.P = (int)((room - lists) / piece);
  if (g.P > kRingMaxPieces) g.P = kRingMaxPieces;
  const size_t smem = g.P * piece + lists;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_kernel(kern, kRingSmem, true, d.device, allowed);
  if (e != cudaSuccess) return cuda_status(e);
  int64_t clusters = occupancy_clusters((const void *)kern, T + 128, smem, C, d.device);
  if (clusters < 1) return RR_ERR_UNSUPPORTED;
  if (clusters > g.items) clusters = g.items;
  if (log_enabled())
    std::fprintf(stderr,
                 "[rr] distill mode=%d rows=%lld V=%lld K=%d C=%d clusters=%lld slice=%d units, %d pieces of "
                 "%d, ring of %d, threads=%d smem=%zu\n",
                 MODE, (long long)rows, (long long)a.V, a.K, C, (long long)clusters, g.slice_units, g.np,
                 PU, g.P, T, smem);
  return cuda_status(launch_kernel(kern, dim3((unsigned)(clusters * C)), dim3(T + 128), smem, s, C, a, g,
                                   d.err_word));
}

// Consumer threads and shared memory of a CTA by its slice (16-byte units).
// Measured, 2^30 elements of bf16 in rows of 131072 / 32768 / 8192 (16384 /
// 4096 / 1024 units), GB/s:
//   loss and gradient  512 threads, 224 KiB: 6580 / 5540 / -;  256, 112 KiB:
//                      5280 / 5970 / 3880;  128, 56 KiB: - / 5990 / 4630
//   loss               256, 56 KiB: 7000 / 4580 / -;  128, 37 KiB: 6840 / 5520 / 2850
//   gradient           256, 74 KiB: 6350;  512, 224 KiB: 5940;  128, 56 KiB: 6330
struct RingSize {
  int T;
  size_t room;
};
RingSize ring_size(int mode, int64_t slice) {
  if (mode == kLoss) return slice > 6144 ? RingSize{256, 56 << 10} : RingSize{128, 37 << 10};
  if (mode == kGrad) return slice > 1536 ? RingSize{256, 74 << 10} : RingSize{128, 56 << 10};
  if (slice > 6144) return {512, kRingSmem};
  return slice > 1536 ? RingSize{256, 112 << 10} : RingSize{128, 56 << 10};
}

template <class E, int MODE>
int ring_plan(const DistillArgs &a, int64_t rows, cudaStream_t s, const DevInfo &d) {
  constexpr int64_t N = 16 / (int64_t)sizeof(E);
  // units of a row, the most at any of the rows' addresses
  const bool flush = (uintptr_t)a.x % 16 == 0 && (rows == 1 || (a.ldx * (int64_t)sizeof(E)) % 16 == 0);
  const int64_t units = flush ? (a.V + N - 1) / N : (a.V + 2 * N - 2) / N;
  auto slice = [&](int64_t n) { return (units + n - 1) / n; };
  auto resident = [&](int64_t n) {   // CTAs on the GPU
    return d.sm_count * (int64_t)(kRingSmem / ring_size(MODE, slice(n)).room);
  };
  RingShape g = {};
  g.slices = 1;
  int C = 1;
  if (MODE == kGrad) {
    // slices of at most 64 KiB, shorter ones while no CTA has four
    int64_t n = slice(4096);
    while (rows * n < 8 * d.sm_count && slice(n + 1) >= 512) ++n;
    g.slices = (int)n;
    g.items = rows * n;
  } else {
    const int most = d.cluster_launch ? (cluster_cap() < 16 ? cluster_cap() : 16) : 1;
    // rows in flight within the L2 (kBoth reads them twice): 262144 bf16, 76
    // MiB with a CTA a row, 781 us and with two 687; 10^6 bf16, with 1 / 2 / 4 /
    // 8 CTAs 936 / 902 / 707 / 845 (2^30 elements)
    if (MODE == kBoth)
      while (C * 2 <= most && slice(C) * 16 * resident(C) > (int64_t(75) << 20)) C *= 2;
    // every SM at work: 16 rows of 131072 bf16 with 4 / 8 / 16 CTAs 7.2 / 7.0 /
    // 7.4 us
    while (C * 2 <= most && rows * C * 2 <= (MODE == kBoth ? resident(C) : 2 * d.sm_count) &&
           slice(C * 2) >= 1024)
      C *= 2;
    if (slice(C) > INT_MAX / 2) return RR_ERR_UNSUPPORTED;
    g.items = rows;
  }
  for (;;) {
    const int64_t n = MODE == kGrad ? g.slices : C;
    g.slice_units = (int)slice(n);
    const RingSize z = ring_size(MODE, slice(n));
    int st;
    if (z.T == 128) st = ring_launch<E, MODE, 128>(a, g, C, z.room, rows, s, d);
    else if (z.T == 256 || MODE != kBoth) st = ring_launch<E, MODE, 256>(a, g, C, z.room, rows, s, d);
    else st = ring_launch<E, MODE, MODE == kBoth ? 512 : 256>(a, g, C, z.room, rows, s, d);
    if (st != RR_ERR_UNSUPPORTED || C == 1) return st;
    C /= 2;   // a cluster that cannot run here
  }
}
}  // namespace

int launch_distill(const DistillArgs &a, int dtype, int64_t rows, cudaStream_t s, const DevInfo &d) {
  if (dtype == RR_BF16)
    return a.dx ? ring_plan<unsigned short, kBoth>(a, rows, s, d) : ring_plan<unsigned short, kLoss>(a, rows, s, d);
  return a.dx ? ring_plan<float, kBoth>(a, rows, s, d) : ring_plan<float, kLoss>(a, rows, s, d);
}

int launch_distill_grad(const DistillArgs &a, int dtype, int64_t rows, cudaStream_t s, const DevInfo &d) {
  return dtype == RR_BF16 ? ring_plan<unsigned short, kGrad>(a, rows, s, d)
                          : ring_plan<float, kGrad>(a, rows, s, d);
}

}  // namespace rr
