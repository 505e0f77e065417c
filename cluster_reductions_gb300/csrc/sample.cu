// sample.cu -- a token from each row of logits with temperature, top-k,
// top-p and min-p, drawn with a given uniform number.
//
//   w_j = exp((x_j - max x) / T); tokens are ordered by (x descending, index
//   ascending).  top-k keeps the first k; top-p keeps those of them before
//   which less than top_p of their mass lies; min-p keeps those with
//   w_j >= min_p.  The token is the first kept one, in index order, whose
//   running mass exceeds u times the kept mass.
//
// A token is a whole number, so the answer has to be the one that exact
// arithmetic gives.  fp32 sums over 10^5 weights are off by 1e-7 of the
// total and would choose a neighbour in some per cent of the rows.  So the
// weights are whole numbers of 2^-K of the largest, K = 61 - ceil(log2 V), and
// every sum is a 64-bit integer sum: exact, and the same however the row is
// split.  A weight is right to about 2^-31 of itself and, cut to a whole number,
// to 2^-K of the largest (44 bits at V = 131072, 41 at 2^20); together the cuts
// are less than V 2^-K of the mass (2^-27 and 2^-21), by which the draw or the
// end of top-p can differ from what exact weights would give.
//
// The weight.  With t = (x - max) * 256 log2(e) / T taken in two floats
// (hi = the nearest whole number, g the rest), w = 2^(hi/256) * 2^(g/256):
// 2^((hi mod 256)/256) from a table of 31-bit whole numbers, 2^(g/256) - 1 (at
// most 0.0014) from three terms of its series, their product in 64 bits.
//
// What bounds it: integer instructions and the chain of a row's phases, not
// DRAM (each row is read two or three times, after the first out of L2).  Of
// 36 K cycles that a row of 32003 bf16 alone on an SM takes under top-p, the
// maximum is 3 K, counting the values 8 K, weighing 4096 bins and finding the
// cut 9 K, the kept mass by segment 8 K, the draw 4 K.  Measured: 512 such rows
// 49 us (665 GB/s), 256 x 131072 bf16 with mixed settings 65 us, 64 x 100003
// fp32 without filters 18.3 us, 1 x 131072 bf16 under top-k and top-p 15 us.
#include <climits>
#include <cstdio>

#include "rr.h"
#include "rr_internal.h"
#include "token.cuh"

namespace rr {
namespace {

// ---- weights ----------------------------------------------------------------
// 2^(i/256) * 2^30, rounded; by repeated square roots (Newton) and products
// at compile time.
struct Pow2Table {
  uint32_t v[256];
};
constexpr double ct_sqrt(double a) {
  double r = a;
  for (int i = 0; i < 60; ++i) r = 0.5 * (r + a / r);
  return r;
}
constexpr Pow2Table make_table() {
  Pow2Table t{};
  double root = 2.0;
  for (int i = 0; i < 8; ++i) root = ct_sqrt(root);   // 2^(1/256)
  // i = 16 a + b: errors of at most 30 products of 2^-53
  double coarse = 1.0, step = 1.0;
  for (int i = 0; i < 16; ++i) step *= root;
  for (int a = 0; a < 16; ++a) {
    double f = coarse;
    for (int b = 0; b < 16; ++b) {
      t.v[16 * a + b] = (uint32_t)(f * 1073741824.0 + 0.5);
      f *= root;
    }
    coarse *= step;
  }
  return t;
}
__constant__ Pow2Table c_pow2 = make_table();

constexpr float kMagic = 12582912.0f;             // 1.5 * 2^23: its sums are whole
constexpr int kMagicBits = 0x4b400000;
constexpr float kLargest = 3.402823466e38f;

// p >> n, 0 for n >= 64 (C++ leaves that open, the instruction does not).
__device__ __forceinline__ uint64_t shift_right(uint64_t p, int n) {
  uint64_t r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(n));
  return r;
}

// The row's scale: t = (x - m) c in 1/256 octaves, c = chi + clo.  With
// |m c| < 2^21 x c is cut into its nearest whole number and a rest, and m c
// (whole part in off, rest in the row's table) taken from them: sub is 0.
// Else sub is m: then every x that has weight lies within m / 128 of m, so
// x - m is exact.
struct RowScale {
  float m, sub, chi, clo;
  float off;     // magic - the whole part of m c
  float low;     // x below it has weight 0 (62 - base octaves)
  int base;      // 61 - K

  // whole part of t: at most 1, monotone in x; x >= low
  __device__ __forceinline__ int whole(float x) const {
    return __float_as_int(fmaf(fminf(x, kLargest) - sub, chi, off)) - kMagicBits;
  }
  // the weight of x >= low, by the row's table tab of 2^(i/256) 2^30 (times
  // 2^(-rest of m c))
  __device__ __forceinline__ uint64_t weight(float x, const uint32_t *tab) const {
    int bits;
    const uint64_t p = product(x, tab, bits);
    return shifted(p, bits);
  }
  __device__ __forceinline__ uint64_t shifted(uint64_t p, int bits) const {
    return shift_right(p, base + (kMagicBits >> 8) - (bits >> 8));   // (no borrow: the magic's low 22 bits are 0)
  }
  // the same before its shift: about 2^61 times 2^((hi & 255) / 256) (within
  // 2^(1/256) of it), hi = whole(x) = bits - kMagicBits
  __device__ __forceinline__ uint64_t product(float x, const uint32_t *tab, int &bits) const {
    const float d = fminf(x, kLargest) - sub;
    const float hm = fmaf(d, chi, off);
    const float g = fmaf(d, clo, fmaf(d, chi, off - hm));
    bits = __float_as_int(hm);
    // (2^(g/256) - 1) * 2^31 = 2^31 (L + (L^2/2 + L^3/6 g) g) g, L = ln 2 / 256
    constexpr double L = 0.69314718055994530942 / 256, B = 2147483648.0;
    constexpr float a1 = (float)(L * B), a2 = (float)(L * L / 2 * B), a3 = (float)(L * L * L / 6 * B);
    const float em = fmaf(fmaf(fmaf(a3, g, a2), g, a1), g, kMagic);
    const uint32_t e = (uint32_t)__float_as_int(em) + (0x80000000u - (uint32_t)kMagicBits);
    return (uint64_t)tab[bits & 255] * e;
  }
};

// The scale of a row of maximum m (finite) at temperature T > 0 (inv: 1 / T),
// and its table, by all threads; a barrier has to follow.  In pairs of fp32:
// fp64 has so few units here that this alone took 16 us in it.
template <int T>
__device__ __forceinline__ RowScale make_scale(float m, float temp, float inv, int base, uint32_t *tab) {
  constexpr double c1 = 369.32993046757463;         // 256 log2(e)
  constexpr float kh = (float)c1, kl = (float)(c1 - (double)kh);
  RowScale r;
  r.m = m;
  r.base = base;
  r.chi = fminf(kh * inv, 1e37f);
  // what is left of kh + kl after chi T, by inv; past inv's range there is none
  r.clo = r.chi < 1e37f && r.chi > 1e-30f ? (fmaf(-r.chi, temp, kh) + kl) * inv : 0.0f;
  const float mh = m * r.chi, ml = fmaf(m, r.chi, -mh) + m * r.clo;
  const bool wide = !(fabsf(mh) < 2097152.0f);
  const float whole = wide ? 0.0f : rintf(mh);
  r.sub = wide ? m : 0.0f;
  r.off = kMagic - whole;
  r.low = fmaxf(fmaf((float)(base - 62) * (256.0f / kh), temp, m), -kLargest);
  // 2^(-rest / 256) * 2^31; the same factor in every weight, so what its
  // series leaves out does not matter
  const float rest = wide ? 0.0f : (mh - whole) + ml;
  const float z = -rest * (float)(0.69314718055994530942 / 256);
  const float f1 = z * fmaf(z, fmaf(z, 1.0f / 6, 0.5f), 1.0f);
  const uint64_t f = (uint64_t)((int64_t)2147483648ll + __float2int_rn(f1 * 2147483648.0f));
  for (int i = threadIdx.x; i < 256; i += T)
    tab[i] = (uint32_t)(((uint64_t)c_pow2.v[i] * f + (1u << 30)) >> 31);
  return r;
}

// log(w / total), w <= total: from the difference where the quotient is near 1.
__device__ __forceinline__ float log_share(uint64_t w, uint64_t total) {
  const float t = __ull2float_rn(total);
  return w > total / 2 ? log1pf(-__ull2float_rn(total - w) / t) : logf(__ull2float_rn(w) / t);
}

// The entry of wt, whose masses go on from e, that holds the target (its mass
// in w), or -1.
template <int P>
__device__ __forceinline__ int entry_at(const uint64_t (&wt)[P], uint64_t e, uint64_t target, uint64_t &w) {
  int at = -1;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (e <= target && target < e + wt[i]) {
      at = i;
      w = wt[i];
    }
    e += wt[i];
  }
  return at;
}

// Order of the values as whole numbers.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);   // -0 ties with +0
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// ceil(f * z) for f in (0, 1) and floor of the same, z < 2^63.
__device__ __forceinline__ uint64_t scaled(float f, uint64_t z, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const uint64_t mant = (b & 0x7fffff) | (ex ? 0x800000 : 0);
  const int q = 150 - (ex ? ex : 1);              // f = mant * 2^-q, q >= 24
  const uint64_t lo = mant * z, hi = __umul64hi(mant, z);
  if (q >= 128) return up ? 1 : 0;
  uint64_t r, rest;
  if (q >= 64) {
    r = q == 64 ? hi : hi >> (q - 64);
    rest = lo | (q == 64 ? 0 : hi & (((uint64_t)1 << (q - 64)) - 1));
  } else {
    r = (hi << (64 - q)) | (lo >> q);
    rest = lo & (((uint64_t)1 << q) - 1);
  }
  return r + (up && rest ? 1 : 0);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// ---- the row ------------------------------------------------------------------
// The row seen in 16-byte units: unit u holds elements u * N - off + j, the
// first and last ones in part.  What lies outside the row reads as -inf,
// which has no weight and no place in the order.
//
// A warp takes kSub x 32 units together (a segment): in index order, that is
// by (segment, 32 units, lane, element).
template <class E, int kSub>
struct Row {
  static constexpr int N = 16 / (int)sizeof(E), kSegUnits = 32 * kSub;
  const E *x;
  int V, off, units;
  uint4 *edge;          // shared: the first and the last unit
  __device__ Row(const E *p, int v, uint4 *e) : x(p), V(v), edge(e) {
    off = (int)(((uintptr_t)p & 15) / sizeof(E));
    units = (V + off + N - 1) / N;
  }
  // fills `edge`; a barrier has to follow
  __device__ __forceinline__ void load_edges() const {
    if (threadIdx.x < 2 * N) {
      const int u = threadIdx.x < N ? 0 : units - 1, j = threadIdx.x & (N - 1), i = first(u) + j;
      E *e = reinterpret_cast<E *>(edge) + threadIdx.x;
      if constexpr (sizeof(E) == 2) *e = i >= 0 && i < V ? x[i] : (E)0xff80;
      else *e = i >= 0 && i < V ? x[i] : -INFINITY;
    }
  }
  __device__ __forceinline__ int first(int u) const { return u * N - off; }
  __device__ __forceinline__ uint4 raw(int u) const {
    constexpr uint32_t kNone = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;   // -inf
    if (u >= units) return make_uint4(kNone, kNone, kNone, kNone);
    if (u == 0 || u == units - 1) return edge[u != 0];
    return __ldg(reinterpret_cast<const uint4 *>(x + first(u)));
  }
  // the segment's part of this lane: units u, u + 32, ...
  __device__ __forceinline__ void segment(int u, uint4 (&w)[kSub]) const {
    const int s0 = u - (int)(threadIdx.x & 31);   // the segment's first unit
    if (first(s0) >= 0 && first(s0 + kSegUnits) <= V) {
      const uint4 *p = reinterpret_cast<const uint4 *>(x + first(u));
#pragma unroll
      for (int b = 0; b < kSub; ++b) w[b] = __ldg(p + 32 * b);
    } else {
#pragma unroll
      for (int b = 0; b < kSub; ++b) w[b] = raw(u + 32 * b);
    }
  }
  __device__ __forceinline__ void values(const uint4 &w, float (&e)[N]) const {
    split<E, 16>(w, e);
  }
  // the largest element of a unit; NaN when there is one
  __device__ __forceinline__ float largest(const uint4 &w) const {
    float v;
    if constexpr (sizeof(E) == 2) {
      const uint32_t h = max2(max2(w.x, w.y), max2(w.z, w.w));
      v = max_nan(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
    } else {
      v = max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                  max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    return v;
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // f(unit, its 16 bytes) for a segment's part, one after the other (a loop,
  // for the code's size)
  template <class F>
  static __device__ __forceinline__ void parts(int u, uint4 (&w)[kSub], F f) {
#pragma unroll 1
    for (int b = 0; b < kSub; ++b) {
      f(u + 32 * b, w[0]);
#pragma unroll
      for (int k = 1; k < kSub; ++k) w[k - 1] = w[k];
    }
  }
  // f(first unit of the lane, its kSub units of a segment) for segments [a, b),
  // one after the other to a warp of T threads
  template <int T, class F>
  __device__ __forceinline__ void each(int a, int b, F f) const {
#pragma unroll 1
    for (int g = a + (int)(threadIdx.x >> 5); g < b; g += T / 32) {
      const int u = g * kSegUnits + (int)(threadIdx.x & 31);
      uint4 w[kSub];
      segment(u, w);
      f(u, w);
    }
  }
};

constexpr int kBins = 4096;   // of 1/64 octave below the maximum, the first of 1/256
constexpr int kCap = 2048;    // entries of the sorted list
constexpr int kWhole = 512;   // of one that holds all that is kept
constexpr int kShort = 128;   // of one that a warp sorts alone
constexpr size_t kSampleSmem = 200 << 10;

// A prefix of the order: every token with key above `key`, and the first
// `ties` of those at it.
struct Cut {
  uint32_t key;
  uint32_t ties;     // UINT32_MAX: no cut, everything is kept
  uint64_t mass;     // of the prefix
};

template <int T>
struct Shared {
  uint64_t nears[kCap];       // the list of the values nearest to 0
  uint32_t cnt[kBins];
  union {
    uint64_t mass[kBins];     // the narrowing's
    uint64_t list[kCap];
  };
  uint32_t tab[256];
  uint64_t wa[32], wb[32], wc[32];
  uint4 edge[2];
  uint4 order;                // what the first CTA wants of this one: x 0 nothing
  float peak;                 // the CTA's maximum
  float best[T];              // its threads'
  uint64_t near;              // its mass of the values nearest to 0
  Cut cut;                    // the first CTA's
  int keyed;
  int found, found2;
  uint32_t fcnt, n, lo, hi;
  uint64_t fmass;
};

// Exclusive sums of two numbers over the block, and their totals.
template <int T>
__device__ __forceinline__ void block_scan(uint64_t &a, uint64_t &b, uint64_t &ta, uint64_t &tb,
                                           Shared<T> &sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint64_t ia = warp_scan(a, lane), ib = warp_scan(b, lane);
  __syncthreads();
  if (lane == 31) {
    sh.wa[w] = ia;
    sh.wb[w] = ib;
  }
  __syncthreads();
  const uint64_t va = lane < T / 32 ? sh.wa[lane] : 0, vb = lane < T / 32 ? sh.wb[lane] : 0;
  const uint64_t sa = warp_scan(va, lane), sb = warp_scan(vb, lane);
  ta = __shfl_sync(0xffffffffu, sa, 31);
  tb = __shfl_sync(0xffffffffu, sb, 31);
  a = ia - a + __shfl_sync(0xffffffffu, sa - va, w);
  b = ib - b + __shfl_sync(0xffffffffu, sb - vb, w);
}

// The block's sum, in every thread.
template <int T>
__device__ __forceinline__ uint64_t block_total(uint64_t v, Shared<T> &sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.wa[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < T / 32 ? sh.wa[threadIdx.x & 31] : 0);
}

template <int T>
__device__ __forceinline__ void clear_counts(Shared<T> &sh) {
  for (int i = threadIdx.x; i < kBins; i += T) sh.cnt[i] = 0;
  __syncthreads();
}

// (64 bins are an octave of the weights: bins 1 to 64 are shifted by one more
// than bin 0, and so on)
__device__ __forceinline__ int bin_of(int whole) { return min((max(-whole, 0) + 3) >> 2, kBins - 1); }

// The bins between which the shortest prefix of `want` mass ends: [found,
// found2]; found = -1 when there is less than `want`.  n receives the tokens
// up to found2, or some more.  sh.cnt[b] is the sum of bin b's products (see
// RowScale) without their low 31 + base bits, so that V of them stay below
// 2^32: a product is q 2^(31 + base) and less than one unit more, a weight is
// that shifted right by base + o, o the bin's octave, and less than 1 less.
// The tokens of the bin are at most its sum over the least q, 2^(30 - base)
// less 0.4%.
template <int T>
__device__ __forceinline__ void bracket(Shared<T> &sh, uint64_t want, int base) {
  constexpr int W = T / 32, PER = kBins / T;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, b0 = w * (kBins / W) + lane;
  auto bounds = [&](int b, uint64_t &up, uint64_t &down, uint32_t &n) {
    const uint64_t q = sh.cnt[b];
    const int s = 31 - (b + 63) / 64;
    n = q ? (uint32_t)((q >> (30 - base)) + (q >> (36 - base)) + 2) : 0;
    const uint64_t lo = s >= 0 ? q << s : q >> -s;
    up = q ? (s >= 0 ? (q + n) << s : ((q + n) >> -s) + 1) : 0;
    down = lo > n ? lo - n : 0;
  };
  uint64_t up = 0, down = 0;
  uint32_t cnt = 0;
#pragma unroll 1
  for (int i = 0; i < PER; ++i) {
    uint64_t u, d;
    uint32_t n;
    bounds(b0 + 32 * i, u, d, n);
    up += u;
    down += d;
    cnt += n;
  }
  up = warp_sum(up);
  down = warp_sum(down);
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) {
    sh.wa[w] = up;
    sh.wb[w] = down;
    sh.wc[w] = cnt;
  }
  if (threadIdx.x == 0) sh.found = -1;
  __syncthreads();
  const uint64_t vu = lane < W ? sh.wa[lane] : 0, vd = lane < W ? sh.wb[lane] : 0;
  const uint32_t vc = lane < W ? (uint32_t)sh.wc[lane] : 0;
  uint64_t eu = warp_sum(lane < w ? vu : 0), ed = warp_sum(lane < w ? vd : 0);
  const uint64_t td = warp_sum(vd);
  uint32_t ec = __reduce_add_sync(0xffffffffu, lane < w ? vc : 0);
  const uint32_t tc = __reduce_add_sync(0xffffffffu, vc);
  if (threadIdx.x == 0 && td < want) {   // the upper bounds alone may reach it
    sh.found2 = kBins - 1;
    sh.n = tc;
  }
  const bool first = eu < want && eu + up >= want, last = ed < want && ed + down >= want;
  if (first || last) {   // in this warp's stretch
    bool open1 = first, open2 = last;
#pragma unroll 1
    for (int i = 0; i < PER && (open1 || open2); ++i) {
      const int b = b0 + 32 * i;
      uint64_t u, d;
      uint32_t n;
      bounds(b, u, d, n);
      const uint64_t iu = eu + warp_scan(u, lane), id = ed + warp_scan(d, lane);
      const uint32_t ic = ec + (uint32_t)warp_scan((uint64_t)n, lane);
      const uint32_t over1 = __ballot_sync(0xffffffffu, iu >= want);
      const uint32_t over2 = __ballot_sync(0xffffffffu, id >= want);
      if (open1 && over1) {
        if (lane == __ffs(over1) - 1) sh.found = b;
        open1 = false;
      }
      if (open2 && over2) {
        if (lane == __ffs(over2) - 1) {
          sh.found2 = b;
          sh.n = ic;
        }
        open2 = false;
      }
      eu = __shfl_sync(0xffffffffu, iu, 31);
      ed = __shfl_sync(0xffffffffu, id, 31);
      ec = __shfl_sync(0xffffffffu, ic, 31);
    }
  }
  __syncthreads();
}

// bracket() by count: one bin.
template <int T>
__device__ __forceinline__ void count_bin(Shared<T> &sh, uint32_t want) {
  constexpr int PER = kBins / T;
  const int b0 = threadIdx.x * PER, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) c += sh.cnt[b0 + i];
  uint32_t incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.wa[w] = incl;
  if (threadIdx.x == 0) sh.found = -1;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < w ? (uint32_t)sh.wa[lane] : 0u);
  uint32_t e = before + incl - c;
  if (e < want && e + c >= want) {
    int b = b0;
    while (e + sh.cnt[b] < want) e += sh.cnt[b++];
    sh.found = sh.found2 = b;
    sh.n = e + sh.cnt[b];
  }
  __syncthreads();
}

// Ascending order of list[0 .. n), n <= kCap (bitonic; filled up to a power
// of two).
template <int T>
__device__ __forceinline__ void sort_list(uint64_t *list, int n) {
  int size = 64;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += T) list[i] = ~0ull;
  __syncthreads();
  if (size == 64) {   // one warp, a pair a lane
    if (threadIdx.x < 32) {
      for (int k = 2; k <= 64; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          const int t = threadIdx.x, a = 2 * t - (t & (j - 1)), b = a + j;
          const uint64_t x = list[a], y = list[b];
          if ((x > y) == ((a & k) == 0)) {
            list[a] = y;
            list[b] = x;
          }
          __syncwarp();
        }
    }
    __syncthreads();
    return;
  }
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int t = threadIdx.x; t < size / 2; t += T) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;
        const uint64_t x = list[a], y = list[b];
        if ((x > y) == ((a & k) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
}

// Ascending order of kShort entries in a warp's registers, entry lane * P + i
// in v[i] of a lane (bitonic; strides below P inside the lane, the others by
// shuffles).
constexpr int kShortLane = kShort / 32;
__device__ __forceinline__ void sort_short(uint64_t (&v)[kShortLane]) {
  constexpr int P = kShortLane;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int k = 2; k <= kShort; k *= 2) {
#pragma unroll 1
    for (int j = k / 2; j >= P; j /= 2) {
      // the lower place keeps the smaller where bit k of its index is clear
      const bool small = ((lane * P & k) == 0) == ((lane * P & j) == 0);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, v[i], j / P);
        v[i] = (v[i] < o) == small ? v[i] : o;
      }
    }
#pragma unroll
    for (int j = P / 2; j > 0; j /= 2) {
      if (j >= k) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (i & j) continue;
        const bool up = ((lane * P + i) & k) == 0;
        const uint64_t a = v[i], b = v[i + j];
        v[i] = (a < b) == up ? a : b;
        v[i + j] = (a < b) == up ? b : a;
      }
    }
  }
}

// The cut at `want` tokens or mass inside a list sorted by order, before which
// lie `count` tokens and `mass`.  *last: its last entry that is kept.
template <int T, class W>
__device__ __forceinline__ Cut cut_in_list(const uint64_t *list, int n, uint64_t count, uint64_t mass,
                                           bool by_mass, uint64_t want, Shared<T> &sh, int *last, W weight) {
  constexpr int PER = kCap / T;
  uint64_t wt[PER], s = 0, none = 0, total, tn;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = (int)threadIdx.x * PER + i;
    key[i] = at < n ? ~(uint32_t)(list[at] >> 32) : 0;
    wt[i] = at < n ? weight(of_key(key[i])) : 0;   // in range: x >= low
    s += wt[i];
  }
  block_scan<T>(s, none, total, tn, sh);
  const uint64_t rest = want - (by_mass ? mass : count);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = (int)threadIdx.x * PER + i;
    if (at < n && (by_mass ? (s < rest && s + wt[i] >= rest) : (uint64_t)at + 1 == rest)) {
      int f = 0, l = at;   // the first of its key
      while (f < l) {
        const int mid = (f + l) / 2;
        if (~(uint32_t)(list[mid] >> 32) == key[i]) l = mid;
        else f = mid + 1;
      }
      sh.cut = Cut{key[i], (uint32_t)(at - f + 1), mass + s + wt[i]};
      sh.hi = (uint32_t)at;
    }
    s += wt[i];
  }
  __syncthreads();
  *last = (int)sh.hi;
  return sh.cut;
}

// What the list holds: order (key descending, index ascending), or by index.
__device__ __forceinline__ uint64_t by_order(uint32_t key, int i) {
  return (uint64_t)~key << 32 | (uint32_t)i;
}

// A bin for every bf16 value from the maximum down to `low`, but for those
// nearest to 0, which share one (there are 254 binades): [0, P) positive ones,
// P the near ones, (P, NB) negative ones, NB what lies below.  Counts of
// values say as much as the values: masses, and where a prefix of the order
// ends, come from 4096 bins instead of V tokens.  Near is what the bins have no
// room for, at most 2^-6: normal logits have values below that in four of five
// parts of a segment, each with a weight of its own, but rarely below 2^-10.
struct KeyBins {
  static constexpr int kNear = (127 - 6) << 7, kLeast = 4096;   // bits of 2^-6 and 2^-95
  int near;            // bits of the least value that is not near
  int top, P, shift, NB;
  uint32_t pos, neg;   // what the halves of a word add to theirs, by sign

  __device__ __forceinline__ KeyBins(float m, float low) {
    const int mu = (int)(__float_as_uint(m + 0.0f) >> 16), mag = mu & 0x7fff;
    const bool below = (mu & 0x8000) != 0;
    const int lb = (int)(__float_as_uint(low) >> 16), lmag = (lb & 0x8000) ? lb & 0x7fff : 0;
    // NB = P + 1 + (n1 - near) + 1 has to stay below kBins
    const int pmag = below ? 0 : mag;
    near = max(kLeast, (pmag + lmag + 5 - kBins) / 2);
    if (lmag < near) near = max(near, pmag + 4 - kBins);
    if (pmag < near) near = max(near, lmag + 3 - kBins);
    near = below && mag >= kLeast ? kLeast : min(near, kNear);
    P = !below && mag >= near ? mag - near + 1 : 0;
    top = P + near - 1;                            // the maximum's bits, if it is not near or negative
    const int n0 = below && mag >= near ? mag : near;
    const int n1 = max(lmag, n0);                  // `low` rounds towards 0: n1 is at most it
    shift = P + 1 - n0;
    NB = n1 + shift + 1;
    pos = (uint32_t)top << 16 | (uint32_t)(top + 1);
    neg = (uint32_t)(shift - 1) << 16 | ((uint32_t)shift & 0xffffu);
  }
  // Bins of the two values of a word (at most the maximum), by halves; NB or
  // more for what lies below.  Near ones count as the largest of them, which
  // comes out as bin P: bin = top - mag, or mag + shift for negative ones.  As
  // shift < 0 (P < NB < kBins = kLeast) the lower half always carries into
  // the upper one, which pos and neg allow for.
  // (mag: their bits but for the sign, near - 1 for near ones)
  __device__ __forceinline__ uint32_t of(uint32_t w, uint32_t &mag) const {
    mag = __vmaxu2(w & 0x7fff7fffu, (uint32_t)(near - 1) * 0x10001u);
    uint32_t s;   // the halves' signs, 0 or 0xffff
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(s) : "r"(w));
    return (mag ^ ~s) + ((s & neg) | (~s & pos));
  }
  // whether one of those bits (the least of many, by halves) is a near one's
  __device__ __forceinline__ bool any_near(uint32_t mag) const {
    return (int)min(mag & 0xffffu, mag >> 16) < near;
  }
  __device__ __forceinline__ bool is_near(float x) const { return fabsf(x) < __uint_as_float((uint32_t)near << 16); }
  // value of a bin other than P
  __device__ __forceinline__ float value(int b) const {
    return __uint_as_float((uint32_t)(b < P ? top - b : 0x8000 | (b - shift)) << 16);
  }
};
__device__ __forceinline__ uint32_t word_of(const uint4 &q, int i) {
  return i == 0 ? q.x : (i == 1 ? q.y : (i == 2 ? q.z : q.w));
}
// bf16 element j of a unit, j not known at compile time
__device__ __forceinline__ float element_of(const uint4 &q, int j) {
  return __uint_as_float((word_of(q, j / 2) >> (16 * (j & 1)) & 0xffffu) << 16);
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  return (uint64_t)ld_dsmem_u32(addr + 4) << 32 | ld_dsmem_u32(addr);
}

// n to the number at addr, in any CTA's shared memory; ordered before a later
// cluster_sync().
__device__ __forceinline__ void add_dsmem_u32(uint32_t addr, uint32_t n) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(n) : "memory");
}

// One row by a cluster of C CTAs.  Each goes over its share of the segments
// for the maximum, the counts of bf16 values and the last pass; the first CTA
// joins them and decides.  Where lists are made instead, the others count and
// gather for it on order (kCount, kGather), until it meets them without one
// at the kernel's end; sorting and narrowing it does alone.  True when that
// last meeting is behind this CTA.
// (MANY: C > 1.)
//
// What holds between the stages: every count that a cut is taken from (bins,
// lists) is one of tokens with weight, x >= low, so a list has the entry that
// its bin's count promises, and a count below top_k means that top-k keeps
// all that has weight.  `cut` keeps wholly what lies above its key and the
// first `ties` of what is at it; seg holds a segment's mass above the key (of
// what min_p leaves) and tie the number of its tokens at the key.
enum Order : uint32_t { kNothing, kCount, kGather };

template <class E, int T, int kSub, bool MANY>
__device__ __forceinline__ bool sample_row(const SampleArgs &a, unsigned char *smem) {
  Shared<T> &sh = *reinterpret_cast<Shared<T> *>(smem);
  uint64_t *seg = reinterpret_cast<uint64_t *>(smem + sizeof(Shared<T>));   // mass of a segment
  constexpr int W = T / 32, PER = kCap / T;
  const uint32_t C = MANY ? cluster_nctarank() : 1, rank = MANY ? cluster_ctarank() : 0;
  const int64_t r = MANY ? cluster_id_x() : blockIdx.x;
  Row<E, kSub> row(reinterpret_cast<const E *>(a.x) + r * a.ldx, a.V, sh.edge);
  constexpr int N = 16 / (int)sizeof(E), kSegUnits = 32 * kSub;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int segs = (row.units + kSegUnits - 1) / kSegUnits;
  uint32_t *tie = reinterpret_cast<uint32_t *>(seg + segs);                 // ties of a segment
  const int share = (segs + (int)C - 1) / (int)C;
  const int s0 = min(segs, (int)rank * share), s1 = min(segs, s0 + share);   // this CTA's segments
  const float temp = a.temperature_rows ? a.temperature_rows[r] : a.temperature;
  const float inv = 1.0f / temp;
  const float u = a.u[r];
  const int top_k = a.top_k_rows ? a.top_k_rows[r] : a.top_k;
  const float top_p = a.top_p_rows ? a.top_p_rows[r] : a.top_p;
  const float min_p = a.min_p_rows ? a.min_p_rows[r] : a.min_p;
  auto answer = [&](int token, float lp) {
    a.out[r] = token;
    if (a.logprob) a.logprob[r] = lp;
  };

  row.load_edges();
  if (MANY && tid == 0) sh.order.x = kNothing;
  if (sizeof(E) == 2)
    for (int i = tid; i < kBins; i += T) sh.cnt[i] = 0;
  __syncthreads();
  // the maximum, NaN when there is one
  float mine = -INFINITY;
  row.template each<T>(s0, s1, [&](int, uint4 (&v)[kSub]) {
#pragma unroll
    for (int b = 0; b < kSub; ++b) mine = max_nan(mine, row.largest(v[b]));
  });
  float m = warp_allreduce<MaxF32, 32>(mine);
  if (lane == 0) sh.wa[w] = __float_as_uint(m);
  __syncthreads();
  m = warp_allreduce<MaxF32, 32>(lane < W ? __uint_as_float((uint32_t)sh.wa[lane]) : -INFINITY);
  if (C > 1) {
    if (tid == 0) sh.peak = m;
    sh.best[tid] = mine;
    cluster_sync();
    m = warp_allreduce<MaxF32, 32>(
        lane < (int)C ? ld_dsmem_f32(map_peer(smem_u32(&sh.peak), (uint32_t)lane)) : -INFINITY);
  }
  if (m != m || m == -INFINITY) {
    if (rank == 0 && tid == 0) answer(-1, __int_as_float(0x7fc00000));
    return false;
  }
  if (!(temp > 0.0f)) {   // the first place of the maximum
    if (rank > 0) return false;
    int at = INT_MAX;
    row.template each<T>(0, segs, [&](int un, uint4 (&v)[kSub]) {
      row.parts(un, v, [&](int ub, const uint4 &q) {
        if (row.largest(q) != m) return;
        float e[N];
        row.values(q, e);
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
          if (e[j] == m) at = min(at, row.first(ub) + j);
      });
    });
    at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();
    if (lane == 0) sh.wa[w] = (uint32_t)at;
    __syncthreads();
    if (w == 0) {
      at = __reduce_min_sync(0xffffffffu, lane < W ? (int)sh.wa[lane] : INT_MAX);
      if (lane == 0) answer(at, 0.0f);
    }
    return false;
  }
  // +inf shares all the mass: it counts as the largest number, and nothing
  // below it has weight
  const bool inf = m == INFINITY;
  m = fminf(m, kLargest);
  RowScale rs = make_scale<T>(m, temp, inv, a.base, sh.tab);
  if (inf) rs.low = INFINITY;
  __syncthreads();
  const uint64_t wmax = rs.weight(m, sh.tab);
  const uint64_t least = !(min_p > 0.0f) ? 0 : (min_p >= 1.0f ? wmax : scaled(min_p, wmax, true));
  auto target_of = [&](uint64_t total) {   // total >= 1: the maximum is kept
    const uint64_t t = u > 0.0f ? (u < 1.0f ? scaled(u, total, false) : total) : 0;
    return t < total ? t : total - 1;
  };

  // this CTA's counts to the first one's
  auto give_counts = [&]() {
    for (int i = tid; i < kBins; i += T)
      if (const uint32_t n = sh.cnt[i]) add_dsmem_u32(map_peer(smem_u32(&sh.cnt[i]), 0), n);
  };
  Cut cut{0, UINT32_MAX, 0};
  bool summed = false;   // seg and tie hold what `cut` keeps
  const bool by_k = top_k > 0 && top_k < a.V;
  const bool filtered = by_k || top_p < 1.0f;
  // bf16, unless top-k alone leaves a short list: from the values' counts.
  // sh.mass then holds the weight of each bin that is kept whole.
  bool keyed = false;
  const KeyBins kb(m, rs.low);
  if constexpr (sizeof(E) == 2) {
    keyed = !inf && kb.NB < kBins && (by_k ? top_k > kWhole / 2 : top_p < 1.0f);
    if (keyed) {
      // (sh.cnt was cleared at the start)
      uint64_t near = 0;
      uint32_t bare = 0;   // near ones without weight, which bin P must not count
      row.template each<T>(s0, s1, [&](int un, uint4 (&v)[kSub]) {
        row.parts(un, v, [&](int, const uint4 &q) {
          uint32_t least = ~0u;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            uint32_t mag;
            const uint32_t b = kb.of(word_of(q, i), mag);
            least = __vminu2(least, mag);
            if ((int)(b & 0xffffu) < kb.NB) atomicAdd(&sh.cnt[b & 0xffffu], 1u);
            if ((int)(b >> 16) < kb.NB) atomicAdd(&sh.cnt[b >> 16], 1u);
          }
          if (kb.any_near(least)) {   // few parts have one
#pragma unroll 1
            for (int j = 0; j < N; ++j) {
              const float x = element_of(q, j);
              if (!kb.is_near(x)) continue;
              if (x >= rs.low) near += rs.weight(x, sh.tab);
              else ++bare;
            }
          }
        });
      });
      near = warp_sum(near);
      bare = __reduce_add_sync(0xffffffffu, bare);
      if (lane == 0) {
        sh.wc[w] = near;
        if (bare) atomicSub(&sh.cnt[kb.P], bare);   // (modulo 2^32: in any order with the others' counts)
      }
      if (tid == 0) sh.found = sh.found2 = -1;
      __syncthreads();
      uint64_t nears = warp_sum(lane < W ? sh.wc[lane] : 0), total;
      if (C > 1) {
        if (tid == 0) sh.near = nears;
        if (rank > 0) give_counts();
        cluster_sync();   // the counts are ready
        if (rank == 0) nears = warp_sum(lane < (int)C ? ld_dsmem_u64(map_peer(smem_u32(&sh.near), lane)) : 0);
      }
      if (rank == 0) {
        // a stretch of the bins for each warp, 32 by 32 (8 and more bytes
        // apart, one to a thread, they would meet in the banks)
        constexpr int BPER = kBins / T;
        const int b0 = w * (kBins / W) + lane;
        const bool used = w * (kBins / W) <= kb.NB;
        uint32_t c = 0;
        uint64_t ms = 0;
        if (used) {
#pragma unroll 4
          for (int i = 0; i < BPER; ++i) {
            const int b = b0 + 32 * i;
            const uint32_t n = sh.cnt[b];
            const float v = kb.value(b);
            const uint64_t y = rs.weight(v, sh.tab);   // (anything where the bin has no value)
            const uint64_t x = b < kb.NB && b != kb.P && n && v >= rs.low ? y : 0;
            sh.mass[b] = x;
            c += b == kb.P || x ? n : 0;   // tokens with weight
            ms += b == kb.P ? nears : x * n;
          }
          c = __reduce_add_sync(0xffffffffu, c);
          ms = warp_sum(ms);
        }
        if (lane == 0) {
          sh.wa[w] = ms;
          sh.wb[w] = c;
        }
        __syncthreads();
        const uint64_t va = lane < W ? sh.wa[lane] : 0;
        const uint32_t vb = lane < W ? (uint32_t)sh.wb[lane] : 0;
        total = warp_sum(va);
        const uint64_t em = warp_sum(lane < w ? va : 0);
        const uint32_t ec = __reduce_add_sync(0xffffffffu, lane < w ? vb : 0);
        int cb = kb.NB;   // the bin where the prefix ends
        for (int stage = by_k ? 0 : 1; stage < (top_p < 1.0f ? 2 : 1); ++stage) {
          const bool by_mass = stage == 1;
          uint64_t want = (uint64_t)top_k;
          if (by_mass) want = top_p > 0.0f ? scaled(top_p, cb < kb.NB ? cut.mass : total, true) : 1;
          if (by_mass && by_k) __syncthreads();   // all have read what the other stage found
          int *found = by_mass ? &sh.found2 : &sh.found;
          const uint64_t before = by_mass ? em : ec, here = by_mass ? ms : c;
          if (before < want && before + here >= want) {   // in this warp's stretch
            uint64_t pc = ec, pm = em;
#pragma unroll 1
            for (int i = 0; i < BPER; ++i) {
              const int b = b0 + 32 * i;
              const uint64_t x = sh.mass[b], nc = b == kb.P || x ? sh.cnt[b] : 0, nm = b == kb.P ? nears : x * nc;
              const uint64_t ic = pc + warp_scan(nc, lane), im = pm + warp_scan(nm, lane);
              const uint32_t over = __ballot_sync(0xffffffffu, (by_mass ? im : ic) >= want);
              if (over) {
                if (lane == __ffs(over) - 1) {
                  pc = ic - nc;
                  pm = im - nm;
                  const uint64_t need = by_mass ? (x ? (want - pm + x - 1) / x : 0) : want - pc;
                  *found = b;
                  sh.cut = Cut{0, (uint32_t)need, pm + need * x};
                  sh.fcnt = (uint32_t)pc;
                  sh.fmass = pm;
                  sh.n = 0;
                }
                break;
              }
              pc = __shfl_sync(0xffffffffu, ic, 31);
              pm = __shfl_sync(0xffffffffu, im, 31);
            }
          }
          __syncthreads();
          if (*found < 0) continue;   // fewer than top_k tokens have weight
          cb = *found;
          if (cb != kb.P) {
            cut = sh.cut;
            cut.key = key_of(kb.value(cb));
            continue;
          }
          // among the near ones: those in a list
          uint64_t *list = sh.nears;
          row.template each<T>(0, segs, [&](int un, uint4 (&v)[kSub]) {
            row.parts(un, v, [&](int ub, const uint4 &q) {
#pragma unroll
              for (int j = 0; j < N; ++j) {
                const uint32_t bits = word_of(q, j / 2) >> (16 * (j & 1)) & 0xffffu;
                const float x = __uint_as_float(bits << 16);
                if ((int)(bits & 0x7fff) < kb.near && x >= rs.low) {
                  const uint32_t k = atomicAdd(&sh.n, 1u);
                  if (k < kCap) list[k] = by_order(key_of(x), row.first(ub) + j);
                }
              }
            });
          });
          __syncthreads();
          if (sh.n > kCap) {   // too many: the long way
            keyed = false;
            break;
          }
          const int n = (int)sh.n;
          const uint64_t count = sh.fcnt, mass = sh.fmass;
          sort_list<T>(list, n);
          int last;
          cut = cut_in_list<T>(list, n, count, mass, by_mass, want, sh, &last,
                               [&](float x) { return rs.weight(x, sh.tab); });
          __syncthreads();
        }
        if (!keyed)
          cut = Cut{0, UINT32_MAX, 0};
        else if (used)
          for (int i = 0; i < BPER; ++i)
            if (b0 + 32 * i >= cb || sh.mass[b0 + 32 * i] < least) sh.mass[b0 + 32 * i] = 0;
        __syncthreads();
      }
      if (C > 1) {
        if (rank == 0 && tid == 0) {
          sh.cut = cut;
          sh.keyed = keyed;
        }
        cluster_sync();   // the first CTA has decided
        if (rank > 0) {
          keyed = ld_dsmem_u32(map_peer(smem_u32(&sh.keyed), 0)) != 0;
          if (keyed) {
            cut.key = ld_dsmem_u32(map_peer(smem_u32(&sh.cut.key), 0));
            cut.ties = ld_dsmem_u32(map_peer(smem_u32(&sh.cut.ties), 0));
            for (int i = tid; i < kBins; i += T) sh.mass[i] = ld_dsmem_u64(map_peer(smem_u32(&sh.mass[i]), 0));
            __syncthreads();
          }
        }
      }
    }
  }
  // counts of the bins in segments [a, b), by mass what bracket() takes, with
  // the masses' sum in z
  auto count_pass = [&](bool by_mass, int a, int b, uint64_t &z) {
    row.template each<T>(a, b, [&](int un, uint4 (&v)[kSub]) {
      row.parts(un, v, [&](int, const uint4 &q) {
        if (!(row.largest(q) >= rs.low)) return;
        float e[N];
        row.values(q, e);
        if (by_mass) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            int bits;
            const uint64_t p = rs.product(e[j], sh.tab, bits);
            if (e[j] >= rs.low) {
              atomicAdd(&sh.cnt[bin_of(bits - kMagicBits)], (uint32_t)(p >> (31 + rs.base)));
              z += rs.shifted(p, bits);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (e[j] >= rs.low) atomicAdd(&sh.cnt[bin_of(rs.whole(e[j]))], 1u);
        }
      });
    });
  };
  // tokens of bins [lo, hi] to the list, what lies above them summed: the
  // whole of it, and by segment what min_p leaves of it
  auto gather_pass = [&](int lo, int hi, int a, int b, uint64_t &above, uint64_t &count) {
    // what is below bin `hi` for sure: t is within 1 of its whole part, and
    // the difference's own rounding is less than 1 in 2^20 of m
    const float edge = fmaxf(rs.low, hi < kBins - 1 ? m - (float)(4 * hi + 6) / rs.chi - 1e-6f * fabsf(m) : rs.low);
    row.template each<T>(a, b, [&](int un, uint4 (&v)[kSub]) {
      uint64_t s = 0;
      const int sg = un / kSegUnits;
      float best = row.largest(v[0]);
#pragma unroll
      for (int b = 1; b < kSub; ++b) best = fmaxf(best, row.largest(v[b]));
      if (__any_sync(0xffffffffu, best >= edge)) row.parts(un, v, [&](int ub, const uint4 &q) {
        if (!(row.largest(q) >= edge)) return;
        float e[N];
        row.values(q, e);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (e[j] >= edge) {
            const int at = bin_of(rs.whole(e[j]));
            if (at < lo) {
              const uint64_t x = rs.weight(e[j], sh.tab);
              above += x;
              ++count;
              if (x >= least) s += x;
            } else if (at <= hi) {
              const uint32_t k = atomicAdd(&sh.n, 1u);
              if (k < kCap) sh.list[k] = by_order(key_of(e[j]), row.first(ub) + j);
            }
          }
      });
      if (lo > 0) s = warp_sum(s);
      if (lane == 0) {
        seg[sg] = s;
        tie[sg] = 0;
      }
    });
  };
  auto send = [&](uint4 order) {   // a cluster_sync() has to follow
    if (tid > 0 && tid < (int)C) st_dsmem_u4(map_peer(smem_u32(&sh.order), (uint32_t)tid), order);
  };
  if (MANY && rank > 0 && filtered && !keyed)
    for (;;) {
      cluster_sync();   // an order, or the first CTA's end
      const uint4 order = sh.order;
      if (order.x == kNothing) return true;
      if (order.x == kCount) {
        uint64_t z = 0;
        clear_counts<T>(sh);
        count_pass(order.y != 0, s0, s1, z);
        z = block_total<T>(z, sh);
        if (tid == 0) sh.near = z;
        give_counts();
      } else {
        uint64_t above = 0, count = 0, ta, tc;
        if (tid == 0) sh.n = 0;
        __syncthreads();
        gather_pass((int)order.y, (int)order.z, s0, s1, above, count);
        block_scan<T>(above, count, ta, tc, sh);
        if (tid == 0) {
          sh.fmass = ta;
          sh.fcnt = (uint32_t)tc;
        }
      }
      __syncthreads();
      if (tid == 0) sh.order.x = kNothing;
      cluster_sync();   // done
    }
  for (int stage = keyed ? 2 : (by_k ? 0 : 1); stage < (top_p < 1.0f ? 2 : 1); ++stage) {
    const bool by_mass = stage == 1;
    // the most tokens that a list for top-k has to hold are few when the
    // threads' own maxima bound them from below
    bool maxima = !by_mass && top_k <= kWhole / 2;
    uint64_t want = (uint64_t)top_k;
    for (;;) {
      clear_counts<T>(sh);
      if (maxima) {
        for (uint32_t k = 0; k < C; ++k) {
          const float x = k == 0 ? mine : ld_dsmem_f32(map_peer(smem_u32(&sh.best[tid]), k));
          if (x >= rs.low) atomicAdd(&sh.cnt[bin_of(rs.whole(x))], 1u);
        }
      } else {
        uint64_t z = 0;
        const bool sum = by_mass && cut.ties == UINT32_MAX;
        if (MANY) {
          send(make_uint4(kCount, by_mass, 0, 0));
          cluster_sync();
        }
        count_pass(by_mass, MANY ? s0 : 0, MANY ? s1 : segs, z);
        if (MANY) cluster_sync();   // every share is counted
        if (by_mass) {
          uint64_t total = cut.mass;
          if (sum) {
            total = block_total<T>(z, sh);
            if (MANY)
              total += warp_sum(lane > 0 && lane < (int)C ? ld_dsmem_u64(map_peer(smem_u32(&sh.near), lane)) : 0);
          }
          want = top_p > 0.0f ? scaled(top_p, total, true) : 1;
        }
      }
      __syncthreads();
      if (by_mass) bracket<T>(sh, want, rs.base);
      else count_bin<T>(sh, (uint32_t)want);
      if (sh.found < 0) {
        if (!maxima) break;   // fewer than top_k tokens have weight
        maxima = false;
        __syncthreads();
        continue;
      }
      const int hi = sh.found2;
      const int lo = maxima || sh.n <= kWhole ? 0 : sh.found;
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      uint64_t above = 0, count = 0, ta, tc;
      if (MANY) {
        send(make_uint4(kGather, (uint32_t)lo, (uint32_t)hi, 0));
        cluster_sync();
      }
      gather_pass(lo, hi, MANY ? s0 : 0, MANY ? s1 : segs, above, count);
      block_scan<T>(above, count, ta, tc, sh);
      uint32_t n = sh.n;
      if (MANY) {
        cluster_sync();   // every share is gathered
        const bool peer = lane > 0 && lane < (int)C;
        const uint32_t nk = lane == 0 ? n : (peer ? ld_dsmem_u32(map_peer(smem_u32(&sh.n), lane)) : 0);
        ta += warp_sum(peer ? ld_dsmem_u64(map_peer(smem_u32(&sh.fmass), lane)) : 0);
        tc += __reduce_add_sync(0xffffffffu, peer ? ld_dsmem_u32(map_peer(smem_u32(&sh.fcnt), lane)) : 0u);
        n = __reduce_add_sync(0xffffffffu, nk);
        if (n <= kCap && w > 0 && w < (int)C) {   // a warp for each of the others
          const uint32_t at = __reduce_add_sync(0xffffffffu, lane < w ? nk : 0u), more = __shfl_sync(0xffffffffu, nk, w);
          for (uint32_t i = lane; i < more; i += 32)
            sh.list[at + i] = ld_dsmem_u64(map_peer(smem_u32(&sh.list[i]), (uint32_t)w));
        }
        if (lo > 0)
          for (int i = share + tid; i < segs; i += T) {
            seg[i] = ld_dsmem_u64(map_peer(smem_u32(&seg[i]), (uint32_t)(i / share)));
            tie[i] = 0;
          }
        __syncthreads();
      }
      if (maxima && n > kWhole) {
        maxima = false;
        __syncthreads();
        continue;
      }
      if (lo == 0 && n <= kShort) {
        // the whole prefix in a short list: the rest of the way by one warp
        if (w > 0) return false;
        constexpr int P = kShortLane;
        uint64_t wt[P], put[P], s = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) put[i] = lane * P + i < (int)n ? sh.list[lane * P + i] : ~0ull;
        sort_short(put);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int at = lane * P + i;
          wt[i] = at < (int)n && !(by_k && at >= top_k) ? rs.weight(of_key(~(uint32_t)(put[i] >> 32)), sh.tab) : 0;
          s += wt[i];
        }
        uint64_t incl = warp_scan(s, lane), e = incl - s;
        uint64_t total = __shfl_sync(0xffffffffu, incl, 31), upto = total;
        if (top_p < 1.0f) upto = by_mass ? want : (top_p > 0.0f ? scaled(top_p, total, true) : 1);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const bool kept = wt[i] > 0 && e < upto && wt[i] >= least;
          put[i] = kept ? put[i] << 32 | ~(uint32_t)(put[i] >> 32) : ~0ull;
          e += wt[i];
        }
        sort_short(put);
        s = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          wt[i] = put[i] != ~0ull ? rs.weight(of_key((uint32_t)put[i]), sh.tab) : 0;
          s += wt[i];
        }
        incl = warp_scan(s, lane);
        e = incl - s;
        total = __shfl_sync(0xffffffffu, incl, 31);
        const uint64_t target = target_of(total);
        uint64_t x;
        const int hit = entry_at(wt, e, target, x);
        if (hit >= 0) {
          uint64_t token = put[0];
#pragma unroll
          for (int i = 1; i < P; ++i) token = hit == i ? put[i] : token;
          answer((int)(token >> 32), log_share(x, total));
        }
        return false;
      }
      if (n <= kCap) {
        sort_list<T>(sh.list, (int)n);
        if (lo == 0) {
          uint64_t wt[PER], s = 0, none = 0, total, tn;
          uint32_t key[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int at = tid * PER + i;
            key[i] = at < (int)n ? ~(uint32_t)(sh.list[at] >> 32) : 0;
            wt[i] = at < (int)n ? rs.weight(of_key(key[i]), sh.tab) : 0;   // in range: x >= low
            if (by_k && at >= top_k) wt[i] = 0;
            s += wt[i];
          }
          block_scan<T>(s, none, total, tn, sh);
          // the whole prefix is in the list: the rest of the way is too
          const uint64_t upto = top_p < 1.0f ? (by_mass ? want : (top_p > 0.0f ? scaled(top_p, total, true) : 1)) : total;
          uint64_t put[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int at = tid * PER + i;
            const bool kept = wt[i] > 0 && s < upto && wt[i] >= least;
            put[i] = kept ? sh.list[at] << 32 | key[i] : ~0ull;
            s += wt[i];
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (tid * PER + i < (int)n) sh.list[tid * PER + i] = put[i];
          __syncthreads();
          sort_list<T>(sh.list, (int)n);
          s = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int at = tid * PER + i;
            put[i] = at < (int)n ? sh.list[at] : ~0ull;
            wt[i] = put[i] != ~0ull ? rs.weight(of_key((uint32_t)put[i]), sh.tab) : 0;
            s += wt[i];
          }
          block_scan<T>(s, none, total, tn, sh);
          const uint64_t target = target_of(total);
          uint64_t x;
          const int hit = entry_at(wt, s, target, x);
          if (hit >= 0) answer((int)(sh.list[tid * PER + hit] >> 32), log_share(x, total));
          return false;
        }
        int last;
        cut = cut_in_list<T>(sh.list, (int)n, tc, ta, by_mass, want, sh, &last,
                             [&](float x) { return rs.weight(x, sh.tab); });
        // the list's kept tokens to their segments
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at = tid * PER + i;
          if (at <= last) {
            const int sg = ((int)(uint32_t)sh.list[at] + row.off) / (N * kSegUnits);
            const uint32_t key = ~(uint32_t)(sh.list[at] >> 32);
            const uint64_t x = rs.weight(of_key(key), sh.tab);
            if (key == cut.key) atomicAdd(&tie[sg], 1u);
            else if (x >= least)
              atomicAdd(reinterpret_cast<unsigned long long *>(&seg[sg]), (unsigned long long)x);
          }
        }
        summed = true;
        __syncthreads();
        break;
      }
      // too many for the list (ties): narrow the bins' range of keys with
      // histograms of it until it is one key
      uint32_t klo = UINT32_MAX, khi = 0;
      if (tid == 0) {
        sh.lo = UINT32_MAX;
        sh.hi = 0;
      }
      __syncthreads();
      row.template each<T>(0, segs, [&](int un, uint4 (&v)[kSub]) {
        row.parts(un, v, [&](int, const uint4 &q) {
          float e[N];
          row.values(q, e);
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (e[j] >= rs.low) {
              const int at = bin_of(rs.whole(e[j]));
              if (at >= lo && at <= hi) {
                klo = min(klo, key_of(e[j]));
                khi = max(khi, key_of(e[j]));
              }
            }
        });
      });
      if (klo <= khi) {
        atomicMin(&sh.lo, klo);
        atomicMax(&sh.hi, khi);
      }
      __syncthreads();
      klo = sh.lo;
      khi = sh.hi;
      cut.mass = ta;
      summed = false;
      uint64_t cnt = tc;
      do {
        int shift = 0;
        while (((uint64_t)(khi - klo) >> shift) >= kBins) ++shift;
        for (int i = tid; i < kBins; i += T) {
          sh.cnt[i] = 0;
          sh.mass[i] = 0;
        }
        __syncthreads();
        row.template each<T>(0, segs, [&](int un, uint4 (&v)[kSub]) {
          row.parts(un, v, [&](int, const uint4 &q) {
            float e[N];
            row.values(q, e);
#pragma unroll
            for (int j = 0; j < N; ++j) {
              const uint32_t k = key_of(e[j]);
              if (e[j] >= rs.low && k >= klo && k <= khi) {
                const int at = (int)((khi - k) >> shift);
                atomicAdd(&sh.cnt[at], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[at]),
                          (unsigned long long)rs.weight(e[j], sh.tab));
              }
            }
          });
        });
        __syncthreads();
        constexpr int BPER = kBins / T;
        uint64_t c = 0, ms = 0, tcn, tms;
        for (int i = 0; i < BPER; ++i) {
          c += sh.cnt[tid * BPER + i];
          ms += sh.mass[tid * BPER + i];
        }
        uint64_t ec = c, em = ms;
        block_scan<T>(ec, em, tcn, tms, sh);
        const uint64_t rest = want - (by_mass ? cut.mass : cnt);
        const uint64_t before = by_mass ? em : ec, here = by_mass ? ms : c;
        if (before < rest && before + here >= rest) {
          for (int i = 0; i < BPER; ++i) {
            const uint64_t cn = ec + sh.cnt[tid * BPER + i], mn = em + sh.mass[tid * BPER + i];
            if ((by_mass ? mn : cn) >= rest) {
              sh.found = tid * BPER + i;
              sh.fcnt = (uint32_t)ec;
              sh.fmass = em;
              break;
            }
            ec = cn;
            em = mn;
          }
        }
        __syncthreads();
        cut.mass += sh.fmass;
        cnt += sh.fcnt;
        const uint32_t top = khi - ((uint32_t)sh.found << shift), span = (1u << shift) - 1;
        klo = top - klo > span ? top - span : klo;
        khi = top;
        __syncthreads();
      } while (klo < khi);
      const uint64_t wk = rs.weight(of_key(klo), sh.tab);
      // by mass: the bin's mass reaches `want`, so wk > 0
      const uint64_t need = by_mass ? (want - cut.mass + wk - 1) / wk : want - cnt;
      cut.key = klo;
      cut.ties = (uint32_t)need;
      cut.mass += need * wk;
      break;
    }
  }

  const uint64_t wcut = cut.ties == UINT32_MAX ? 0 : rs.weight(of_key(cut.key), sh.tab);
  // what min_p leaves out for sure: below m + T log(min_p), by some
  float low = rs.low;
  if (min_p > 0.0f)
    low = fmaxf(low, m - temp * (1e-4f - 1.0001f * logf(fminf(min_p, 1.0f))) - 3e-7f * fabsf(m));
  // mass above the cut and ties at it, by segment
  const bool cuts = cut.ties != UINT32_MAX;
  const bool shared = C > 1 && (keyed || !filtered);   // by all CTAs
  const int g0 = shared ? s0 : 0, g1 = shared ? s1 : segs;
  const float above = cuts ? of_key(cut.key) : -INFINITY;
  // the least element with mass of its own (NaN, which nothing reaches, where the cut is at +inf)
  const float least_x =
      above < INFINITY ? fmaxf(low, nextafterf(above, INFINITY)) : __int_as_float(0x7fc00000);
  if (keyed) {
    if constexpr (sizeof(E) == 2) {
      const uint32_t last = (uint32_t)kb.NB * 0x10001u;
      // the cut's bits in both halves, if it is not near (NaN's, which none has, else)
      const bool near_tie = cuts && kb.is_near(above);
      const uint32_t tied = cuts && !near_tie ? (__float_as_uint(above) >> 16) * 0x10001u : 0x7fff7fffu;
      row.template each<T>(g0, g1, [&](int un, uint4 (&v)[kSub]) {
        uint64_t s = 0;
        uint32_t n = 0;
        row.parts(un, v, [&](int, const uint4 &q) {
          const float top = row.largest(q);
          if (!(top >= low && top >= above)) return;
          uint32_t near_by = ~0u, ties = ~0u;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            uint32_t mag;
            const uint32_t b = __vminu2(kb.of(word_of(q, i), mag), last);
            near_by = __vminu2(near_by, mag);
            ties = __vminu2(ties, word_of(q, i) ^ tied);
            s += sh.mass[b & 0xffffu] + sh.mass[b >> 16];
          }
          if (!(ties & 0xffffu) || !(ties >> 16)) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
              const uint32_t x = word_of(q, i) ^ tied;
              n += !(x & 0xffffu);
              n += !(x >> 16);
            }
          }
          if (kb.any_near(near_by)) {   // few parts have one
#pragma unroll 1
            for (int j = 0; j < N; ++j) {
              const float x = element_of(q, j);
              if (!kb.is_near(x)) continue;
              n += near_tie && x == above;
              if (x >= least_x) {
                const uint64_t y = rs.weight(x, sh.tab);
                if (y >= least) s += y;
              }
            }
          }
        });
        s = warp_sum(s);
        n = cuts ? __reduce_add_sync(0xffffffffu, n) : 0;
        if (lane == 0) {
          seg[un / kSegUnits] = s;
          tie[un / kSegUnits] = n;
        }
      });
    }
  } else if (!summed)
    row.template each<T>(g0, g1, [&](int un, uint4 (&v)[kSub]) {
      uint64_t s = 0;
      uint32_t n = 0;
      // eight elements at a time, whichever the type, to overlap their chains
      constexpr int Q = 8 / N < kSub ? 8 / N : kSub, M = Q * N;
#pragma unroll 1
      for (int b = 0; b < kSub; b += Q) {
        float e[M], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < Q; ++k) {
          float q[N];
          row.values(v[k], q);
#pragma unroll
          for (int j = 0; j < N; ++j) e[k * N + j] = q[j];
          top = fmaxf(top, row.largest(v[k]));
        }
#pragma unroll
        for (int k = Q; k < kSub; ++k) v[k - Q] = v[k];
        if (!(top >= low && top >= above)) continue;
        uint64_t x[M];   // (of what is below `low`: anything)
#pragma unroll
        for (int j = 0; j < M; ++j) x[j] = rs.weight(e[j], sh.tab);
        if (least > 0) {
#pragma unroll
          for (int j = 0; j < M; ++j)
            if (x[j] < least) x[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < M; ++j)
          if (e[j] >= least_x) s += x[j];
        if (cuts) {
#pragma unroll
          for (int j = 0; j < M; ++j) n += e[j] == above;
        }
      }
      s = warp_sum(s);
      n = cuts ? __reduce_add_sync(0xffffffffu, n) : 0;
      if (lane == 0) {
        seg[un / kSegUnits] = s;
        tie[un / kSegUnits] = n;
      }
    });
  if (shared) {
    cluster_sync();   // every share is summed
    if (rank > 0) return false;
    for (int i = share + tid; i < segs; i += T) {
      const uint32_t k = (uint32_t)(i / share);
      seg[i] = ld_dsmem_u64(map_peer(smem_u32(&seg[i]), k));
      tie[i] = ld_dsmem_u32(map_peer(smem_u32(&tie[i]), k));
    }
  }
  __syncthreads();
  // one warp: ties to masses, the total, and the segment that holds the draw
  if (w == 0) {
    uint64_t before = 0, total = 0;
    for (int b = 0; b < segs; b += 32) {
      const int i = b + lane;
      uint64_t v = i < segs ? seg[i] : 0;
      if (cut.ties != UINT32_MAX) {
        const uint64_t n = i < segs ? tie[i] : 0;
        const uint64_t incl = warp_scan(n, lane);
        const uint64_t first = before + incl - n;
        const uint64_t kept = wcut < least || first >= cut.ties ? 0 : min(n, (uint64_t)cut.ties - first);
        v += kept * wcut;
        if (i < segs) {
          seg[i] = v;
          tie[i] = (uint32_t)kept;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
      total += v;
    }
    __syncwarp();
    total = warp_sum(total);
    const uint64_t target = target_of(total);
    uint64_t run = 0;
    int hit = -1;
    for (int b = 0; b < segs && hit < 0; b += 32) {
      const uint64_t v = b + lane < segs ? seg[b + lane] : 0;
      const uint64_t incl = run + warp_scan(v, lane);
      const uint32_t over = __ballot_sync(0xffffffffu, incl > target);
      if (over) {
        const int l = __ffs(over) - 1;
        hit = b + l;
        run = __shfl_sync(0xffffffffu, incl - v, l);
      } else {
        run = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      sh.found = hit;
      sh.wa[0] = run;
      sh.wa[1] = total;
      sh.wa[2] = target;
    }
  }
  __syncthreads();
  // the segment's elements, 32 units to a warp
  if (w < kSub) {
    const int hit = sh.found, un = hit * kSegUnits + 32 * w + lane;
    if (hit < 0) {   // no mass: the maximum has some, so it cannot be; nothing is read there
      if (tid == 0) answer(-1, __int_as_float(0x7fc00000));
      return false;
    }
    const uint64_t total = sh.wa[1], target = sh.wa[2];
    const uint32_t kept = tie[hit];
    float e[N];
    row.values(row.raw(un), e);
    uint32_t n = 0;
    uint64_t s = 0, x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = rs.weight(e[j], sh.tab);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!(e[j] >= least_x && x[j] >= least)) x[j] = 0;
      n += cuts && e[j] == above;
      s += x[j];
    }
    const uint32_t tied = (uint32_t)warp_scan(n, lane);
    // ties before this warp's, then its masses
    if (lane == 31) sh.wb[w] = tied;
    named_sync(1, 32 * kSub);
    uint32_t place = tied - n;
    for (int k = 0; k < w; ++k) place += (uint32_t)sh.wb[k];
    s += (place >= kept ? 0 : min(n, kept - place)) * wcut;
    const uint64_t incl = warp_scan(s, lane);
    if (lane == 31) sh.wb[kSub + w] = incl;
    named_sync(1, 32 * kSub);
    uint64_t acc = sh.wa[0] + incl - s;
    for (int k = 0; k < w; ++k) acc += sh.wb[kSub + k];
    if (acc <= target && target < acc + s) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (cuts && e[j] == above && place++ < kept) x[j] = wcut;
      uint64_t share;
      const int hit = entry_at(x, acc, target, share);
      answer(row.first(un) + hit, log_share(share, total));
    }
  }
  return false;
}

template <class E, int T, int SUB, bool MANY>
__global__ void __launch_bounds__(T, 1024 / T)
k_sample(SampleArgs a) {
  pdl_begin();
  extern __shared__ __align__(16) unsigned char smem[];
  const bool met = sample_row<E, T, SUB, MANY>(a, smem);
  if (MANY && !met) cluster_sync();   // no CTA leaves while a peer may read it
}

}  // namespace

int sample_base(int64_t V) {
  int lg = 0;
  while (((int64_t)1 << lg) < V) ++lg;
  return lg;   // K = 61 - lg: V weights of at most 2^K stay below 2^62
}

namespace {
template <class E, int SUB>
int64_t segments(int64_t V) {
  constexpr int n = 16 / (int)sizeof(E);
  return ((V + 2 * n) / n + 32 * SUB) / (32 * SUB);
}

template <class E, int T, int SUB, bool MANY>
int sample_launch(const SampleArgs &a, int64_t rows, int C, cudaStream_t s, const DevInfo &d) {
  const size_t smem = sizeof(Shared<T>) + (size_t)segments<E, SUB>(a.V) * 12;
  static std::atomic<uint64_t> allowed;
  const cudaError_t e = allow_kernel(k_sample<E, T, SUB, MANY>, kSampleSmem, false, d.device, allowed);
  if (e != cudaSuccess) return cuda_status(e);
  if (smem > kSampleSmem) return RR_ERR_INVALID;
  while (C > 1 && occupancy_clusters((const void *)k_sample<E, T, SUB, MANY>, T, smem, C, d.device) < 1) C /= 2;
  if (C == 1 && MANY) return sample_launch<E, T, SUB, false>(a, rows, 1, s, d);
  if (rows * C > INT_MAX) return RR_ERR_INVALID;
  if (log_enabled())
    std::fprintf(stderr, "[rr] sample rows=%lld V=%d base=%d C=%d threads=%d part=%d smem=%zu\n",
                 (long long)rows, a.V, a.base, C, T, SUB, smem);
  return cuda_status(launch_kernel(k_sample<E, T, SUB, MANY>, dim3((unsigned)(rows * C)), dim3(T), smem, s,
                                   MANY ? C : 0, a));
}

// CTAs of 512 threads, two to an SM, where there are rows for both or a row
// has no work for more; of 1024 where a row has an SM for itself.  us, 1024
// against 512 threads (bf16, top-p; mixed settings; fp32 without filters):
//   V 131072, 100 rows: 39, 47; 36, 43; 29, 34     V 32003: 18, 19; 22, 22; 11, 12
//             153 rows: 62, 65; 37, 44; 63, 59              30, 26; 24, 27; 20, 17
//             512 rows: 147, 135; 103, 96; 133, 128         61, 48; 62, 46; 48, 38
// Rows of up to 2048 units go in segments of half the size, for more warps:
//   V 8000, 2048 rows: 187, 106; 223, 124; 86, 52 and 95; 103; 54 in those.
template <class E>
int sample_plan(const SampleArgs &a, int64_t rows, cudaStream_t s, const DevInfo &d) {
  constexpr int64_t kShortRow = 32 << 10;
  if (a.V * (int64_t)sizeof(E) <= kShortRow) return sample_launch<E, 512, 2, false>(a, rows, 1, s, d);
  if (rows > d.sm_count) return sample_launch<E, 512, 4, false>(a, rows, 1, s, d);
  // a CTA a row, or a cluster while there are not rows for every SM and each
  // of its warps has a segment (64 rows of 100003 fp32 without filters: 23 us
  // with a CTA each, 18.3 with two)
  const int64_t segs = segments<E, 4>(a.V);
  const int most = d.cluster_launch ? (cluster_cap() < 8 ? cluster_cap() : 8) : 1;
  int C = 1;
  while (C * 2 <= most && rows * C * 2 <= d.sm_count && segs >= (int64_t)C * 2 * 32) C *= 2;
  return C > 1 ? sample_launch<E, 1024, 4, true>(a, rows, C, s, d)
               : sample_launch<E, 1024, 4, false>(a, rows, 1, s, d);
}
}  // namespace

int launch_sample(SampleArgs a, int dtype, int64_t rows, cudaStream_t s, const DevInfo &d) {
  a.base = sample_base(a.V);
  return dtype == RR_BF16 ? sample_plan<unsigned short>(a, rows, s, d) : sample_plan<float>(a, rows, s, d);
}

}  // namespace rr
