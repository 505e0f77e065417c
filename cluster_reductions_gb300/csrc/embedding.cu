// embedding.cu -- the embedding lookup with scaling, and its gradient by
// sorted tokens.
//
//   lookup    out[i, :] = round(scale * W[tok_i, :])
//   gradient  dW[v, :]  = (dW[v, :] +) scale * sum over {i : tok_i = v} of dy[i, :]
//
// A token outside [0, V) is padding: a row of zeros, and no part of the
// gradient.  Both move bytes and compute next to nothing: DRAM bounds them.
//
// The gradient adds each table row's terms in increasing i, in fp32 (a long
// run in pieces, the pieces joined in a fixed order), with no float atomics, so
// its bits do not depend on scheduling.  Three launches:
//
//   k_token_sort   the first cluster sorts (token, i) stably by token: a
//                  radix sort from the lowest digit, up to 9 bits a pass, the
//                  digit counts of its CTAs exchanged through distributed
//                  shared memory.  The other clusters meanwhile write zeros
//                  to dW (dense form), which takes longer than the sort.
//   k_embed_grad   a CTA per (chunk of 16 to 256 sorted entries, column tile)
//                  adds the rows of each run of equal tokens in registers.  A
//                  run no longer than a chunk goes to dW, whole, from the
//                  chunk it starts in; a longer one is cut at the chunks'
//                  borders, its pieces go to the workspace in fp32.
//   k_embed_join   adds the pieces of each long run in order.
#include <climits>
#include <cstdio>

#include "rr.h"
#include "rr_internal.h"
#include "token.cuh"

namespace rr {
namespace {

// ---- lookup ---------------------------------------------------------------
constexpr int kEmbThreads = 256;
constexpr int kEmbUnroll = 4;   // accesses a lane has in flight

// A segment of 2^lg lanes per piece of a row: kEmbUnroll << lg accesses of
// VB bytes.  pieces = ceil(accesses per row / (kEmbUnroll << lg)).
template <class E, int VB>
__global__ void __launch_bounds__(kEmbThreads)
k_embed(const E *__restrict__ w, const void *__restrict__ tok, bool wide, int64_t items,
        int pieces, int acc_per_row, int64_t V, int64_t D, float scale, E *__restrict__ out,
        int lg) {
  pdl_begin();
  using A = typename Access<VB>::type;
  constexpr int N = VB / (int)sizeof(E);
  const int lane = threadIdx.x & ((1 << lg) - 1);
  const int64_t item = (int64_t)blockIdx.x * (kEmbThreads >> lg) + (threadIdx.x >> lg);
  if (item >= items) return;
  const int64_t row = item / pieces;
  const int a0 = (int)(item - row * pieces) * (kEmbUnroll << lg) + lane;
  const int64_t t = load_token(tok, wide, row, V);
  A *dst = reinterpret_cast<A *>(out + row * D);
  if (t < 0) {
#pragma unroll
    for (int k = 0; k < kEmbUnroll; ++k)
      if (a0 + (k << lg) < acc_per_row) dst[a0 + (k << lg)] = A{};
    return;
  }
  const A *src = reinterpret_cast<const A *>(w + t * D);
  A v[kEmbUnroll];
#pragma unroll
  for (int k = 0; k < kEmbUnroll; ++k)
    if (a0 + (k << lg) < acc_per_row) v[k] = __ldg(src + a0 + (k << lg));
#pragma unroll
  for (int k = 0; k < kEmbUnroll; ++k)
    if (a0 + (k << lg) < acc_per_row) {
      float e[N];
      split<E, VB>(v[k], e);
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] *= scale;
      __stcs(dst + a0 + (k << lg), join<E, N>(e));
    }
}

template <class E, int VB>
int embed_launch(const void *w, int64_t V, int64_t D, const void *tok, bool wide, int64_t n,
                 float scale, void *out, cudaStream_t s) {
  const int64_t acc = D * (int64_t)sizeof(E) / VB;
  int lg = 0;
  while (lg < 5 && ((int64_t)kEmbUnroll << lg) < acc) ++lg;
  const int64_t pieces = (acc + ((int64_t)kEmbUnroll << lg) - 1) / ((int64_t)kEmbUnroll << lg);
  const int64_t items = n * pieces;
  const int64_t per = kEmbThreads >> lg;
  const int64_t grid = (items + per - 1) / per;
  if (grid > INT_MAX) return RR_ERR_INVALID;
  if (log_enabled())
    std::fprintf(stderr, "[rr] embedding n=%lld D=%lld access=%d lanes=%d grid=%lld\n",
                 (long long)n, (long long)D, VB, 1 << lg, (long long)grid);
  return cuda_status(launch_kernel(k_embed<E, VB>, dim3((unsigned)grid), dim3(kEmbThreads), 0, s, 0,
                                   (const E *)w, tok, wide, items, (int)pieces, (int)acc, V, D,
                                   scale, (E *)out, lg));
}

// ---- gradient: sort --------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;                 // widest digit
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortEach = 4096;              // entries of a CTA beside a fill
constexpr int kSortChip = 8192;              // most entries it keeps in shared memory
// the warps' counts, and two lists of keys and positions
constexpr size_t sort_smem(int bits, int per) { return ((size_t)kSortWarps << bits) * 4 + (size_t)per * 16; }
constexpr uint32_t kZeros = kSortWarps * 2 * 4 * 128;   // bytes of it that a fill copies from: 32 KiB

struct SortArgs {
  const void *tok;
  bool wide;
  int n;           // entries
  int64_t V;       // key of a padding token: behind every row of the table
  int bits, passes;
  int per;         // entries of a CTA, a multiple of 1024
  int *key[2], *pos[2];  // the sorted list in [0] (CHIP); else pass p writes p & 1
  int *runs;             // the list of long runs: their count first
};

// Zeros over [p, p + bytes), by CTA `me` of `of`; p 2-byte aligned.  Bulk
// copies of `zeros` (kZeros bytes of shared memory, cleared here) by one
// thread: the copy engine keeps the writes coming without the CTA's warps.
__device__ __forceinline__ void fill_zero(unsigned char *p, size_t bytes, size_t me, size_t of,
                                          void *zeros) {
  const int tid = threadIdx.x;
  for (int i = tid; i < (int)(kZeros / 16); i += kSortThreads)
    reinterpret_cast<uint4 *>(zeros)[i] = make_uint4(0, 0, 0, 0);
  const size_t head = min(bytes, (size_t)(-(uintptr_t)p & 15));
  const size_t body = (bytes - head) & ~(size_t)15, tail = bytes - head - body;
  if (me == 0 && tid < (int)(head / 2)) reinterpret_cast<unsigned short *>(p)[tid] = 0;
  if (me == 0 && tid < (int)(tail / 2)) reinterpret_cast<unsigned short *>(p + head + body)[tid] = 0;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    for (size_t o = (size_t)me * kZeros; o < body; o += (size_t)of * kZeros) {
      const uint32_t len = (uint32_t)min((size_t)kZeros, body - o);
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p + head + o),
                   "r"(smem_u32(zeros)), "r"(len)
                   : "memory");
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

__device__ __forceinline__ int token_key(const SortArgs &a, int i) {
  const int64_t t = load_token(a.tok, a.wide, i, a.V);
  return (int)(t < 0 ? a.V : t);
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Cluster 0 sorts; clusters 1.. fill.  CTA r holds the list's places [r per,
// (r + 1) per), and warp w of it a contiguous share of those: (r, w, order
// inside the warp) is the list's order, and every step below keeps it, so the
// sort is stable.
//
// CHIP: between the passes the list is in the CTAs' shared memory, written by
// its new places' peers; global memory, which the fill keeps busy, sees the
// tokens once and the sorted list once (the whole gradient: 4099 tokens of
// 32003 x 1029 fp32 33.2 us against 38.6, 16384 of 131072 x 4096 bf16 204
// against 209).  Else, for lists too long for that, through global memory.
template <bool CHIP>
__global__ void __launch_bounds__(kSortThreads)
k_token_sort(SortArgs a, unsigned char *fill, size_t fill_bytes) {
  pdl_begin();
  extern __shared__ __align__(128) uint32_t hist[];   // [warp][bin]
  __shared__ uint32_t total[kSortBins];           // this CTA's count of each digit
  __shared__ uint32_t start[kSortBins];           // where its entries of a digit go
  __shared__ uint32_t wsum[kSortWarps];
  const uint32_t C = cluster_nctarank(), r = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (cluster_id_x() > 0) {
    fill_zero(fill, fill_bytes, blockIdx.x - C, gridDim.x - C, hist);
    return;
  }
  if (a.n > 0 && r == 0 && tid == 0) *a.runs = 0;
  const int per_warp = a.per / kSortWarps;
  const int64_t first = (int64_t)((int)r * kSortWarps + w) * per_warp;
  const int w0 = first < a.n ? (int)first : a.n;
  const int w1 = a.n - w0 < per_warp ? a.n : w0 + per_warp;
  const int bins = 1 << a.bits;
  const int busy = a.n > 0 ? min(kSortWarps, (a.n + per_warp - 1) / per_warp) : 0;   // warps with entries
  uint32_t *mine = hist + w * bins;
  // CHIP: keys and positions of the CTA's places, two of each
  uint32_t *const list = hist + kSortWarps * bins;
  const int base0 = (int)r * a.per;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    uint32_t *const ck = list + (size_t)(pass & 1) * 2 * a.per, *const cp = ck + a.per;
    auto key_at = [&](int i) {
      if (CHIP) return (int)ck[i - base0];
      return pass > 0 ? __ldcg(a.key[(pass - 1) & 1] + i) : token_key(a, i);
    };
    for (int i = tid; i < busy * bins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    for (int b = w0; b < w1; b += 32) {
      const int i = b + lane;
      int d = -1;
      if (i < w1) {
        int key;
        if (CHIP && pass == 0) {
          key = token_key(a, i);
          ck[i - base0] = (uint32_t)key;
        } else {
          key = key_at(i);
        }
        d = (key >> shift) & (bins - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (d >= 0 && lane == __ffs(peers) - 1) mine[d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    if (tid < bins) {   // counts -> offsets of each warp inside the CTA's share of the digit
      uint32_t acc = 0;
#pragma unroll 8
      for (int k = 0; k < busy; ++k) {
        const uint32_t c = hist[k * bins + tid];
        hist[k * bins + tid] = acc;
        acc += c;
      }
      total[tid] = acc;
    }
    cluster_sync();
    // entries of smaller digits, and of this digit in earlier CTAs
    uint32_t all = 0, before = 0;
    if (tid < bins) {
#pragma unroll 16
      for (uint32_t k = 0; k < 16; ++k) {
        const uint32_t c = k < C ? ld_dsmem_u32(map_peer(smem_u32(total + tid), k)) : 0;
        if (k < r) before += c;
        all += c;
      }
    }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    uint32_t below = wsum[lane] & (lane < w ? ~0u : 0u);   // of the warps before this one
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
    if (tid < bins) start[tid] = incl - all + before + below;
    __syncthreads();
    const bool last = pass == a.passes - 1;
    int *const ok = a.key[CHIP ? 0 : pass & 1], *const op = a.pos[CHIP ? 0 : pass & 1];
    const uint32_t peer_list = smem_u32(list + (size_t)((pass + 1) & 1) * 2 * a.per);
    for (int b = w0; b < w1; b += 32) {
      const int i = b + lane;
      int key = 0, pos = i, d = -1;
      if (i < w1) {
        key = key_at(i);
        if (pass > 0) pos = CHIP ? (int)cp[i - base0] : __ldcg(a.pos[(pass - 1) & 1] + i);
        d = (key >> shift) & (bins - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      uint32_t at = 0;
      if (d >= 0) at = start[d] + mine[d] + __popc(peers & ((1u << lane) - 1));
      __syncwarp();
      if (d >= 0) {
        if (lane == __ffs(peers) - 1) mine[d] += __popc(peers);
        if (!CHIP || last) {
          ok[at] = key;
          op[at] = pos;
        } else {
          const uint32_t rank = at / (uint32_t)a.per, o = at - rank * (uint32_t)a.per;
          const uint32_t dst = map_peer(peer_list, rank);
          st_dsmem_u32(dst + 4 * o, (uint32_t)key);
          st_dsmem_u32(dst + 4 * ((uint32_t)a.per + o), (uint32_t)pos);
        }
      }
      __syncwarp();
    }
    // the next pass reads what its peers wrote; nobody reads `total` any more
    cluster_sync();
  }
}

// ---- gradient: sums ---------------------------------------------------------
constexpr int kGradThreads = 128;
constexpr int kGradBatch = 8;     // rows a thread has in flight
constexpr int kGradMinChunk = 16;
constexpr int kGradMaxChunk = 256;

// N elements of type G at p, aligned to min(16, N * sizeof(G)) bytes.
template <class G, int N>
__device__ __forceinline__ void load_n(const G *p, float (&e)[N]) {
  constexpr int VB = N * (int)sizeof(G) > 16 ? 16 : N * (int)sizeof(G);
  constexpr int M = VB / (int)sizeof(G);
#pragma unroll
  for (int k = 0; k < N / M; ++k) {
    float q[M];
    split<G, VB>(*reinterpret_cast<const typename Access<VB>::type *>(p + k * M), q);
#pragma unroll
    for (int j = 0; j < M; ++j) e[k * M + j] = q[j];
  }
}
template <class G, int N>
__device__ __forceinline__ void store_n(G *p, const float (&e)[N]) {
  constexpr int VB = N * (int)sizeof(G) > 16 ? 16 : N * (int)sizeof(G);
  constexpr int M = VB / (int)sizeof(G);
#pragma unroll
  for (int k = 0; k < N / M; ++k) {
    float q[M];
#pragma unroll
    for (int j = 0; j < M; ++j) q[j] = e[k * M + j];
    *reinterpret_cast<typename Access<VB>::type *>(p + k * M) = join<G, M>(q);
  }
}

// dW[v, c..c+N) = (dW +) scale * sum: one fp32 product (and sum), one rounding.
template <class G, int N>
__device__ __forceinline__ void write_grad(G *p, float (&acc)[N], float scale, bool add) {
  float o[N];
  if (add) {
    load_n<G, N>(p, o);
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = fmaf(acc[j], scale, o[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = acc[j] * scale;
  }
  store_n<G, N>(p, o);
}

// Pieces of long runs: piece[chunk][0] of the run that enters the chunk
// from the left, piece[chunk][1] of the one that starts in it and leaves it.
template <class E, class G, int N>
__global__ void __launch_bounds__(kGradThreads)
k_embed_grad(const E *__restrict__ dy, const int *__restrict__ key, const int *__restrict__ pos,
             int n, int64_t V, int64_t D, int L, int tiles, float scale, bool add,
             G *__restrict__ dw, float *__restrict__ piece, int *__restrict__ runs) {
  pdl_begin();
  __shared__ int skey[2 * kGradMaxChunk], spos[2 * kGradMaxChunk];
  __shared__ int span[3];   // of the entries beside the chunk that belong to its first / last run
  const int chunk = blockIdx.x / tiles, tile = blockIdx.x - chunk * tiles;
  const int j0 = chunk * L, cnt = min(L, n - j0), more = min(2 * L, n - j0);
  if (key[j0] >= V) return;   // only padding from here on
  for (int i = threadIdx.x; i < more; i += kGradThreads) {
    skey[i] = key[j0 + i];
    spos[i] = pos[j0 + i];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    // equal neighbours before the chunk and after it, up to L of each, and
    // the first run's entries inside it
    const int lane = threadIdx.x, t0 = skey[0], t1 = skey[cnt - 1];
    int back = 0, in = 0, ahead = 0;
    for (int o = 0; o < L; o += 32) {
      const int i = j0 - 1 - o - lane;
      const uint32_t m = __ballot_sync(0xffffffffu, i >= 0 && key[i >= 0 ? i : 0] == t0);
      back += __ffs(~m) ? __ffs(~m) - 1 : 32;
      if (~m) break;
    }
    for (int o = 0; o < cnt; o += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, o + lane < cnt && skey[o + lane] == t0);
      in += __ffs(~m) ? __ffs(~m) - 1 : 32;
      if (~m) break;
    }
    for (int o = cnt; o < more; o += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, o + lane < more && skey[o + lane] == t1);
      ahead += __ffs(~m) ? __ffs(~m) - 1 : 32;
      if (~m) break;
    }
    if (lane == 0) {
      span[0] = back;
      span[1] = in;
      span[2] = ahead;
    }
  }
  __syncthreads();
  const int back = span[0], in = span[1], ahead = span[2];
  const bool one = in == cnt;                       // a single run fills the chunk
  // runs of more than L entries are cut at the chunks' borders and joined;
  // of the others, all entries go to the chunk they start in
  const bool long0 = back > 0 && back + in + (one ? ahead : 0) > L;
  int tail = 0;                                     // the last run's entries inside the chunk
  if (ahead > 0 && !(one && back > 0)) {
    const int t1 = skey[cnt - 1];
    tail = 1;
    while (tail < cnt && skey[cnt - 1 - tail] == t1) ++tail;
  }
  const bool long1 = tail > 0 && tail + ahead > L;  // it starts here
  const int begin = back > 0 && !long0 ? in : 0;
  const int end = tail > 0 && !long1 ? cnt + ahead : cnt;
  if (long1 && tile == 0 && threadIdx.x == 0 && skey[cnt - 1] < V) runs[1 + atomicAdd(runs, 1)] = chunk;
  const int64_t c = ((int64_t)tile * kGradThreads + threadIdx.x) * N;
  if (c >= D) return;
  float acc[N];
  int cur = -1;
  bool entered = false;
  for (int b = begin; b < end; b += kGradBatch) {
    typename Access<N * (int)sizeof(E)>::type v[kGradBatch];
#pragma unroll
    for (int k = 0; k < kGradBatch; ++k)
      if (b + k < end && skey[b + k] < V)
        v[k] = ld_once<N * (int)sizeof(E)>(dy + (int64_t)spos[b + k] * D + c);
#pragma unroll
    for (int k = 0; k < kGradBatch; ++k) {
      if (b + k >= end) break;
      const int t = skey[b + k];
      if (t != cur) {
        if (cur >= 0) {
          if (entered) store_n<float, N>(piece + (int64_t)chunk * 2 * D + c, acc);
          else write_grad<G, N>(dw + (int64_t)cur * D + c, acc, scale, add);
        }
        entered = b + k == 0 && long0;
        cur = t < V ? t : -1;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
      }
      if (cur >= 0) {
        float e[N];
        split<E, N * (int)sizeof(E)>(v[k], e);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += e[j];
      }
    }
  }
  if (cur >= 0) {
    if (entered) store_n<float, N>(piece + (int64_t)chunk * 2 * D + c, acc);
    else if (long1) store_n<float, N>(piece + ((int64_t)chunk * 2 + 1) * D + c, acc);
    else write_grad<G, N>(dw + (int64_t)cur * D + c, acc, scale, add);
  }
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// A CTA per (run, 32 N columns): its warps take equal shares of the run's
// pieces, in order, and the shares are added in order.
template <class G, int N>
__global__ void __launch_bounds__(kJoinThreads)
k_embed_join(const int *__restrict__ key, int n, int64_t D, int L, int tiles, float scale, bool add,
             G *__restrict__ dw, const float *__restrict__ piece, const int *__restrict__ runs) {
  pdl_begin();
  __shared__ float part[kJoinWarps][32 * N];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t items = (int64_t)*runs * tiles;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int chunk = runs[1 + item / tiles];
    const int64_t c = ((item % tiles) * 32 + lane) * N;
    const int t = key[(chunk + 1) * L];
    // the run's last chunk: the first that does not start with it, less one
    int last = chunk + 1;
    for (;;) {
      const int64_t at = (int64_t)(last + 1 + lane) * L;
      const uint32_t ends = __ballot_sync(0xffffffffu, at >= n || key[at] != t);
      if (ends) {
        last += __ffs(ends) - 1;
        break;
      }
      last += 32;
    }
    // pieces chunk (its second place), chunk + 1 .. last (their first)
    const int count = last - chunk + 1, share = (count + kJoinWarps - 1) / kJoinWarps;
    const int k0 = min(w * share, count), k1 = min(k0 + share, count);
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    if (c < D) {
#pragma unroll 8
      for (int k = k0; k < k1; ++k) {
        float e[N];
        load_n<float, N>(piece + ((int64_t)(chunk + k) * 2 + (k == 0)) * D + c, e);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += e[j];
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) part[w][j * 32 + lane] = acc[j];
    __syncthreads();
    if (w == 0 && c < D) {
      for (int k = 1; k < kJoinWarps; ++k) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += part[k][j * 32 + lane];
      }
      write_grad<G, N>(dw + (int64_t)t * D + c, acc, scale, add);
    }
    __syncthreads();
  }
}

// Entries of a chunk: 16, for a short way through a short list (a CTA's
// rows come one batch of 8 after another), doubled while there would be over
// 4096 CTAs (the longer the list, the fewer pieces of a run to join).
int grad_chunk(int64_t n, int64_t D) {
  int L = kGradMinChunk;
  while (L < kGradMaxChunk && ((n + L - 1) / L) * ((D + 511) / 512) > 4096) L *= 2;
  return L;
}

int64_t grad_tiles(int64_t D, int width) {
  return (D + (int64_t)kGradThreads * width - 1) / ((int64_t)kGradThreads * width);
}

// Widest column group whose accesses of dy and dW are aligned (16 bytes at
// most each; fp32 dW under bf16 dy takes two).
int grad_column(const void *dy, int dtype, const void *dw, int dw_dtype, int64_t D) {
  const int64_t es = dtype == RR_BF16 ? 2 : 4, gs = dw_dtype == RR_BF16 ? 2 : 4;
  int width = dtype == RR_BF16 ? 8 : 4;
  auto fits = [&](int64_t w) {
    const int64_t gb = w * gs < 16 ? w * gs : 16;
    const int64_t pb = w * 4 < 16 ? w * 4 : 16;   // the fp32 pieces
    return D % w == 0 && (uintptr_t)dy % (w * es) == 0 && (D * es) % (w * es) == 0 &&
           (uintptr_t)dw % gb == 0 && (D * gs) % gb == 0 && (D * 4) % pb == 0;
  };
  while (width > 1 && !fits(width)) width /= 2;
  return width;
}

// The list of long runs: a count and a chunk each.
size_t runs_bytes(int64_t chunks) { return ((size_t)(chunks + 1) * 4 + 255) & ~(size_t)255; }

size_t list_bytes(int64_t n) { return ((size_t)n * 4 + 255) & ~(size_t)255; }

template <class E, class G, int N>
int grad_launch(const void *dy, const int *key, const int *pos, int n, int64_t V, int64_t D,
                float scale, bool add, void *dw, float *piece, int *runs, cudaStream_t s,
                const DevInfo &d) {
  const int L = grad_chunk(n, D);
  const int64_t tiles = grad_tiles(D, N);
  const int64_t chunks = ((int64_t)n + L - 1) / L;   // (embedding_grad_fits: tiles x chunks fit a grid)
  const dim3 grid((unsigned)(tiles * chunks)), block(kGradThreads);
  if (log_enabled())
    std::fprintf(stderr, "[rr] embedding gradient n=%d D=%lld chunk=%d width=%d grid=%u\n", n,
                 (long long)D, L, N, grid.x);
  cudaError_t e = launch_kernel(k_embed_grad<E, G, N>, grid, block, 0, s, 0, (const E *)dy, key, pos,
                                n, V, D, L, (int)tiles, scale, add, (G *)dw, piece, runs);
  if (e != cudaSuccess || chunks < 2) return cuda_status(e);
  // at most a run for every chunk but the last; how many there are is on the GPU
  const int64_t jt = (D + 32 * N - 1) / (32 * N), most = (chunks - 1) * jt, fit = 4 * (int64_t)d.sm_count;
  return cuda_status(launch_kernel(k_embed_join<G, N>, dim3((unsigned)(most < fit ? most : fit)),
                                   dim3(kJoinThreads), 0, s, 0, key, n, D, L, (int)jt, scale, add, (G *)dw,
                                   (const float *)piece, (const int *)runs));
}

template <class E, class G>
int grad_width(int width, const void *dy, const int *key, const int *pos, int n, int64_t V,
               int64_t D, float scale, bool add, void *dw, float *piece, int *runs, cudaStream_t s,
               const DevInfo &d) {
  switch (width) {
    case 8:
      if constexpr (sizeof(E) == 2)
        return grad_launch<E, G, 8>(dy, key, pos, n, V, D, scale, add, dw, piece, runs, s, d);
    case 4: return grad_launch<E, G, 4>(dy, key, pos, n, V, D, scale, add, dw, piece, runs, s, d);
    case 2: return grad_launch<E, G, 2>(dy, key, pos, n, V, D, scale, add, dw, piece, runs, s, d);
    default: return grad_launch<E, G, 1>(dy, key, pos, n, V, D, scale, add, dw, piece, runs, s, d);
  }
}

}  // namespace

int launch_embedding(const void *w, int64_t V, int64_t D, int dtype, const void *tok, bool wide,
                     int64_t n, float scale, void *out, cudaStream_t s) {
  const int64_t es = dtype == RR_BF16 ? 2 : 4;
  const int vb = access_bytes((uintptr_t)w | (uintptr_t)out | (uintptr_t)(D * es));
  if (dtype == RR_BF16) {
    switch (vb) {
      case 16: return embed_launch<unsigned short, 16>(w, V, D, tok, wide, n, scale, out, s);
      case 8: return embed_launch<unsigned short, 8>(w, V, D, tok, wide, n, scale, out, s);
      case 4: return embed_launch<unsigned short, 4>(w, V, D, tok, wide, n, scale, out, s);
      default: return embed_launch<unsigned short, 2>(w, V, D, tok, wide, n, scale, out, s);
    }
  }
  switch (vb) {
    case 16: return embed_launch<float, 16>(w, V, D, tok, wide, n, scale, out, s);
    case 8: return embed_launch<float, 8>(w, V, D, tok, wide, n, scale, out, s);
    default: return embed_launch<float, 4>(w, V, D, tok, wide, n, scale, out, s);
  }
}

size_t embedding_grad_ws_bytes(int64_t n, int64_t D) {
  if (n == 0) return 0;
  const int L = grad_chunk(n, D);
  const int64_t chunks = (n + L - 1) / L;
  return 4 * list_bytes(n) + runs_bytes(chunks) + (chunks > 1 ? (size_t)chunks * 2 * D * sizeof(float) : 0);
}

bool embedding_grad_fits(const void *dy, int64_t n, int64_t D, int dtype, const void *dw, int dw_dtype) {
  if (n == 0) return true;
  const int L = grad_chunk(n, D);
  return grad_tiles(D, grad_column(dy, dtype, dw, dw_dtype, D)) * ((n + L - 1) / L) <= INT_MAX;
}

int launch_embedding_grad(const void *dy, int64_t n, int64_t D, int dtype, const void *tok,
                          bool wide, int64_t V, float scale, void *dw, int dw_dtype, bool add,
                          void *ws, cudaStream_t s, const DevInfo &d) {
  const int64_t gs = dw_dtype == RR_BF16 ? 2 : 4;
  SortArgs a;
  a.tok = tok;
  a.wide = wide;
  a.n = (int)n;
  a.V = V;
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;   // keys 0 .. V
  a.passes = (bits + kSortBits - 1) / kSortBits;
  a.bits = (bits + a.passes - 1) / a.passes;
  unsigned char *p = (unsigned char *)ws;
  for (int k = 0; k < 2; ++k) {
    a.key[k] = (int *)(p + (size_t)(2 * k) * list_bytes(n));
    a.pos[k] = (int *)(p + (size_t)(2 * k + 1) * list_bytes(n));
  }
  int *runs = (int *)(p + 4 * list_bytes(n));
  a.runs = runs;
  const int64_t chunks = (n + grad_chunk(n, D) - 1) / grad_chunk(n, D);
  float *piece = (float *)((unsigned char *)runs + runs_bytes(chunks));
  const size_t fill_bytes = add ? 0 : (size_t)V * D * gs;
  // a CTA per 1024 entries, up to a cluster of 16; beside a fill, which takes
  // longer, per 4096 and of 4: larger ones leave more SMs out (131072 x 4096
  // bf16 beside 16384 tokens 208 us in all, with 8 219, with 16 245; alone,
  // 4096 tokens take 30 us in a cluster of 4 and 41 in one CTA)
  int C = 1;
  while (C < (fill_bytes ? 4 : 16) && (int64_t)C * (fill_bytes ? kSortEach : kSortThreads) < n) C *= 2;
  auto per = [&](int c) { return (int)((n + (int64_t)c * kSortThreads - 1) / ((int64_t)c * kSortThreads)) * kSortThreads; };
  static std::atomic<uint64_t> allowed_chip{0}, allowed_long{0};
  cudaError_t e = allow_kernel(k_token_sort<true>, sort_smem(kSortBits, kSortChip), true, d.device, allowed_chip);
  if (e == cudaSuccess)
    e = allow_kernel(k_token_sort<false>, sort_smem(kSortBits, 0), true, d.device, allowed_long);
  if (e != cudaSuccess) return cuda_status(e);
  bool chip;
  size_t smem;
  const void *func;
  for (;; C /= 2) {
    a.per = per(C);
    chip = a.per <= kSortChip;
    smem = sort_smem(a.bits, chip ? a.per : 0);
    if (smem < kZeros) smem = kZeros;
    func = chip ? (const void *)k_token_sort<true> : (const void *)k_token_sort<false>;
    if (C == 1 || (d.cluster_launch && occupancy_clusters(func, kSortThreads, smem, C, d.device) >= 1)) break;
  }
  // as many as run at once (each has an equal part, and one that starts when
  // the others end takes 110 us more), and no more than there are pieces of 64 KiB
  int64_t fill = 0;
  if (fill_bytes) {
    fill = (C > 1 ? occupancy_clusters(func, kSortThreads, smem, C, d.device)
                  : occupancy_blocks(func, kSortThreads, smem, d.device) * d.sm_count) - 1;
    const int64_t most = (int64_t)(fill_bytes / ((size_t)C * 65536)) + 1;
    if (fill > most) fill = most;
    if (fill < 1) fill = 1;
  }
  if (log_enabled())
    std::fprintf(stderr, "[rr] token sort n=%d passes=%d bits=%d C=%d on chip=%d fill=%lld clusters\n",
                 a.n, a.passes, a.bits, C, chip, (long long)fill);
  e = launch_kernel(chip ? k_token_sort<true> : k_token_sort<false>, dim3((unsigned)(C * (1 + fill))),
                    dim3(kSortThreads), smem, s, C, a, (unsigned char *)dw, fill_bytes);
  if (e != cudaSuccess || n == 0) return cuda_status(e);
  const int out = chip ? 0 : (a.passes - 1) & 1;
  const int *key = a.key[out], *pos = a.pos[out];
  const int width = grad_column(dy, dtype, dw, dw_dtype, D);
  if (dtype == RR_F32)
    return grad_width<float, float>(width, dy, key, pos, a.n, V, D, scale, add, dw, piece, runs, s, d);
  if (dw_dtype == RR_F32)
    return grad_width<unsigned short, float>(width, dy, key, pos, a.n, V, D, scale, add, dw, piece, runs, s, d);
  return grad_width<unsigned short, unsigned short>(width, dy, key, pos, a.n, V, D, scale, add, dw,
                                                    piece, runs, s, d);
}

}  // namespace rr
