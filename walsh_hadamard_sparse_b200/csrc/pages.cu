// The page table (which pages hold which sequence's tokens) and the moves of
// cached rows: growing, shrinking and forking of sequences, copies of pages, and
// tokens that move together.
//
// The table calls are a chain of short dependent steps over a few hundred
// kilobytes (counts, prefix sums in the order of the sequences, the free pages in
// ascending order), so latency bounds them, not memory. One cluster of CTAs does
// a call in one launch: its barriers take the place of launches, and what the
// CTAs tell each other goes through the workspace (written before a barrier,
// read past L1 after it). Nothing in the workspace is read that the call has not
// written. A step of 64 sequences (8 forked, all grown, some released): 34 us for its
// calls; of 2048 sequences over 200 thousand pages: 72 us.
//
// The moves are bound by memory where they are large, by a launch where not: pages
// copied and 8 of 64 tokens kept for 512 sequences, 8 heads of 128, 8 bits, 319 MB:
// 89 us, 3.6 TB/s of the 6.5 that a copy moves; for one sequence, 6 us. Kept tokens of a
// long context move one after the other: 32768 of 65536 tokens, 7.4 ms.

#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace qwha {
namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int64_t kNone = INT64_MAX;

// What the CTAs of a call tell each other, at the head of the workspace.
struct Shared {
  long long wanted[kMaxCtas];  // pages that the CTA's sequences ask for
  long long free[kMaxCtas];    // free pages of the CTA's share of refs
  long long granted[kMaxCtas];  // pages that they get
};

// The sum of the values in warp_s of the warps before this one, and of all (32 warps).
__device__ __forceinline__ long long warps_before(const long long *warp_s, long long *sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long mine = warp_s[lane];
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long p = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += p;
  }
  *sum = __shfl_sync(~0u, upto, 31);
  return __shfl_sync(~0u, upto - mine, warp);
}

// The `v` of the threads before this one in the CTA, and the CTA's sum.
__device__ __forceinline__ long long block_before(long long v, long long *warp_s, long long *sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long upto = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long p = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += p;
  }
  __syncthreads();  // warp_s is free
  if (lane == 31) warp_s[warp] = upto;
  __syncthreads();
  return warps_before(warp_s, sum) + upto - v;
}

// Pages of a sequence's tokens: x / ps rounded up, for 0 <= x (in 32 bits where x fits, a third of the time).
__device__ __forceinline__ int64_t pages_of(int64_t x, int ps) {
  x += ps - 1;
  return x >> 32 ? x / ps : (int64_t)((uint32_t)x / (uint32_t)ps);
}

// The CTA's share [lo, hi) of n things, in order.
__device__ __forceinline__ void share(int64_t n, int part, int parts, int *lo, int *hi) {
  *lo = (int)(n * part / parts), *hi = (int)(n * (part + 1) / parts);
}

// Free pages of this warp's run of refs: how many, and (list) which, from place
// `at` of the ascending list on, as far as `need` pages of it are wanted.
__device__ __forceinline__ long long warp_free(const int32_t *refs, int lo, int hi, int32_t *list, long long at,
                                               long long need, int32_t *take) {
  const int lane = threadIdx.x & 31;
  long long count = 0;
  for (int p0 = lo; p0 < hi; p0 += 32 * 4) {
    int ref[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) ref[u] = p0 + u * 32 + lane < hi ? __ldcg(refs + p0 + u * 32 + lane) : 1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned mask = __ballot_sync(~0u, ref[u] == 0);
      if (list) {
        const long long place = at + count + __popc(mask & ((1u << lane) - 1));
        if (ref[u] == 0 && place < need) list[place] = p0 + u * 32 + lane, take[p0 + u * 32 + lane] = 1;
      }
      count += __popc(mask);
    }
    if (list && at + count >= need) break;
  }
  return count;
}

// Counts the free pages of every CTA's share; on return `before` is the number
// before this warp's run [lo, hi) of refs within the CTA.
__device__ __forceinline__ void count_free(const qwha_page_table &t, int rank, int ctas, Shared *sh, long long *warp_s,
                                           int *lo, int *hi, long long *before) {
  int c0, c1;
  share(t.n_pages, rank, ctas, &c0, &c1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int w0, w1;
  share(c1 - c0, warp, kTableWarps, &w0, &w1);
  *lo = c0 + w0, *hi = c0 + w1;
  const long long mine = warp_free(t.refs, *lo, *hi, nullptr, 0, 0, nullptr);
  __syncthreads();
  if (lane == 0) warp_s[warp] = mine;
  __syncthreads();
  long long all;
  *before = warps_before(warp_s, &all);
  if (threadIdx.x == 0) sh->free[rank] = all;
  __syncthreads();
}

__device__ __forceinline__ long long sum_of(const long long *v, int n) {
  long long s = 0;
  for (int i = 0; i < n; ++i) s += __ldcg(v + i);
  return s;
}

// GUARD: a row that grows from an end inside a page with other users claims a page
// in its place (origin, fresh: where the two are named), or, without these, is left.
// Which rows do is known only behind the pages given back: a barrier more.
template <bool GUARD>
__global__ void __launch_bounds__(kTableThreads, 1)
    resize_kernel(const qwha_page_table t, const int64_t *__restrict__ want, int32_t *origin, int32_t *fresh, Shared *sh,
                  int64_t *from, int32_t *list, unsigned int *err) {
  __shared__ long long warp_s[kTableWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ps = t.page_size;
  const int64_t room = (int64_t)ps * t.max_pages;
  int s0, s1;
  share(t.n_seqs, rank, ctas, &s0, &s1);
  // pages each sequence asks for, and how many are asked for before it in the CTA: from[b], twice that and whether the first
  // of them is claimed
  long long asked = 0;
  auto ask = [&] {
    for (int b0 = s0; b0 < s1; b0 += kTableThreads) {
      const int b = b0 + threadIdx.x;
      long long need = 0;
      int claim = 0;
      if (b < s1) {
        const int64_t w = want[b], h = t.held[b];
        if (w == -1) {
        } else if (w < -1 || w > room || h < 0 || h > room) {
          atomicOr(err, kErrTable);
        } else {
          need = pages_of(w, ps) - pages_of(h, ps);
          if (need < 0) need = 0;
          if constexpr (GUARD) {
            if (w > h) {
              const int64_t end = pages_of(h, ps) - 1;
              if (end >= 0 && (end + 1) * ps != h) {
                const int32_t p = t.pages[(int64_t)b * t.max_pages + end];
                const bool in = p >= 0 && p < t.n_pages;
                claim = !in || __ldcg(t.refs + p) > 1;
                if (claim && !(in && origin)) {  // it cannot be given a page of its own
                  atomicOr(err, kErrTable);
                  claim = -1, need = 0;
                }
              }
              if (claim == 0 && need == 0) t.held[b] = w;
            }
          }
          need += claim > 0;
        }
        if (GUARD && origin) origin[b] = fresh[b] = -1;
      }
      long long sum;
      const long long before = block_before(need, warp_s, &sum);
      if (b < s1) from[b] = need > 0 ? 2 * (asked + before) + (claim > 0) : kNone;
      asked += sum;
    }
    if (threadIdx.x == 0) sh->wanted[rank] = asked;
  };
  if (!GUARD) ask();
  // The ends that are given back: eight lanes a sequence, neighbours to different CTAs, since long ends come together and
  // an SM makes about one atomic operation in two clocks. (What this changes of held is of sequences that do not grow,
  // whose held nobody needs from here on.)
  const int eighth = threadIdx.x & 7, group = threadIdx.x >> 3;
  constexpr int kGroups = kTableThreads / 8;
  for (int b = group * ctas + rank; b < t.n_seqs; b += kGroups * ctas) {
    const int64_t w = want[b], h = t.held[b];
    if (w < 0 || w > room || h < 0 || h > room) continue;
    const int64_t have = pages_of(h, ps), to = pages_of(w, ps);
    int32_t *row = t.pages + (int64_t)b * t.max_pages;
    bool bad = false;
#pragma unroll 4
    for (int64_t j = to + eighth; j < have; j += 8) bad |= (uint32_t)row[j] >= (uint32_t)t.n_pages;
    if (__any_sync(0xffu << (threadIdx.x & 24), bad)) {  // left as it is
      if (bad) atomicOr(err, kErrTable);
      continue;
    }
#pragma unroll 4
    for (int64_t j = to + eighth; j < have; j += 8) {
      const int32_t p = row[j];
      row[j] = -1;
      if (atomicSub(t.refs + p, 1) <= 0) {  // fewer users counted than there are
        atomicAdd(t.refs + p, 1);
        atomicOr(err, kErrTable);
      }
    }
    __syncwarp(0xffu << (threadIdx.x & 24));  // the eight lanes have read held
    if (eighth == 0 && (GUARD ? w <= h : to <= have)) t.held[b] = w;
  }
  cluster.sync();
  if (GUARD) {
    ask();
    cluster.sync();
  }
  const long long total = sum_of(sh->wanted, ctas);
  if (total == 0) return;  // every CTA sees the same
  int lo, hi;
  long long before;
  count_free(t, rank, ctas, sh, warp_s, &lo, &hi, &before);
  cluster.sync();
  const long long n_free = sum_of(sh->free, ctas), asked_before = sum_of(sh->wanted, rank);
  // whose request ends within the free pages, and how many pages are taken
  __shared__ unsigned long long granted_s;
  if (threadIdx.x == 0) granted_s = 0;
  __syncthreads();
  for (int b = s0 + threadIdx.x; b < s1; b += kTableThreads) {
    if (from[b] == kNone) continue;
    const int claim = (int)(from[b] & 1);
    const long long need = pages_of(want[b], ps) - pages_of(t.held[b], ps) + claim, at = asked_before + (from[b] >> 1);
    if (at + need <= n_free) atomicMax(&granted_s, (unsigned long long)(at + need));
    from[b] = at + need <= n_free ? 2 * at + claim : kNone;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh->granted[rank] = (long long)granted_s;
  cluster.sync();
  long long granted = 0;
  for (int i = 0; i < ctas; ++i) granted = max(granted, __ldcg(sh->granted + i));
  const long long free_before = sum_of(sh->free, rank) + before;
  if (free_before < granted) warp_free(t.refs, lo, hi, list, free_before, granted, t.refs);
  cluster.sync();
  for (int b = s0 + group; b < s1; b += kGroups) {
    if (from[b] == kNone) continue;
    const int64_t at = from[b] >> 1, claim = from[b] & 1;
    const int64_t w = want[b], have = pages_of(t.held[b], ps), to = pages_of(w, ps);
    int32_t *row = t.pages + (int64_t)b * t.max_pages;
    for (int64_t j = have + eighth; j < to; j += 8) row[j] = __ldcg(list + at + claim + (j - have));
    if (GUARD && claim && eighth == 0) {
      const int32_t old = row[have - 1], own = __ldcg(list + at);
      row[have - 1] = own;
      atomicSub(t.refs + old, 1);
      origin[b] = old, fresh[b] = own;
    }
    __syncwarp(0xffu << (threadIdx.x & 24));  // the eight lanes have read held
    if (eighth == 0) t.held[b] = w;
  }
}

__global__ void __launch_bounds__(kTableThreads, 1)
    fork_kernel(const qwha_page_table t, const int64_t *__restrict__ src, const int64_t *__restrict__ dst, int m,
                int32_t *origin, int32_t *fresh, Shared *sh, int64_t *from, int64_t *tokens, int32_t *owner,
                int32_t *list, unsigned int *err) {
  __shared__ long long warp_s[kTableWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ps = t.page_size;
  const int64_t room = (int64_t)ps * t.max_pages;
  int m0, m1;
  share(m, rank, ctas, &m0, &m1);
  auto in_table = [&](int64_t b) { return b >= 0 && b < t.n_seqs; };
  for (int i = m0 + threadIdx.x; i < m1; i += kTableThreads)
    if (in_table(src[i]) && in_table(dst[i])) owner[dst[i]] = INT32_MAX;
  // rows whose pages are none, or count no users, are not copied: tokens[i] -1
  for (int i = m0 + warp; i < m1; i += kTableWarps) {
    bool bad = false;
    if (in_table(src[i]) && in_table(dst[i])) {
      const int64_t h = t.held[src[i]];
      const int32_t *row = t.pages + src[i] * t.max_pages;
      if (h > 0 && h <= room)
#pragma unroll 4
        for (int64_t j = lane; j < pages_of(h, ps); j += 32) bad |= (uint32_t)row[j] >= (uint32_t)t.n_pages || t.refs[row[j]] <= 0;
    }
    bad = __any_sync(~0u, bad);
    if (lane == 0) tokens[i] = bad ? -1 : 0;
  }
  cluster.sync();
  for (int i = m0 + threadIdx.x; i < m1; i += kTableThreads)
    if (in_table(src[i]) && in_table(dst[i])) atomicMin(owner + dst[i], i);
  cluster.sync();
  long long asked = 0;
  for (int i0 = m0; i0 < m1; i0 += kTableThreads) {
    const int i = i0 + threadIdx.x;
    long long need = 0;
    if (i < m1) {
      const int64_t a = src[i], b = dst[i];
      int64_t h = -1;
      if (in_table(a) && in_table(b) && __ldcg(owner + b) == i && t.held[b] == 0 && tokens[i] == 0) h = t.held[a];
      if (h > room) h = -1;
      if (h < 0 && a != -1) atomicOr(err, kErrTable);
      tokens[i] = h;
      need = h > 0 && pages_of(h, ps) * ps != h;
    }
    long long sum;
    const long long before = block_before(need, warp_s, &sum);
    if (i < m1) from[i] = asked + before;  // pages that the pairs before it need
    asked += sum;
  }
  if (threadIdx.x == 0) sh->wanted[rank] = asked;
  int lo, hi;
  long long before;
  count_free(t, rank, ctas, sh, warp_s, &lo, &hi, &before);
  cluster.sync();  // held and refs have been read as they were
  const long long n_free = sum_of(sh->free, ctas), wanted = sum_of(sh->wanted, ctas);
  const long long asked_before = sum_of(sh->wanted, rank), granted = min(n_free, wanted);
  const long long free_before = sum_of(sh->free, rank) + before;
  if (free_before < granted) warp_free(t.refs, lo, hi, list, free_before, granted, t.refs);
  cluster.sync();
  for (int i = m0 + warp; i < m1; i += kTableWarps) {
    const int64_t h = tokens[i], full = h < 0 ? 0 : pages_of(h - ps + 1, ps), at = asked_before + from[i];
    const bool needs = h > full * ps, served = h >= 0 && at + needs <= n_free;
    int32_t o = -1, f = -1;
    if (served) {
      const int32_t *row = t.pages + src[i] * t.max_pages;
      int32_t *copy = t.pages + dst[i] * t.max_pages;
      for (int64_t j = lane; j < full; j += 32) {
        const int32_t p = row[j];
        copy[j] = p;
        atomicAdd(t.refs + p, 1);
      }
      if (needs) {
        o = row[full], f = __ldcg(list + at);
        if (lane == 0) copy[full] = f;
      }
      if (lane == 0) t.held[dst[i]] = h;
    }
    if (lane == 0) origin[i] = o, fresh[i] = f;
  }
}

struct TableWs {
  Shared *sh;
  int64_t *from, *tokens;
  int32_t *owner, *list;
  size_t bytes;
};
TableWs carve(void *ws, int64_t n_seqs, int64_t n_pages, int64_t m) {
  const int64_t rows = std::max(n_seqs, m);
  char *p = static_cast<char *>(ws);
  TableWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    char *r = p + at;
    at += align_up(n, 256);
    return r;
  };
  w.sh = reinterpret_cast<Shared *>(take(sizeof(Shared)));
  w.from = reinterpret_cast<int64_t *>(take((size_t)rows * 8));
  w.tokens = reinterpret_cast<int64_t *>(take(m ? (size_t)m * 8 : 0));
  w.owner = reinterpret_cast<int32_t *>(take(m ? (size_t)n_seqs * 4 : 0));
  w.list = reinterpret_cast<int32_t *>(take((size_t)n_pages * 4));
  w.bytes = at;
  return w;
}

template <typename... K, typename... A>
cudaError_t launch_table(void (*kernel)(K...), int64_t pages, int64_t rows, cudaStream_t s, A... args) {
  // One CTA for a small table: a cluster's barriers cost more than they save there (a call that grows or cuts all rows, us
  // with one CTA and with eight: 64 rows, 2048 pages 7.4 and 9.8; 64, 16384 9.0 and 10.3; 64, 65536 12.8 and 10.8; 256, 16384 11.7
  // and 11.5; 1024, 16384 21.6 and 11.8).
  const int ctas = pages <= 16384 && rows <= 256 ? 1 : kMaxCtas;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(ctas), c.blockDim = dim3(kTableThreads), c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = ctas, a[0].val.clusterDim.y = 1, a[0].val.clusterDim.z = 1;
  c.attrs = a, c.numAttrs = ctas > 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<K>(args)...);
}

// ---------------------------------------------------------------- rows that move

constexpr int kMoveThreads = 256;

// The widest access that n bytes and everything at multiples of n bytes allow.
__host__ __device__ __forceinline__ int width_of(int64_t n) {
  return n % 16 == 0 ? 16 : n % 8 == 0 ? 8 : n % 4 == 0 ? 4 : n % 2 == 0 ? 2 : 1;
}

// Eight loads of a thread in flight.
template <typename V>
__device__ __forceinline__ void copy_run(char *dst, const char *src, int64_t bytes) {
  constexpr int U = 8;
  const int64_t n = bytes / (int64_t)sizeof(V);
  for (int64_t i = threadIdx.x; i < n; i += kMoveThreads * U) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kMoveThreads < n) v[u] = reinterpret_cast<const V *>(src)[i + u * kMoveThreads];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kMoveThreads < n) reinterpret_cast<V *>(dst)[i + u * kMoveThreads] = v[u];
  }
}
__device__ __forceinline__ void copy_bytes(char *dst, const char *src, int64_t bytes, int width) {
  switch (width) {
    case 16: copy_run<uint4>(dst, src, bytes); break;
    case 8: copy_run<uint2>(dst, src, bytes); break;
    case 4: copy_run<uint32_t>(dst, src, bytes); break;
    case 2: copy_run<uint16_t>(dst, src, bytes); break;
    default: copy_run<uint8_t>(dst, src, bytes);
  }
}

constexpr int64_t kPiece = kMoveThreads * 8 * 16;  // bytes a CTA copies at a time

// blockIdx.y: 3 cache + 0 codes, 1 scales, 2 zero points.
__global__ void __launch_bounds__(kMoveThreads) copy_pages_kernel(const __grid_constant__ CachePair c,
                                                                  const int32_t *__restrict__ from,
                                                                  const int32_t *__restrict__ to, int m, unsigned int *err) {
  const int what = blockIdx.y % 3;
  const qwha_cache &a = c.cache[blockIdx.y / 3];
  const int64_t row = (int64_t)a.page_size * a.heads, groups = row * (a.head_dim / a.group);
  const int64_t bytes = what == 0 ? row * (a.head_dim / 8 * a.bits) : what == 1 ? groups * 4 : groups;
  char *base = what == 0 ? reinterpret_cast<char *>(a.codes) : what == 1 ? reinterpret_cast<char *>(a.scales) : reinterpret_cast<char *>(a.zeros);
  const int width = width_of(bytes);
  const int64_t pieces = (bytes + kPiece - 1) / kPiece;
  // pieces of a page one after the other in one CTA's turns, while pages alone fill the grid
  for (int64_t w = blockIdx.x; w < m * pieces; w += gridDim.x) {
    const int i = pieces == 1 ? (int)w : (int)(w / pieces);
    const int64_t lo = (w - i * pieces) * kPiece, hi = lo + kPiece < bytes ? lo + kPiece : bytes;
    const int64_t f = from[i], t = to[i];
    if (f == -1 || t == -1) continue;
    if (f < 0 || t < 0 || f >= a.n_pages || t >= a.n_pages) {
      if (threadIdx.x == 0) atomicOr(err, kErrPage);
      continue;
    }
    copy_bytes(base + t * bytes + lo, base + f * bytes + lo, hi - lo, width);
  }
}

// Tokens that move down: a thread owns some bytes of a token's rows and carries
// them from token to token in ascending order, eight reads ahead of their
// writes. keep ascends, so keep[i] >= i and the place that move i writes is read
// by no later move: nothing has to wait for another thread.
constexpr int kAhead = 8;
constexpr int kMoves = 128;  // moves whose slots are looked up at a time, one a thread

template <typename V>
__device__ __forceinline__ void move_column(char *base, int64_t row, int64_t at, const int64_t *from, const int64_t *to,
                                            int n) {
  for (int i = 0; i < n; i += kAhead) {
    V v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u < n && from[i + u] >= 0) v[u] = *reinterpret_cast<const V *>(base + from[i + u] * row + at);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u < n && from[i + u] >= 0) *reinterpret_cast<V *>(base + to[i + u] * row + at) = v[u];
  }
}
// A token's bytes in one cache: codes, scales and zero points, each in accesses as
// wide as its rows allow.
struct Columns {
  int64_t row[3], count[3];
  int width[3];
  __host__ __device__ explicit Columns(const qwha_cache &a) {
    const int64_t groups = (int64_t)a.heads * (a.head_dim / a.group);
    row[0] = (int64_t)a.heads * (a.head_dim / 8 * a.bits), row[1] = groups * 4, row[2] = groups;
    for (int i = 0; i < 3; ++i) width[i] = width_of(row[i]), count[i] = row[i] / width[i];
  }
  __host__ __device__ int64_t total() const { return count[0] + count[1] + count[2]; }
};

__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const __grid_constant__ CachePair c, const int32_t *__restrict__ pages, int max_pages,
                   const int64_t *__restrict__ first, const int32_t *__restrict__ keep, int width, unsigned int *err) {
  __shared__ int64_t from_s[kMoves], to_s[kMoves];
  __shared__ int stop_s;
  const qwha_cache &a = c.cache[blockIdx.y];
  const int b = blockIdx.z;
  const int32_t *row = keep + (int64_t)b * width;
  const Columns col(a);
  auto slot = [&](int64_t t) -> int64_t {
    if (t < 0) return -1;
    const int64_t pg = t >> 32 ? t / a.page_size : (int64_t)((uint32_t)t / (uint32_t)a.page_size);
    if (pg >= max_pages) return -1;
    const int64_t page = pages[(int64_t)b * max_pages + pg];
    return page < 0 || page >= a.n_pages ? -1 : page * a.page_size + (t - pg * a.page_size);
  };
  for (int i0 = 0; i0 < width; i0 += kMoves) {
    const int n = width - i0 < kMoves ? width - i0 : kMoves;
    __syncthreads();
    if (threadIdx.x == 0) stop_s = n;
    __syncthreads();
    const int i = threadIdx.x, k = i < n ? row[i0 + i] : 0;
    if (i < n) {
      const int last = i0 + i ? row[i0 + i - 1] : -1;
      if (k <= last || k < 0) atomicMin(&stop_s, i);
    }
    __syncthreads();
    const int stop = stop_s;
    // -1 ends the row; anything else that does not ascend breaks it off
    if (threadIdx.x == 0 && stop < n && row[i0 + stop] != -1) atomicOr(err, kErrTable);
    if (i < stop) {
      int64_t f = -1, t = -1;
      if (k != i0 + i) {
        f = slot(first[b] + k), t = slot(first[b] + i0 + i);
        if (f < 0 || t < 0) {
          f = -1;
          atomicOr(err, kErrPage);
        }
      }
      from_s[i] = f, to_s[i] = t;
    }
    __syncthreads();
    for (int64_t x = blockIdx.x * kMoveThreads + threadIdx.x; x < col.total(); x += (int64_t)gridDim.x * kMoveThreads) {
      const int what = x < col.count[0] ? 0 : x < col.count[0] + col.count[1] ? 1 : 2;
      const int64_t in = what == 0 ? x : what == 1 ? x - col.count[0] : x - col.count[0] - col.count[1];
      const int64_t bytes = what == 0 ? col.row[0] : what == 1 ? col.row[1] : col.row[2];
      const int w = what == 0 ? col.width[0] : what == 1 ? col.width[1] : col.width[2];
      char *base = what == 0 ? reinterpret_cast<char *>(a.codes) : what == 1 ? reinterpret_cast<char *>(a.scales) : reinterpret_cast<char *>(a.zeros);
      switch (w) {
        case 16: move_column<uint4>(base, bytes, in * 16, from_s, to_s, stop); break;
        case 8: move_column<uint2>(base, bytes, in * 8, from_s, to_s, stop); break;
        case 4: move_column<uint32_t>(base, bytes, in * 4, from_s, to_s, stop); break;
        case 2: move_column<uint16_t>(base, bytes, in * 2, from_s, to_s, stop); break;
        default: move_column<uint8_t>(base, bytes, in, from_s, to_s, stop);
      }
    }
    if (stop < n) break;
  }
}

}  // namespace

size_t pages_workspace(int64_t n_seqs, int64_t n_pages, int64_t m) { return carve(nullptr, n_seqs, n_pages, m).bytes; }

cudaError_t launch_pages_resize(const qwha_page_table &t, const int64_t *want, int32_t *from, int32_t *to, void *ws,
                                cudaStream_t s) {
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  const TableWs w = carve(ws, t.n_seqs, t.n_pages, 0);
  return launch_table(t.guard || from ? resize_kernel<true> : resize_kernel<false>, t.n_pages, t.n_seqs, s, t, want, from, to,
                      w.sh, w.from, w.list, err);
}

cudaError_t launch_pages_fork(const qwha_page_table &t, const int64_t *src, const int64_t *dst, int32_t m,
                              int32_t *from, int32_t *to, void *ws, cudaStream_t s) {
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  const TableWs w = carve(ws, t.n_seqs, t.n_pages, m);
  return launch_table(fork_kernel, t.n_pages, m, s, t, src, dst, m, from, to, w.sh, w.from, w.tokens, w.owner, w.list, err);
}

cudaError_t launch_copy_pages(const CachePair &c, int n_caches, const int32_t *from, const int32_t *to, int32_t m,
                              cudaStream_t s) {
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  int64_t most = 1;
  for (int i = 0; i < n_caches; ++i) {
    const qwha_cache &a = c.cache[i];
    most = std::max<int64_t>(most, cdiv((int64_t)a.page_size * a.heads * (a.head_dim / 8 * a.bits), kPiece));
  }
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)m * most, (int64_t)sm_count() * 64), (unsigned)n_caches * 3);
  copy_pages_kernel<<<grid, kMoveThreads, 0, s>>>(c, from, to, m, err);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CachePair &c, int n_caches, const int32_t *pages, int32_t max_pages,
                           const int64_t *first, const int32_t *keep, int32_t width, int32_t n_seqs, cudaStream_t s) {
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  int64_t columns = 1;
  for (int i = 0; i < n_caches; ++i) {
    columns = std::max(columns, Columns(c.cache[i]).total());
  }
  for (int32_t b0 = 0; b0 < n_seqs; b0 += 65535) {
    const int32_t here = std::min(n_seqs - b0, 65535);
    compact_kernel<<<dim3((unsigned)cdiv(columns, kMoveThreads), (unsigned)n_caches, (unsigned)here), kMoveThreads, 0, s>>>(
        c, pages + (int64_t)b0 * max_pages, max_pages, first + b0, keep + (int64_t)b0 * width, width, err);
  }
  return cudaGetLastError();
}

}  // namespace qwha
