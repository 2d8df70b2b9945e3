// What the kernels of attention over the quantized cache share: how the work is
// cut, the rows' queries and masks, and how a row is finished.
//
// The work of a call is the list of its units, in this order: sequence, block of
// cached heads, part of their query heads, tile of the sequence's new tokens, run
// of 2^kt_log2 cached tokens. Its length follows from lengths that only the device
// knows, so each CTA adds them up itself and takes an equal share of the units,
// whatever sequences they belong to: one long sequence and many short ones fill
// the GPU alike. A segment is what a CTA does of one tile of rows; a tile whose
// run is cut between CTAs leaves its pieces (maximum, sum, values, all fp32) in
// the workspace, and a second launch joins them in order of the cached tokens.
#pragma once

#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace qwha {
namespace attn {

// How far scales may lie apart on tcgen05 (attention_tc.cu): the largest of its group of
// values, or of a head's keys, is at least 2^4 in f16, so that one within 2^-13 of it has
// 2^-9, of which the second piece, to 2^-25, keeps all but 2^-16.
constexpr float kSpreadTc = 8192.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int clamp_rows(int64_t v, int64_t lo, int64_t hi) { return (int)(v < lo ? lo : v > hi ? hi : v); }

// One sequence of the call. Row numbers fit 31 bits (checked on the host), and so
// do cached tokens (`cap` is cut there).
struct Seq {
  int row0, rows;      // its new tokens: rows of q
  int past, seen;      // tokens before them; tokens that some row sees
  int tiles;           // tiles of new tokens
  bool flat;           // every tile runs over `seen` tokens

  __device__ __forceinline__ Seq(const AttnArgs &a, int b) {
    row0 = clamp_rows(a.q_start[b], 0, a.n);
    rows = clamp_rows(a.q_start[b + 1], row0, a.n) - row0;
    past = clamp_rows(a.past[b], 0, a.cap);
    const int fresh = a.tree && rows > 64 ? 64 : rows;
    flat = a.tree || (long long)past + fresh > a.cap;
    seen = (long long)past + fresh > a.cap ? a.cap : past + fresh;
    tiles = rows <= a.tq ? rows > 0 : (rows + a.tq - 1) / a.tq;
  }
  // units of one block of heads and part: sum over the tiles
  __device__ __forceinline__ long long per_block(const AttnArgs &a) const { return upto(a, tiles); }
  // Whether the sequence's token j sees cached token t (bits: its mask of a tree).
  __device__ __forceinline__ bool sees(const AttnArgs &a, int j, unsigned long long bits, int t) const {
    const int u = t - past;
    return u < 0 || (a.tree ? u < 64 && (bits >> u & 1) : u <= j);
  }
  __device__ __forceinline__ int length(const AttnArgs &a, int tile) const {
    const long long end = (long long)(tile + 1) * a.tq;
    return flat || end >= rows ? seen : past + (int)end;
  }
  __device__ __forceinline__ int units(const AttnArgs &a, int tile) const {
    const int n = (length(a, tile) + (1 << a.kt_log2) - 1) >> a.kt_log2;
    return n > 0 ? n : 1;
  }
  // Units of the tiles before `tile`: sums of floor((tq i + c) / kt), by the
  // steps of Euclid's algorithm.
  __device__ long long upto(const AttnArgs &a, int tile) const {
    if (tile <= 0) return 0;
    if (flat || tile == 1) return (long long)tile * units(a, 0);
    const bool all = tile == tiles;
    long long n = all ? tile - 1 : tile, sum = all ? units(a, tile - 1) : 0;
    long long m = 1 << a.kt_log2, s = a.tq, c = (long long)past + a.tq + m - 1;
    for (;;) {
      sum += n * (n - 1) / 2 * (s / m) + n * (c / m);
      s %= m, c %= m;
      const long long top = s * n + c;
      if (top < m) break;
      n = top / m, c = top % m;
      const long long t = m;
      m = s, s = t;
    }
    return sum;
  }
};

// The quotient by the parts of a group, which is nearly always whole.
__device__ __forceinline__ int block_of(const AttnArgs &a, int block) { return a.parts == 1 ? block : block / a.parts; }

// Where a CTA is in the list.
struct Place {
  int b, block, tile, unit;  // block: of heads and parts together
};

// A CTA's share of the units and where it begins. Little work goes to as many CTAs as
// it has units, although that makes more pieces (two units to a CTA at the least: 43
// us for 30 with 5 fp32 trees of 7 tokens behind 700, 19.3 for 18.6 with one token
// behind 700). All threads of the CTA (whole warps) call it.
__device__ __forceinline__ long long my_share(const AttnArgs &a, Place *at) {
  __shared__ long long warp_s[32];
  __shared__ Place place_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, THREADS = blockDim.x;
  const long long blocks = a.blocks;
  long long all = 0, mine = 0;
  auto add_up = [&](int b0) {  // units of sequence b0 + thread, of those before it, of all of these
    const int b = b0 + threadIdx.x;
    mine = b < a.n_seqs ? Seq(a, b).per_block(a) * blocks : 0;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long p = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += p;
    }
    __syncthreads();
    if (lane == 31) warp_s[warp] = upto;
    __syncthreads();
    long long before = upto - mine, sum = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += warp_s[w];
      sum += warp_s[w];
    }
    all = sum;
    return before;
  };
  long long before = add_up(0), total = all;
  for (int b0 = THREADS; b0 < a.n_seqs; b0 += THREADS) {
    add_up(b0);
    total += all;
  }
  const int ctas = total < gridDim.x ? (int)total : gridDim.x, c = blockIdx.x;
  if (c >= ctas) return 0;
  // (any function that grows with c and ends at total would do: no 64-bit division)
  const double each = (double)total / ctas;
  const long long u0 = (long long)(each * c), u1 = c + 1 == ctas ? total : (long long)(each * (c + 1));
  if (u0 == u1) return 0;
  long long done = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += THREADS) {
    if (a.n_seqs > THREADS) before = add_up(b0);
    if (u0 >= done + before && u0 < done + before + mine) {
      const Seq s(a, b0 + threadIdx.x);
      long long r = u0 - done - before;
      Place p;
      p.b = b0 + threadIdx.x;
      const long long each = s.per_block(a);
      p.block = r >> 32 | each >> 32 ? (int)(r / each) : (int)((unsigned int)r / (unsigned int)each);
      r -= p.block * each;
      int lo = 0, hi = s.tiles;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.upto(a, mid) <= r) lo = mid;
        else hi = mid;
      }
      p.tile = lo, p.unit = (int)(r - s.upto(a, lo));
      place_s = p;
    }
    done += all;
  }
  __syncthreads();
  *at = place_s;
  return u1 - u0;
}

// The rows of a segment: tokens [j0, j0 + tokens) of the sequence, and of each
// `heads` query heads from `head` on; row r is token j0 + r / heads.
struct Rows {
  int row0, j0, tokens, heads, head;  // row0: the sequence's first row of q
  int n;                              // tokens * heads
  int all;                            // tokens of the sequence
  __device__ __forceinline__ int token(int r) const { return tokens == 1 ? 0 : r / heads; }  // (no division for one)
  __device__ __forceinline__ int64_t q_row(int r) const { return row0 + j0 + token(r); }
  __device__ __forceinline__ int q_head(int r) const { return head + r - token(r) * heads; }
};
// kv: the cached head.
__device__ __forceinline__ Rows rows_of(const AttnArgs &a, const Seq &s, int kv, int part, int tile) {
  Rows r;
  r.row0 = s.row0, r.j0 = tile * a.tq;
  r.tokens = s.rows - r.j0 < a.tq ? s.rows - r.j0 : a.tq;
  const int h0 = part * a.gh, h1 = h0 + a.gh < a.grp ? h0 + a.gh : a.grp;
  r.heads = h1 - h0, r.head = kv * a.grp + h0;
  r.n = r.tokens * r.heads, r.all = s.rows;
  return r;
}

__device__ __forceinline__ int page_of(const AttnArgs &a, int t) {
  return (int)((unsigned long long)(unsigned int)t * a.page_mul >> a.page_shift);
}

// Slot of token t of sequence b, -1 (reported) where the table or the cache ends.
__device__ __forceinline__ int64_t slot_of(const AttnArgs &a, int b, int t) {
  const int pg = page_of(a, t);
  int64_t page = -1;
  if (pg < a.max_pages) page = a.pages[(int64_t)b * a.max_pages + pg];
  if (page >= 0 && page < a.k.n_pages) return page * a.k.page_size + (t - pg * a.k.page_size);
  atomicOr(a.err, kErrPage);
  return -1;
}

// x H over blocks of had (0: nothing) for a row of D values in shared memory that
// one warp owns, times unit.
__device__ __forceinline__ void warp_rotate(float *x, int D, int had, float unit) {
  const int lane = threadIdx.x & 31;
  if (had < 2) return;
  for (int h = 1; h < had; h *= 2) {
    __syncwarp();
    for (int p = lane; p < D / 2; p += 32) {
      const int i = (p & ~(h - 1)) * 2 + (p & (h - 1));
      const float u = x[i], v = x[i + h];
      x[i] = u + v, x[i + h] = u - v;
    }
  }
  __syncwarp();
  for (int d = lane; d < D; d += 32) x[d] *= unit;
  __syncwarp();
}

// Writes a finished row: x [D] (shared, owned by the warp) is the sum of p v in
// the cache's rotated frame, l the sum of p, m the maximum (base 2).
__device__ __forceinline__ void warp_finish(const AttnArgs &a, float *x, float m, float l, int64_t row, int head) {
  const int lane = threadIdx.x & 31, D = a.v.head_dim;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int d = lane; d < D; d += 32) x[d] *= inv;
  warp_rotate(x, D, a.v.had_block, a.unit_v);
  __syncwarp();
  const int64_t at = (row * a.q_heads + head) * D;
  if (a.f32) {
    for (int d = lane; d < D; d += 32) static_cast<float *>(a.out)[at + d] = x[d];
  } else {
    for (int d = lane * 2; d < D; d += 64)
      *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + at + d) = pack_bf16x2(x[d], x[d + 1]);
  }
  if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// A row's query in the cache's rotated frame, times scale log2(e), in x [D].
__device__ __forceinline__ void warp_query(const AttnArgs &a, float *x, int64_t row, int head) {
  const int lane = threadIdx.x & 31, D = a.k.head_dim;
  const int64_t at = row * a.q_stride + (int64_t)head * D;
  for (int d = lane; d < D; d += 32)
    x[d] = a.f32 ? static_cast<const float *>(a.q)[at + d] : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at + d]);
  warp_rotate(x, D, a.k.had_block, a.unit_k);
  __syncwarp();
  for (int d = lane; d < D; d += 32) x[d] *= a.scale2;
  __syncwarp();
}

// A piece in the workspace: row r of slot s holds m, l and D values. Slot 2 c is
// the piece with which CTA c goes on with a tile that another began, slot 2 c + 1
// the one it began and left.
// (part_desc: sequence, block, tile and these; 0: none, as of a CTA without units)
enum { kPieceThere = 1, kPieceEnds = 2, kPieceCoarse = 4 };  // coarse (slot 2 c, there or not): of any of the CTA's tiles
__device__ __forceinline__ float *piece_stats(const AttnArgs &a, int slot, int r) {
  return a.part_stats + ((int64_t)slot * a.part_rows + r) * 2;
}
__device__ __forceinline__ float *piece_values(const AttnArgs &a, int slot, int r) {
  return a.part + ((int64_t)slot * a.part_rows + r) * a.v.head_dim;
}

}  // namespace attn
}  // namespace qwha
