// A paged cache of quantized rows (keys or values of attention heads): writing
// rows into its slots and reading sequences back.
//
// A slot holds one token; each of its heads is a row of head_dim codes in the
// base weight's format, W = scales * (q - zeros) per group. Optionally the row
// is rotated by the orthonormal Hadamard matrix first (blocks of had_block), so
// that a channel with large values is spread over the block and the groups'
// steps shrink; reading rotates back (H is its own inverse).
//
// The quantizer is defined bit for bit, so that a cache written here equals one
// written by any other statement of the formulas (bf16 rows in fp32, fp32 rows
// in fp64: a code next to a border decides a whole step, far more than the
// row's own type carries; no contraction):
//   v   = butterflies 1, 2, 4, ..., had_block/2, then * (1/sqrt(had_block))
//   lo  = min(0, min v), hi = max(0, max v)                  per group
//   s   = fp32((hi - lo) * (1/qmax)), qmax = 2^bits - 1; s < 2^-126 counts as 1
//   inv = 1 / s, half = 0.5 + 2^-12
//   z   = min(floor(-lo * inv + half), qmax)
//   q   = clamp(floor(v * inv + (z + half)), 0, qmax)
// bf16 values lie exactly half-way between two codes in one group of a few
// (qmax = 15 divides many ranges); with the border 2^-12 of a step below the
// half those go up whatever the last bit of inv is.
// A group whose s is not finite (an infinity, a NaN, an overflow) is stored as
// s = NaN, codes and zero point 0: it reads back as NaN and harms no other group.

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace qwha {
namespace {

constexpr int kCacheThreads = 256;

// Arithmetic of the quantizer for rows of type T.
template <typename T>
struct wide;
template <>
struct wide<__nv_bfloat16> {
  using type = float;
};
template <>
struct wide<float> {
  using type = double;
};

__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ double mul(double a, double b) { return __dmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ double add(double a, double b) { return __dadd_rn(a, b); }

template <int H, typename A>
__device__ __forceinline__ void stage8(A *v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(i & H)) {
      const A a = v[i], b = v[i + H];
      v[i] = a + b;
      v[i + H] = a - b;
    }
}

// The Hadamard blocks of a row spread over lanes, eight consecutive elements
// each; stages 1, 2, 4 inside a lane, the others between lanes.
template <typename A>
__device__ __forceinline__ void rotate8(A *v, int had_block, A scale, int lane) {
  if (had_block < 2) return;
  stage8<1>(v);
  if (had_block >= 4) stage8<2>(v);
  if (had_block >= 8) stage8<4>(v);
  for (int o = 1; o * 8 < had_block; o *= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const A p = __shfl_xor_sync(~0u, v[i], o);
      v[i] = upper ? p - v[i] : v[i] + p;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mul(v[i], scale);
}

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ double min_nan(double a, double b) { return a < b || a != a ? a : b; }
__device__ __forceinline__ double max_nan(double a, double b) { return a > b || a != a ? a : b; }

// min and max over the `gl` neighbouring lanes of a group.
template <typename A>
__device__ __forceinline__ void group_range(A &lo, A &hi, int gl, int lane) {
  if ((gl & (gl - 1)) == 0) {
    for (int o = 1; o < gl; o *= 2) {
      lo = min_nan(lo, __shfl_xor_sync(~0u, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(~0u, hi, o));
    }
    return;
  }
  const A l0 = lo, h0 = hi;
  const int at = lane % gl;  // the caller numbers lanes from the row's first
  for (int d = 1; d < gl; ++d) {
    const int turn = at + d < gl ? d : d - gl;
    lo = min_nan(lo, __shfl_sync(~0u, l0, (int)((threadIdx.x & 31) + turn)));
    hi = max_nan(hi, __shfl_sync(~0u, h0, (int)((threadIdx.x & 31) + turn)));
  }
}

__device__ __forceinline__ void store_run(uint8_t *p, const uint32_t *q, int bits) {
  if (bits == 8) {
    uint2 w;
    w.x = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
    w.y = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
    *reinterpret_cast<uint2 *>(p) = w;
    return;
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= q[i] << (bits * i);
  if (bits == 4) *reinterpret_cast<uint32_t *>(p) = w;
  else if (bits == 2) *reinterpret_cast<uint16_t *>(p) = (uint16_t)w;
  else p[0] = (uint8_t)w, p[1] = (uint8_t)(w >> 8), p[2] = (uint8_t)(w >> 16);
}

__device__ __forceinline__ void load_run(const uint8_t *p, float *q, int bits) {
  uint32_t w, hi = 0;
  if (bits == 8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w = v.x, hi = v.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (float)((w >> (8 * i)) & 255u), q[i + 4] = (float)((hi >> (8 * i)) & 255u);
    return;
  }
  if (bits == 4) w = *reinterpret_cast<const uint32_t *>(p);
  else if (bits == 2) w = *reinterpret_cast<const uint16_t *>(p);
  else w = (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
  const uint32_t mask = (1u << bits) - 1u;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = (float)((w >> (bits * i)) & mask);
}

constexpr int kTileTokens = 64;  // tokens of a CTA's tile, at most

// The (token, head) pairs of a tile, `step` apart: no division per pair.
struct Walk {
  int token, head, heads, step_tokens, step_heads;
  __device__ __forceinline__ Walk(int first, int step, int heads_) : heads(heads_) {
    token = first / heads, head = first - token * heads;
    step_tokens = step / heads, step_heads = step - step_tokens * heads;
  }
  __device__ __forceinline__ void next() {
    token += step_tokens, head += step_heads;
    if (head >= heads) head -= heads, ++token;
  }
};

// Slot of written row i: -1 where the row is skipped.
__device__ __forceinline__ int64_t write_slot(const qwha_cache &a, const int64_t *slots, int64_t i, unsigned int *err) {
  const int64_t s = slots[i];
  if (s >= -1 && s < a.n_pages * a.page_size) return s;
  atomicOr(err, kErrSlot);
  return -1;
}

// Slot of output row i, which belongs to the sequence b with row_start[b] <= i <
// row_start[b + 1] and is its token first[b] + i - row_start[b]; -1 where the
// page table or the cache ends.
__device__ __forceinline__ int64_t read_slot(const qwha_cache &a, const ReadArgs &r, int64_t i, unsigned int *err) {
  int lo = 0, hi = r.n_seqs;  // row_start[lo] <= i < row_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (r.row_start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int64_t pos = i - r.row_start[lo] + (r.first ? r.first[lo] : 0), pg = pos / a.page_size;
  int64_t page = -1;
  if (pos >= 0 && pg < r.max_pages) page = r.pages[(int64_t)lo * r.max_pages + pg];
  if (page >= 0 && page < a.n_pages) return page * a.page_size + (pos - pg * a.page_size);
  atomicOr(err, kErrPage);
  return -1;
}

// Scale, zero point and the factor of the codes of a group with range [lo, hi].
template <typename A>
struct Step {
  float s;
  A inv, z;
  bool bad;
  __device__ __forceinline__ Step(A lo, A hi, A qmax, A step, A half) {
    s = (float)mul(add(hi, -lo), step);
    bad = !(s <= 3.402823466e38f);
    if (s < 1.1754943508e-38f) s = 1.f;
    inv = (A)1 / (A)s;
    z = floor(add(mul(-lo, inv), half));
    z = z < qmax ? z : qmax;
  }
};

// Any row of up to 256 elements, eight to a lane: 1 << ll lanes hold a row.
template <typename T>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CachePair c, int ll,
                                                                    const int64_t *__restrict__ slots, int64_t n,
                                                                    int tile, unsigned int *err) {
  using A = typename wide<T>::type;
  __shared__ int64_t slot_s[kTileTokens];
  const qwha_cache &a = c.cache[blockIdx.y];
  const T *rows = static_cast<const T *>(c.rows[blockIdx.y]);
  const int lane = threadIdx.x & ((1 << ll) - 1);
  const bool has = lane * 8 < a.head_dim;
  const int gl = a.group / 8, ng = a.head_dim / a.group, group_at = lane / gl;
  const A qmax = (A)((1 << a.bits) - 1), step = (A)1 / qmax, unit = (A)c.unit[blockIdx.y], half = (A)(0.5 + 1.0 / 4096);
  for (int64_t t0 = (int64_t)blockIdx.x * tile; t0 < n; t0 += (int64_t)gridDim.x * tile) {
    const int tokens = n - t0 < tile ? (int)(n - t0) : tile;
    __syncthreads();  // the last tile's slots are read
    if (threadIdx.x < tokens) slot_s[threadIdx.x] = write_slot(a, slots, t0 + threadIdx.x, err);
    __syncthreads();
    Walk w(threadIdx.x >> ll, kCacheThreads >> ll, a.heads);
    // whole warps stay together: their pairs differ by less than the tile's last ones
    for (int base = 0; base < tokens * a.heads; base += kCacheThreads >> ll, w.next()) {
      const int64_t slot = w.token < tokens ? slot_s[w.token] : -1;
      const bool live = slot >= 0 && has;
      A v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0;
      if (live) {
        const T *src = rows + ((t0 + w.token) * a.heads + w.head) * a.head_dim + lane * 8;
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; u += io<T>::kVec) io<T>::unpack(*reinterpret_cast<const uint4 *>(src + u), f + u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
      }
      rotate8(v, a.had_block, unit, lane);
      A lo = 0, hi = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) lo = min_nan(lo, v[i]), hi = max_nan(hi, v[i]);
      group_range(lo, hi, gl, lane);
      const Step<A> g(lo, hi, qmax, step, half);
      uint32_t q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const A r = add(mul(v[i], g.inv), g.z + half);
        q[i] = g.bad || !(r > (A)0) ? 0u : r < qmax ? (uint32_t)r : (uint32_t)qmax;
      }
      if (live) {
        const int64_t row = slot * a.heads + w.head;
        store_run(a.codes + row * (a.head_dim / 8 * a.bits) + lane * a.bits, q, a.bits);
        if (lane == group_at * gl) {
          a.scales[row * ng + group_at] = g.bad ? __int_as_float(0x7fc00000) : g.s;
          a.zeros[row * ng + group_at] = g.bad ? 0 : (uint8_t)g.z;
        }
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const CachePair c, int ll, const ReadArgs r, int64_t n, int tile, unsigned int *err) {
  __shared__ int64_t slot_s[kTileTokens];
  const qwha_cache &a = c.cache[blockIdx.y];
  T *rows = static_cast<T *>(const_cast<void *>(c.rows[blockIdx.y]));
  const int lane = threadIdx.x & ((1 << ll) - 1);
  const bool has = lane * 8 < a.head_dim;
  const int ng = a.head_dim / a.group, group_at = lane * 8 / a.group;
  const float unit = (float)c.unit[blockIdx.y];
  const int64_t end = r.row_start[r.n_seqs], rows_n = end < n ? end : n;
  for (int64_t t0 = (int64_t)blockIdx.x * tile; t0 < rows_n; t0 += (int64_t)gridDim.x * tile) {
    const int tokens = rows_n - t0 < tile ? (int)(rows_n - t0) : tile;
    __syncthreads();
    if (threadIdx.x < tokens) slot_s[threadIdx.x] = read_slot(a, r, t0 + threadIdx.x, err);
    __syncthreads();
    Walk w(threadIdx.x >> ll, kCacheThreads >> ll, a.heads);
    for (int base = 0; base < tokens * a.heads; base += kCacheThreads >> ll, w.next()) {
      const int64_t slot = w.token < tokens ? slot_s[w.token] : -1;
      const bool live = slot >= 0 && has;
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = 0.f;
      if (live) {
        const int64_t row = slot * a.heads + w.head;
        load_run(a.codes + row * (a.head_dim / 8 * a.bits) + lane * a.bits, v, a.bits);
        const float s = a.scales[row * ng + group_at], z = (float)a.zeros[row * ng + group_at];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __fmul_rn(s, v[u] - z);
      }
      rotate8(v, a.had_block, unit, lane);
      if (live) {
        T *dst = rows + ((t0 + w.token) * a.heads + w.head) * a.head_dim + lane * 8;
#pragma unroll
        for (int u = 0; u < 8; u += io<T>::kVec) *reinterpret_cast<uint4 *>(dst + u) = io<T>::pack(v + u);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Reading on tensor cores. q - zero is an integer of at most 8 bits and a sign,
// so H (q - zero) is exact in matrix instructions of f16 with fp32 sums, and one
// multiplication by scale / sqrt(n) is left per value. A unit is 128 elements in
// a row of a token's heads; the bits e0..e6 of an element's place are split over
// the operands of two products,
//   D[m][n]  = sum_k A[m][k] (q - zero)[k][n],  k = (e2, e3, e4, e0), n = (e1, e5, e6)
//   E[m][n'] = sum_n D[m][n] B[n][n'],
// A and B the Hadamard matrices of those bits (the identity in bits at or above
// had_block), D in the layout of the second product's operand as it stands. A
// lane reads the eight codes that differ in e0..e2, takes the four with its own
// e1, and ends with four neighbours of the row. Bits e5 and e6 that lie between
// two groups of a block are left to fp32 butterflies after the scales.
// A sum of sixteen in D is at most 16 max(zero, 2^bits - 1): exact in f16 up to
// 2048, so with zero points up to 128 and 2 to 4 bits it is one f16. For 8 bits,
// and in a CTA that has met a larger zero point (any byte is valid), it is split
// into two f16 (D - f16(D) is at most 1).
//
// Memory bounds this: 2 bytes written and 0.53 read a value of 4 bits. A CTA
// fetches 256 units of a tile with all its threads and computes from shared
// memory; eight CTAs on an SM overlap each other's phases. Two caches, 8 heads
// of 128, 4 bits, 192526 tokens, bf16: 186 us, 82 % of the copy rate. Loads
// straight to the registers of the lane that uses them, four units in flight a
// warp, took 285 us (waiting for memory), butterflies in registers and between
// lanes 309 us (issue slots).

__device__ __forceinline__ void mma_16816(float *d, const uint32_t *a, const uint32_t *b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
__device__ __forceinline__ void mma_1688(float *d, uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void cp_async16(void *smem, const void *p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(p)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Entry (i, j) of the Kronecker product of [1 1; 1 -1] in the bits of `on` and
// the identity in the others, in f16.
__device__ __forceinline__ uint32_t sign_entry(int i, int j, int on) {
  return (i ^ j) & ~on ? 0u : __popc(i & j & on) & 1 ? 0xbc00u : 0x3c00u;
}

// The lane's eight codes as the register (or two) that hold them.
template <int BITS>
__device__ __forceinline__ uint2 load_codes(const uint8_t *unit, int word) {
  if constexpr (BITS == 8) return *reinterpret_cast<const uint2 *>(unit + 8 * word);
  if constexpr (BITS == 4) return make_uint2(*reinterpret_cast<const uint32_t *>(unit + 4 * word), 0);
  if constexpr (BITS == 2) return make_uint2(*reinterpret_cast<const uint16_t *>(unit + 2 * word), 0);
  const uint32_t *w = reinterpret_cast<const uint32_t *>(unit);  // bytes 3 word .. 3 word + 2
  return make_uint2(w[3 * word / 4], w[(3 * word + 2) / 4]);
}
// b[i]: 1024 + q of the codes e0 = i, e1, e2 = 0 and 1, two f16.
template <int BITS>
__device__ __forceinline__ void spread_codes(uint2 c, int word, int e1, uint32_t *b) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = __byte_perm(c.x, c.y, e1 ? 0x0602 + 0x101 * i : 0x0400 + 0x101 * i) & 0x00ff00ffu;
  } else {
    uint32_t w = c.x;
    if constexpr (BITS == 2) w = __byte_perm(w, 0, 0x4140);
    if constexpr (BITS == 3) {
      w = __funnelshift_r(c.x, c.y, 8 * (3 * word % 4));
      w = (w & 0xfffu) | (w << 4 & 0x0fff0000u);
    }
    w >>= 2 * BITS * e1;
    b[0] = w, b[1] = w >> BITS;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (b[i] & (0x00010001u * ((1u << BITS) - 1u))) | 0x64006400u;
}

constexpr int kTileUnits = 256;
constexpr uint32_t kNoSlot = ~0u;  // in place of a zero point

// Five CTAs to an SM where the loop's 48 registers allow (with the rare split in the kernel the compiler takes 59 and
// leaves room for four: 193 instead of 186 us for the case above).
template <typename T, int BITS>
__global__ void __launch_bounds__(kCacheThreads, BITS % 2 || BITS == 8 ? 4 : 5)
    cache_read_mma_kernel(const CachePair c, const ReadArgs r, int64_t n, int tile, unsigned int *err) {
  constexpr int kWarps = kCacheThreads / 32;
  __shared__ int64_t slot_s[kTileTokens];
  __shared__ __align__(16) uint8_t code_s[kTileUnits * 16 * BITS];
  __shared__ float scale_s[kTileUnits * 4];
  __shared__ uint32_t zero_s[kTileUnits * 4];  // 1024 + zero, two f16
  __shared__ int far_s;  // a zero point above 128 was met: the CTA splits from there on
  if (threadIdx.x == 0) far_s = 0;
  const qwha_cache &a = c.cache[blockIdx.y];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
  const int lg = 31 - __clz(a.group), had = a.had_block > 1 ? a.had_block : 1;
  const int units = a.heads * a.head_dim / 128;  // of a token
  const int word = t + 4 * (g >> 1), e1 = g & 1;
  // the bits of A's and B's indices that are in the block, and for B in the group
  const int on_k = (had > 4) | (had > 8) << 1 | (had > 16) << 2 | (had > 1) << 3;
  const int on_n = (had > 2) | (had > 32 && lg > 5) << 1 | (had > 64 && lg > 6) << 2;
  const bool cross5 = had > 32 && lg <= 5, cross6 = had > 64 && lg <= 6;
  uint32_t ha[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = g + 8 * (i & 1), k = 2 * t + 8 * (i >> 1);
    ha[i] = sign_entry(m, k, on_k) | sign_entry(m, k + 1, on_k) << 16;
  }
  const uint32_t hb = sign_entry(2 * t, g, on_n) | sign_entry(2 * t + 1, g, on_n) << 16;
  const float scale = (float)c.unit[blockIdx.y];
  const int up = lg < 7 ? lg - 5 : 2;  // the lane's group of a unit is its (e5, e6) >> up
  const int pieces = units * BITS, groups = units * 128 >> lg;  // 16-byte pieces of codes and groups of a token
  T *rows = static_cast<T *>(const_cast<void *>(c.rows[blockIdx.y])) + 4 * g + 32 * t;
  const int64_t end = r.row_start[r.n_seqs], rows_n = end < n ? end : n;
  for (int64_t t0 = (int64_t)blockIdx.x * tile; t0 < rows_n; t0 += (int64_t)gridDim.x * tile) {
    const int tokens = rows_n - t0 < tile ? (int)(rows_n - t0) : tile;
    __syncthreads();
    if (threadIdx.x < tokens) slot_s[threadIdx.x] = read_slot(a, r, t0 + threadIdx.x, err);
    const int total = tokens * units;
    for (int u0 = 0; u0 < total; u0 += kTileUnits) {
      __syncthreads();
      const int here = total - u0 < kTileUnits ? total - u0 : kTileUnits;
      for (int i = threadIdx.x; i < here * BITS; i += kCacheThreads) {
        const int at = u0 * BITS + i, token = at / pieces;
        const int64_t slot = slot_s[token];
        if (slot >= 0) cp_async16(code_s + 16 * i, a.codes + (slot * pieces + (at - token * pieces)) * 16);
      }
      const int g0 = u0 * 128 >> lg;
      for (int i = threadIdx.x; i < here * 128 >> lg; i += kCacheThreads) {
        const int token = (g0 + i) / groups;
        const int64_t slot = slot_s[token], group = slot * groups + (g0 + i - token * groups);
        if (slot >= 0) {
          const uint32_t zero = a.zeros[group];
          if (BITS != 8 && zero > 128) far_s = 1;
          scale_s[i] = a.scales[group] * scale, zero_s[i] = (zero | 0x6400u) * 0x10001u;
        } else {
          zero_s[i] = kNoSlot;
        }
      }
      cp_async_wait_all();
      __syncthreads();
      auto compute = [&](auto split) {
        constexpr bool kSplit = decltype(split)::value;
        constexpr int kUnroll = kSplit && BITS != 8 ? 1 : 4;  // the rare one is short
        T *out = rows + (t0 * units + u0 + warp) * 128;
#pragma unroll kUnroll
        for (int u = warp; u < here; u += kWarps, out += kWarps * 128) {
          const int group = u * 128 >> lg;
          const uint32_t zz = zero_s[group + (g >> 1 >> up)];
          const float f = scale_s[group + (t >> up)];
          const bool live = zz != kNoSlot;
          const uint2 code = load_codes<BITS>(code_s + u * (16 * BITS), word);
          uint32_t b[2];
          spread_codes<BITS>(code, word, e1, b);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 d = __hsub2(reinterpret_cast<const __half2 &>(b[i]), reinterpret_cast<const __half2 &>(zz));
            b[i] = reinterpret_cast<const uint32_t &>(d);
          }
          float d[4], e[4];
          mma_16816(d, ha, b);
          const uint32_t d0 = f16x2(d[0], d[1]), d1 = f16x2(d[2], d[3]);
          mma_1688(e, d0, d1, hb);
          if constexpr (kSplit) {
            const float2 f0 = __half22float2(reinterpret_cast<const __half2 &>(d0)),
                         f1 = __half22float2(reinterpret_cast<const __half2 &>(d1));
            float lo[4];
            mma_1688(lo, f16x2(d[0] - f0.x, d[1] - f0.y), f16x2(d[2] - f1.x, d[3] - f1.y), hb);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] += lo[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] *= f;
          if (cross5)
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = fmaf(e[i], t & 1 ? -1.f : 1.f, __shfl_xor_sync(~0u, e[i], 1));
          if (cross6)
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = fmaf(e[i], t & 2 ? -1.f : 1.f, __shfl_xor_sync(~0u, e[i], 2));
          // e0 is the bit of m above g, e1 the lower bit of n'
          if (!live) continue;
          if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(out) = make_float4(e[0], e[2], e[1], e[3]);
          else *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(e[0], e[2]), pack_bf16x2(e[1], e[3]));
        }
      };
      if (BITS == 8 || far_s) compute(std::true_type());
      else compute(std::integral_constant<bool, BITS == 8>());
    }
  }
}

// ---------------------------------------------------------------------------
// Writing bf16 rows in units of 128 elements. The fp32 butterflies and the
// quantizer bound this, not memory: at the copy rate 2.5 bytes a value leave
// about 12 instructions, so every step counts. Eight lanes hold two units, one
// in each half of packed fp32 pairs. A lane begins with sixteen neighbours
// (stages 1, 2, 4, 8), the units turn in shared memory, and it ends with the
// elements l + 8 j (stages 16, 32, 64; l its place among the eight lanes): no
// stage crosses lanes. Ranges of the groups are reduced so that each lane ends
// with one group, computes its step and hands it round. Codes become nibbles
// (8 bits: bytes) by one shifted addition each, and an eight by eight transpose
// in registers brings each lane sixteen neighbours to store.
//
// 32768 tokens into two caches, 8 heads of 128, 4 bits, groups of 64: 76 us at
// 3.1 instructions a clock (the bytes alone: 26 us). With the read-back of the
// same rows 117 us; 282 us with eight elements a lane and butterflies between
// lanes in both kernels, 154 us with sixteen a lane in this one.

using f2 = unsigned long long;  // two fp32 values
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
  f2 d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The products one by one: the assembler contracts a packed product and a packed
// sum, .rn or not, into one rounding, and the quantizer has two.
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(__fmul_rn(a0, b0), __fmul_rn(a1, b1));
}

// Butterflies between v[i] and v[i + H].
template <int H>
__device__ __forceinline__ void stage16(f2 *v) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (!(i & H)) {
      const f2 a = v[i], b = v[i + H];
      v[i] = add2(a, b), v[i + H] = sub2(a, b);
    }
}

// Eight lanes, R's piece k of lane l becomes piece l of lane k.
__device__ __forceinline__ uint32_t turn_halves(uint32_t r, int l, int d) {
  return __byte_perm(r, __shfl_xor_sync(~0u, r, d), l & d ? 0x3276 : 0x5410);
}
__device__ __forceinline__ uint32_t turn_bytes(uint32_t r, int l, int d) {
  return __byte_perm(r, __shfl_xor_sync(~0u, r, d), l & d ? 0x3715 : 0x6240);
}
__device__ __forceinline__ uint32_t turn_nibbles(uint32_t r, int l) {
  const uint32_t keep = l & 1 ? 0xf0f0f0f0u : 0x0f0f0f0fu, x = __shfl_xor_sync(~0u, r, 1);
  return (r & keep) | (__funnelshift_l(x, x, l & 1 ? 28 : 4) & ~keep);
}

// Eight nibbles of two or three bits, closed up.
template <int BITS>
__device__ __forceinline__ uint32_t close_up(uint32_t w) {
  if constexpr (BITS == 2) {
    w = (w & 0x03030303u) | (w >> 2 & 0x0c0c0c0cu);
    w = (w & 0x000f000fu) | (w >> 4 & 0x00f000f0u);
    return (w & 0xffu) | (w >> 8 & 0xff00u);
  } else {
    w = (w & 0x07070707u) | (w >> 1 & 0x38383838u);
    w = (w & 0x003f003fu) | (w >> 2 & 0x0fc00fc0u);
    return (w & 0xfffu) | (w >> 4 & 0xfff000u);
  }
}

// Stores a unit's codes q[j] = 2^23 + code of element l + 8 j (fp32 bits): the
// lane's share are elements 16 l .. 16 l + 15, all zero where `bad`.
template <int BITS>
__device__ __forceinline__ void store_unit(uint8_t *unit, const uint32_t *q, int l, bool live, bool bad) {
  if constexpr (BITS == 8) {
    uint32_t r[4];  // bytes: even j below and above 8, odd j below and above 8
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = 0u - 0x4b000000u;
#pragma unroll
      for (int k = 0; k < 4; ++k) r[i] += q[8 * (i & 1) + 2 * k + (i >> 1)] << (8 * k);
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t x = __shfl_xor_sync(~0u, l & 4 ? r[i] : r[i + 1], 4);
      if (l & 4) r[i] = x;
      else r[i + 1] = x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = turn_bytes(turn_halves(r[i], l, 2), l, 1);
    if (!live) return;
    *reinterpret_cast<uint4 *>(unit + 16 * l) = bad ? make_uint4(0, 0, 0, 0) : make_uint4(r[0], r[1], r[2], r[3]);
  } else {
    uint32_t r[2];  // nibbles: even j, odd j
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[i] = 0u - 0xfb000000u;  // what the exponents of the first two leave
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i] += q[2 * k + i] << (4 * k);
      r[i] = turn_nibbles(turn_bytes(turn_halves(r[i], l, 4), l, 2), l);
      if (bad) r[i] = 0;
    }
    if (!live) return;
    if constexpr (BITS == 4) {
      *reinterpret_cast<uint2 *>(unit + 8 * l) = make_uint2(r[0], r[1]);
    } else if constexpr (BITS == 2) {
      *reinterpret_cast<uint32_t *>(unit + 4 * l) = close_up<2>(r[0]) | close_up<2>(r[1]) << 16;
    } else {
      const uint32_t a = close_up<3>(r[0]), b = close_up<3>(r[1]);
      uint16_t *p = reinterpret_cast<uint16_t *>(unit + 6 * l);
      p[0] = (uint16_t)a, p[1] = (uint16_t)(a >> 16 | b << 8), p[2] = (uint16_t)(b >> 8);
    }
  }
}

// NG groups in a unit.
template <int BITS, int NG>
__global__ void __launch_bounds__(kCacheThreads)
    cache_write_unit_kernel(const CachePair c, const int64_t *__restrict__ slots, int64_t n, int tile,
                            unsigned int *err) {
  constexpr int kWarps = kCacheThreads / 32, kTurn = 128 + 16 + 8;  // pairs of two units, padded: no bank twice
  constexpr int C = 2 * NG, kShift = NG == 1 ? 2 : NG == 2 ? 1 : 0;  // groups of two units; their lanes: c << kShift
  constexpr float qmax = (float)((1 << BITS) - 1);
  __shared__ int64_t slot_s[kTileTokens];
  __shared__ __align__(16) f2 turn_s[kWarps][4][kTurn];
  const qwha_cache &a = c.cache[blockIdx.y];
  const __nv_bfloat16 *rows = static_cast<const __nv_bfloat16 *>(c.rows[blockIdx.y]);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
  const int units = a.heads * a.head_dim / 128, had = a.had_block;
  const float unit = (float)c.unit[blockIdx.y], step = 1.0f / qmax, half = (float)(0.5 + 1.0 / 4096);
  f2 *turn = turn_s[warp][lane >> 3];
  for (int64_t t0 = (int64_t)blockIdx.x * tile; t0 < n; t0 += (int64_t)gridDim.x * tile) {
    const int tokens = n - t0 < tile ? (int)(n - t0) : tile;
    __syncthreads();  // the last tile's slots are read
    if (threadIdx.x < tokens) slot_s[threadIdx.x] = write_slot(a, slots, t0 + threadIdx.x, err);
    __syncthreads();
    const int total = tokens * units;
    Walk w(8 * warp + 2 * (lane >> 3), 8 * kWarps, units);
    for (int at = 8 * warp; at < total; at += 8 * kWarps, w.next()) {
      const int p = at + 2 * (lane >> 3);  // and p + 1
      int64_t to[2];                       // units of the cache, -1: none
      uint4 in[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool wrap = w.head + u == units;
        to[u] = -1;
        in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
        if (p + u < total) {
          const __nv_bfloat16 *src = rows + (t0 * units + p + u) * 128 + 16 * l;
          in[u][0] = ld_stream(src), in[u][1] = ld_stream(src + 8);
          const int64_t slot = slot_s[w.token + wrap];
          if (slot >= 0) to[u] = slot * units + (wrap ? 0 : w.head + u);
        }
      }
      f2 v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 &qa = in[0][i / 4], &qb = in[1][i / 4];
        const uint32_t x = i % 4 == 0 ? qa.x : i % 4 == 1 ? qa.y : i % 4 == 2 ? qa.z : qa.w;
        const uint32_t y = i % 4 == 0 ? qb.x : i % 4 == 1 ? qb.y : i % 4 == 2 ? qb.z : qb.w;
        v[2 * i] = pack2(bf16_lo(x), bf16_lo(y)), v[2 * i + 1] = pack2(bf16_hi(x), bf16_hi(y));
      }
      if (had >= 2) stage16<1>(v);
      if (had >= 4) stage16<2>(v);
      if (had >= 8) stage16<4>(v);
      if (had >= 16) stage16<8>(v);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        *reinterpret_cast<ulonglong2 *>(turn + 18 * l + i) = make_ulonglong2(v[i], v[i + 1]);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = turn[l + 8 * j + 2 * (j / 2)];
      if (had >= 32) stage16<2>(v);
      if (had >= 64) stage16<4>(v);
      if (had >= 128) stage16<8>(v);
      float lo[C], hi[C];
#pragma unroll
      for (int i = 0; i < C; ++i) lo[i] = hi[i] = 0.f;
      const f2 u2 = pack2(unit, unit);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int q = j / (16 / NG);
        v[j] = mul2(v[j], u2);
        float x, y;
        unpack2(v[j], x, y);
        lo[q] = min_nan(lo[q], x), hi[q] = max_nan(hi[q], x);
        lo[NG + q] = min_nan(lo[NG + q], y), hi[NG + q] = max_nan(hi[NG + q], y);
      }
      // each round halves the groups a lane holds; with one left it adds lanes
#pragma unroll
      for (int d = 4, m = C; d; d /= 2) {
        const bool upper = l & d;
        if (m > 1) {
          m /= 2;
#pragma unroll
          for (int i = 0; i < m; ++i) {
            lo[i] = min_nan(upper ? lo[i + m] : lo[i], __shfl_xor_sync(~0u, upper ? lo[i] : lo[i + m], d));
            hi[i] = max_nan(upper ? hi[i + m] : hi[i], __shfl_xor_sync(~0u, upper ? hi[i] : hi[i + m], d));
          }
        } else {
          lo[0] = min_nan(lo[0], __shfl_xor_sync(~0u, lo[0], d));
          hi[0] = max_nan(hi[0], __shfl_xor_sync(~0u, hi[0], d));
        }
      }
      Step<float> g(lo[0], hi[0], qmax, step, half);
      const unsigned bad = __ballot_sync(~0u, g.bad) >> (lane & 24);  // of these eight lanes
      if (g.bad) g.inv = g.z = 0.f;
      {
        const int mine = l >> kShift;
        const int64_t unit_at = mine < NG ? to[0] : to[1];
        if (unit_at >= 0 && (l & ((1 << kShift) - 1)) == 0) {
          const int64_t at_group = unit_at * NG + mine % NG;
          a.scales[at_group] = g.bad ? __int_as_float(0x7fc00000) : g.s;
          a.zeros[at_group] = (uint8_t)g.z;
        }
      }
      uint32_t code[2][16];
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        f2 inv2, up2;
        {
          const float i0 = __shfl_sync(~0u, g.inv, q << kShift, 8), i1 = __shfl_sync(~0u, g.inv, (q + NG) << kShift, 8);
          const float z0 = __shfl_sync(~0u, g.z, q << kShift, 8), z1 = __shfl_sync(~0u, g.z, (q + NG) << kShift, 8);
          inv2 = pack2(i0, i1), up2 = pack2(z0 + half, z1 + half);
        }
#pragma unroll
        for (int j = q * (16 / NG); j < (q + 1) * (16 / NG); ++j) {
          // Not below 0: -lo * inv + half < z + 1 up to 2^-16, and half is 2^-12 above
          // one half, so lo * inv + z + half > 0. Rounding towards zero into 2^23 + code.
          float x, y;
          unpack2(add2(mul2(v[j], inv2), up2), x, y);
          code[0][j] = __float_as_uint(__fadd_rz(fminf(x, qmax), 8388608.f));
          code[1][j] = __float_as_uint(__fadd_rz(fminf(y, qmax), 8388608.f));
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        store_unit<BITS>(a.codes + to[u] * (16 * BITS), code[u], l, to[u] >= 0, bad >> ((l * NG / 8 + u * NG) << kShift) & 1);
    }
  }
}

// Each slot of `slots` sets its bit in `seen`; one that was set already is named
// twice and sets it in `twice`. Which of its rows came second differs from run
// to run, so the rows are looked up once both are complete: the first that is
// outside or named twice is the same one every time.
__global__ void __launch_bounds__(256) mark_slots_kernel(const int64_t *__restrict__ slots, int64_t n,
                                                         int64_t n_slots, uint32_t *seen, uint32_t *twice) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t s = slots[i];
    if (s < 0 || s >= n_slots) continue;
    const uint32_t bit = 1u << (s & 31);
    if (atomicOr(seen + (s >> 5), bit) & bit) atomicOr(twice + (s >> 5), bit);
  }
}
__global__ void __launch_bounds__(256) check_slots_kernel(const int64_t *__restrict__ slots, int64_t n,
                                                          int64_t n_slots, const uint32_t *twice,
                                                          unsigned long long *first_bad) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t s = slots[i];
    if (s == -1) continue;
    const bool out = s < -1 || s >= n_slots;
    if (out || (twice[s >> 5] >> (s & 31) & 1u)) atomicMin(first_bad, (unsigned long long)i * 2 + (out ? 0 : 1));
  }
}

// Tokens of a tile: as many as leave eight CTAs to an SM, so that few rows
// spread over the GPU and many share the look-up of their slots.
int tile_tokens(int64_t n, int n_caches) {
  return (int)std::clamp<int64_t>(n * n_caches / ((int64_t)sm_count() * 8), 1, kTileTokens);
}
dim3 tile_grid(int64_t n, int tile, int n_caches) {
  return dim3((unsigned)std::min<int64_t>(cdiv(n, tile), (int64_t)sm_count() * 128), (unsigned)n_caches);
}

// The second cache by itself: a pair whose caches need different kernels takes a
// launch for each, so that a cache's rows do not depend on its partner.
CachePair second(const CachePair &c) {
  CachePair d = c;
  d.cache[0] = c.cache[1], d.rows[0] = c.rows[1], d.unit[0] = c.unit[1];
  return d;
}

// lanes of the widest row, eight elements each
int lanes_log2(const CachePair &c, int n_caches) {
  int ll = 0;
  for (int i = 0; i < n_caches; ++i) ll = std::max(ll, ilog2(cdiv(c.cache[i].head_dim, 8)));
  return ll;
}

// Whether the kernels of units of 128 elements take the caches: groups of whole
// columns of the first product, blocks inside a unit, and for writing bf16 rows
// and groups inside a unit too.
bool takes_units(const CachePair &c, int n_caches) {
  for (int i = 0; i < n_caches; ++i) {
    const qwha_cache &a = c.cache[i];
    if (a.bits != c.cache[0].bits || (int64_t)a.heads * a.head_dim % 128 || !is_pow2(a.group) || a.group < 32 ||
        a.had_block > 128)
      return false;
  }
  return true;
}
bool writes_units(qwha_dtype dt, const CachePair &c, int n_caches) {
  if (dt != QWHA_BF16 || !takes_units(c, n_caches)) return false;
  const int g = c.cache[0].group;
  return g <= 128 && g == c.cache[n_caches - 1].group;
}
template <int BITS>
void write_units(const CachePair &c, dim3 grid, const int64_t *slots, int64_t n, int tile, unsigned int *err,
                 cudaStream_t s) {
  switch (c.cache[0].group) {
    case 128: cache_write_unit_kernel<BITS, 1><<<grid, kCacheThreads, 0, s>>>(c, slots, n, tile, err); break;
    case 64: cache_write_unit_kernel<BITS, 2><<<grid, kCacheThreads, 0, s>>>(c, slots, n, tile, err); break;
    default: cache_write_unit_kernel<BITS, 4><<<grid, kCacheThreads, 0, s>>>(c, slots, n, tile, err);
  }
}
template <typename T>
void read_mma(const CachePair &c, dim3 grid, int tile, const ReadArgs &r, int64_t n, unsigned int *err,
              cudaStream_t s) {
  switch (c.cache[0].bits) {
    case 2: cache_read_mma_kernel<T, 2><<<grid, kCacheThreads, 0, s>>>(c, r, n, tile, err); break;
    case 3: cache_read_mma_kernel<T, 3><<<grid, kCacheThreads, 0, s>>>(c, r, n, tile, err); break;
    case 4: cache_read_mma_kernel<T, 4><<<grid, kCacheThreads, 0, s>>>(c, r, n, tile, err); break;
    default: cache_read_mma_kernel<T, 8><<<grid, kCacheThreads, 0, s>>>(c, r, n, tile, err);
  }
}

}  // namespace

int cache_max_head_dim() { return 256; }

int cache_write_launches(qwha_dtype dt, const CachePair &c, int n_caches) {
  const bool apart = n_caches == 2 && !writes_units(dt, c, 2) && (writes_units(dt, c, 1) || writes_units(dt, second(c), 1));
  return apart ? 2 : 1;
}
int cache_read_launches(const CachePair &c, int n_caches) {
  return n_caches == 2 && !takes_units(c, 2) && (takes_units(c, 1) || takes_units(second(c), 1)) ? 2 : 1;
}

cudaError_t launch_cache_write(qwha_dtype dt, const CachePair &c, int n_caches, const int64_t *slots, int64_t n,
                               cudaStream_t s) {
  if (cache_write_launches(dt, c, n_caches) == 2) {
    const cudaError_t e = launch_cache_write(dt, c, 1, slots, n, s);
    return e != cudaSuccess ? e : launch_cache_write(dt, second(c), 1, slots, n, s);
  }
  const int tile = tile_tokens(n, n_caches);
  const dim3 grid = tile_grid(n, tile, n_caches);
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  if (writes_units(dt, c, n_caches)) {
    switch (c.cache[0].bits) {
      case 2: write_units<2>(c, grid, slots, n, tile, err, s); break;
      case 3: write_units<3>(c, grid, slots, n, tile, err, s); break;
      case 4: write_units<4>(c, grid, slots, n, tile, err, s); break;
      default: write_units<8>(c, grid, slots, n, tile, err, s);
    }
    return cudaGetLastError();
  }
  const int ll = lanes_log2(c, n_caches);
  if (dt == QWHA_F32) cache_write_kernel<float><<<grid, kCacheThreads, 0, s>>>(c, ll, slots, n, tile, err);
  else cache_write_kernel<__nv_bfloat16><<<grid, kCacheThreads, 0, s>>>(c, ll, slots, n, tile, err);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(qwha_dtype dt, const CachePair &c, int n_caches, const ReadArgs &r, int64_t n,
                              cudaStream_t s) {
  if (cache_read_launches(c, n_caches) == 2) {
    const cudaError_t e = launch_cache_read(dt, c, 1, r, n, s);
    return e != cudaSuccess ? e : launch_cache_read(dt, second(c), 1, r, n, s);
  }
  const int tile = tile_tokens(n, n_caches);
  const dim3 grid = tile_grid(n, tile, n_caches);
  unsigned int *err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  if (takes_units(c, n_caches)) {
    if (dt == QWHA_F32) read_mma<float>(c, grid, tile, r, n, err, s);
    else read_mma<__nv_bfloat16>(c, grid, tile, r, n, err, s);
    return cudaGetLastError();
  }
  const int ll = lanes_log2(c, n_caches);
  if (dt == QWHA_F32) cache_read_kernel<float><<<grid, kCacheThreads, 0, s>>>(c, ll, r, n, tile, err);
  else cache_read_kernel<__nv_bfloat16><<<grid, kCacheThreads, 0, s>>>(c, ll, r, n, tile, err);
  return cudaGetLastError();
}

namespace {
size_t slot_bits_bytes(int64_t n_slots) { return align_up((size_t)cdiv(n_slots, 32) * 4, 256); }
}  // namespace

size_t check_slots_bytes(int64_t n_slots) { return 256 + 2 * slot_bits_bytes(n_slots); }

cudaError_t launch_check_slots(const int64_t *slots, int64_t n, int64_t n_slots, void *ws, unsigned long long *bad,
                               cudaStream_t s) {
  const size_t bits = slot_bits_bytes(n_slots);
  unsigned long long *word = static_cast<unsigned long long *>(ws);
  uint32_t *seen = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + 256), *twice = seen + bits / 4;
  cudaError_t e = cudaMemsetAsync(word, 0xff, sizeof(*word), s);
  if (e == cudaSuccess) e = cudaMemsetAsync(seen, 0, 2 * bits, s);
  if (e != cudaSuccess) return e;
  if (n > 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(cdiv(n, 256), (int64_t)sm_count() * 8);
    mark_slots_kernel<<<grid, 256, 0, s>>>(slots, n, n_slots, seen, twice);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    check_slots_kernel<<<grid, 256, 0, s>>>(slots, n, n_slots, twice, word);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = cudaMemcpyAsync(bad, word, sizeof(*bad), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

}  // namespace qwha
