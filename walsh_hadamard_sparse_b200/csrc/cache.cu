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

// Rows of up to 256 elements, eight to a lane: 1 << ll lanes hold a row.
template <typename T>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CachePair c, int ll,
                                                                    const int64_t *__restrict__ slots, int64_t n,
                                                                    unsigned int *err) {
  using A = typename wide<T>::type;
  const qwha_cache &a = c.cache[blockIdx.y];
  const T *rows = static_cast<const T *>(c.rows[blockIdx.y]);
  const int lane = threadIdx.x & ((1 << ll) - 1);
  const bool has = lane * 8 < a.head_dim;
  const int gl = a.group / 8, ng = a.head_dim / a.group;
  const A qmax = (A)((1 << a.bits) - 1), step = (A)1 / qmax, unit = (A)c.unit[blockIdx.y], half = (A)(0.5 + 1.0 / 4096);
  const int64_t items = n * a.heads, n_slots = a.n_pages * a.page_size;
  const int64_t per = kCacheThreads >> ll;
  for (int64_t base = (int64_t)blockIdx.x * per; base < items; base += (int64_t)gridDim.x * per) {
    const int64_t it = base + (threadIdx.x >> ll);
    bool live = it < items;
    int64_t slot = -1;
    if (live) slot = slots[it / a.heads];
    if (slot < -1 || slot >= n_slots) {
      if (lane == 0) atomicOr(err, kErrSlot);
      slot = -1;
    }
    live = slot >= 0 && has;
    A v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0;
    if (live) {
      const T *src = rows + it * a.head_dim + lane * 8;
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
    float s = (float)mul(add(hi, -lo), step);
    const bool bad = !(s <= 3.402823466e38f);
    if (s < 1.1754943508e-38f) s = 1.f;
    const A inv = (A)1 / (A)s;
    const A zf = floor(add(mul(-lo, inv), half)), z = zf < qmax ? zf : qmax;
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const A r = add(mul(v[i], inv), z + half);
      q[i] = bad || !(r > (A)0) ? 0u : r < qmax ? (uint32_t)r : (uint32_t)qmax;
    }
    if (live) {
      const int64_t row = slot * a.heads + it % a.heads;
      store_run(a.codes + row * (a.head_dim / 8 * a.bits) + lane * a.bits, q, a.bits);
      if (lane % gl == 0) {
        a.scales[row * ng + lane / gl] = bad ? __int_as_float(0x7fc00000) : s;
        a.zeros[row * ng + lane / gl] = bad ? 0 : (uint8_t)z;
      }
    }
  }
}

// Output row i belongs to the sequence b with row_start[b] <= i <
// row_start[b + 1] and is its token first[b] + i - row_start[b].
template <typename T>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const CachePair c, int ll, const int32_t *__restrict__ pages, int max_pages,
                      const int64_t *__restrict__ row_start, const int64_t *__restrict__ first, int n_seqs, int64_t n,
                      unsigned int *err) {
  const qwha_cache &a = c.cache[blockIdx.y];
  T *rows = static_cast<T *>(const_cast<void *>(c.rows[blockIdx.y]));
  const int lane = threadIdx.x & ((1 << ll) - 1);
  const bool has = lane * 8 < a.head_dim;
  const int ng = a.head_dim / a.group;
  const float unit = (float)c.unit[blockIdx.y];
  const int64_t end = row_start[n_seqs];
  const int64_t items = (end < n ? end : n) * a.heads;
  const int64_t per = kCacheThreads >> ll;
  for (int64_t base = (int64_t)blockIdx.x * per; base < items; base += (int64_t)gridDim.x * per) {
    const int64_t it = base + (threadIdx.x >> ll);
    const int64_t i = it / a.heads;
    bool live = it < items;
    int64_t slot = 0;
    if (live) {
      int lo = 0, hi = n_seqs;  // row_start[lo] <= i < row_start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start[mid] <= i) lo = mid;
        else hi = mid;
      }
      const int64_t pos = i - row_start[lo] + (first ? first[lo] : 0);
      const int64_t pg = pos / a.page_size;
      int64_t page = -1;
      if (pos >= 0 && pg < max_pages) page = pages[(int64_t)lo * max_pages + pg];
      if (page < 0 || page >= a.n_pages) {
        if (lane == 0) atomicOr(err, kErrPage);
        live = false;
      }
      slot = page * a.page_size + (pos - pg * a.page_size);
    }
    live = live && has;
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.f;
    const int64_t row = slot * a.heads + it % a.heads;
    if (live) {
      load_run(a.codes + row * (a.head_dim / 8 * a.bits) + lane * a.bits, v, a.bits);
      const int64_t g = row * ng + lane * 8 / a.group;
      const float s = a.scales[g], z = (float)a.zeros[g];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = __fmul_rn(s, v[u] - z);
    }
    rotate8(v, a.had_block, unit, lane);
    if (live) {
      T *dst = rows + it * a.head_dim + lane * 8;
#pragma unroll
      for (int u = 0; u < 8; u += io<T>::kVec) *reinterpret_cast<uint4 *>(dst + u) = io<T>::pack(v + u);
    }
  }
}

// Each slot of `slots` sets its bit; a bit that was set already is a duplicate.
__global__ void __launch_bounds__(256) check_slots_kernel(const int64_t *__restrict__ slots, int64_t n,
                                                          int64_t n_slots, uint32_t *seen,
                                                          unsigned long long *first_bad) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t s = slots[i];
    if (s == -1) continue;
    const bool out = s < -1 || s >= n_slots;
    const bool twice = !out && (atomicOr(seen + (s >> 5), 1u << (s & 31)) >> (s & 31) & 1u);
    if (out || twice) atomicMin(first_bad, (unsigned long long)i * 2 + (twice ? 1 : 0));
  }
}

int lanes_log2(int head_dim) { return ilog2(cdiv(head_dim, 8)); }

unsigned row_grid(int64_t items, int ll) {
  return (unsigned)std::min<int64_t>(cdiv(items, kCacheThreads >> ll), (int64_t)sm_count() * 16);
}

}  // namespace

int cache_max_head_dim() { return 256; }

cudaError_t launch_cache_write(qwha_dtype dt, const CachePair &c, int n_caches, const int64_t *slots, int64_t n,
                               cudaStream_t s) {
  int ll = 0, heads = 0;
  for (int i = 0; i < n_caches; ++i) {
    ll = std::max(ll, lanes_log2(c.cache[i].head_dim));
    heads = std::max(heads, c.cache[i].heads);
  }
  const dim3 grid(row_grid(n * heads, ll), (unsigned)n_caches);
  unsigned int *err = device_error_word();
  if (dt == QWHA_F32) cache_write_kernel<float><<<grid, kCacheThreads, 0, s>>>(c, ll, slots, n, err);
  else cache_write_kernel<__nv_bfloat16><<<grid, kCacheThreads, 0, s>>>(c, ll, slots, n, err);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(qwha_dtype dt, const CachePair &c, int n_caches, const int32_t *pages, int max_pages,
                              const int64_t *row_start, const int64_t *first, int n_seqs, int64_t n, cudaStream_t s) {
  int ll = 0, heads = 0;
  for (int i = 0; i < n_caches; ++i) {
    ll = std::max(ll, lanes_log2(c.cache[i].head_dim));
    heads = std::max(heads, c.cache[i].heads);
  }
  const dim3 grid(row_grid(n * heads, ll), (unsigned)n_caches);
  unsigned int *err = device_error_word();
  if (dt == QWHA_F32)
    cache_read_kernel<float><<<grid, kCacheThreads, 0, s>>>(c, ll, pages, max_pages, row_start, first, n_seqs, n, err);
  else
    cache_read_kernel<__nv_bfloat16>
        <<<grid, kCacheThreads, 0, s>>>(c, ll, pages, max_pages, row_start, first, n_seqs, n, err);
  return cudaGetLastError();
}

size_t check_slots_bytes(int64_t n_slots) { return 256 + align_up((size_t)cdiv(n_slots, 32) * 4, 256); }

cudaError_t launch_check_slots(const int64_t *slots, int64_t n, int64_t n_slots, void *ws, unsigned long long *bad,
                               cudaStream_t s) {
  unsigned long long *word = static_cast<unsigned long long *>(ws);
  uint32_t *seen = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + 256);
  cudaError_t e = cudaMemsetAsync(word, 0xff, sizeof(*word), s);
  if (e == cudaSuccess) e = cudaMemsetAsync(seen, 0, (size_t)cdiv(n_slots, 32) * 4, s);
  if (e != cudaSuccess) return e;
  if (n > 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(cdiv(n, 256), (int64_t)sm_count() * 8);
    check_slots_kernel<<<grid, 256, 0, s>>>(slots, n, n_slots, seen, word);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = cudaMemcpyAsync(bad, word, sizeof(*bad), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

}  // namespace qwha
