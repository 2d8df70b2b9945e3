// The packed matrix-vector product on tensor cores (see gemv.cu): one
// definition for the three code widths, instantiated by gemv_b2/3/4.cu.
//
// Unpacking bounds this kernel more than memory does: at 6.5 TB/s a 4-bit code
// leaves about three instruction slots, and half as many on the integer pipe.
// Two exact representations keep the count below one slot a code:
//   * a code masked out of a 16-bit half at bit o (o <= 7, o + bits <= 10), ORed
//     into the mantissa of the f16 1024, is 1024 + q * 2^o: one instruction for
//     two codes, most need no shift, and subtracting 1024 + zero * 2^o leaves
//     (q - zero) * 2^o, all exact for any zero point of a byte (`less_zero`);
//   * the tokens' values, scaled by a power of two per chunk of 128 columns so
//     that the largest lies in [2^14, 2^15), are f16 numbers too: a bf16 value
//     in one piece (below 2^-24 of the chunk's largest it is held to 2^-32 of
//     that), an fp32 value in three, each of what the one before leaves times
//     2^11 (all 24 bits, down to 2^-54 of the largest); 2^-o is folded into the
//     values (decode_prepare_kernel). Each piece is a column of the instruction.
// The matrix unit (m16n8k16, 8.3 clocks measured for f16 and bf16 alike) adds
// the exact products in fp32 over one quantization group; then, in fp32,
//   acc += scale * (2^k * sum_k (q - zero) x),
// with 2^k per (chunk, token) prepared beside the values. No weight is rounded,
// and a value on a zero weight leaves nothing.
//
// Layout. A warp takes 16 MT rows and a slice of the columns; the warps of a
// CTA are KS slices of kWarps / KS tiles. The four lanes of a row take a run of
// 32 columns each of a 128-column chunk. The order of the columns inside the
// sum is free: a lane's fragment holds codes of its own run in the order the
// masks yield, and the values are stored in that order. Where a group is
// shorter than the chunk (G = 2 or 4 groups in it), the eight columns of the
// instruction are G groups times 8 / G pieces: a column holds its piece on the
// lanes of its group and zeros elsewhere, so no sum crosses a group.
//
// Memory. Codes, scales and zero points go straight to the registers of the
// lane that uses them, DEPTH chunks ahead, past L1; the values come through L1,
// or with OWN from shared memory. No barrier until the slices are added.
//
// 14336 x 4096, 3 bits, one token: 15.5 us; 4096 x 14336, 4 bits, eight tokens:
// 13.2 us (37% of the copy rate). Tried and slower, when these took 18 and 15:
// codes through rings of shared memory filled by bulk copies (18 to 30 us), fp8
// operands (converted on the integer pipe, 26 us), values staged in shared
// memory (18 and 35 us). The arguments are __grid_constant__: a copy of them in
// every thread, for the function that takes them by reference, cost 1 to 2 us.

#pragma once

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "bulk.cuh"
#include "common.cuh"
#include "kernels.h"

namespace qwha {
namespace gemv {

constexpr int kWarps = 8;

// Pair p (0 <= p < 16) of a run of 32 codes: codes first(p) and first(p) +
// gap() in the halves of a register, at bit `unit(p)` of their half.
template <int BITS>
__host__ __device__ constexpr int first(int p) {
  return BITS == 4 ? 8 * (p / 4) + p % 4 : BITS == 2 ? 16 * (p / 8) + p % 8 : p;
}
template <int BITS>
__host__ __device__ constexpr int gap() {
  return BITS == 4 ? 4 : BITS == 2 ? 8 : 16;
}
template <int BITS>
__host__ __device__ constexpr int unit(int p) {
  if (BITS == 4) return p % 2 * 4;
  if (BITS == 2) return p % 4 * 2;
  constexpr int u[16] = {0, 3, 6, 0, 3, 6, 2, 5, 0, 3, 6, 1, 4, 7, 0, 3};
  return u[p];
}

// The sixteen pairs of a run.
template <int BITS>
__device__ __forceinline__ void unpack(const uint32_t *w, uint32_t *q) {
  if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = w[i] >> 8;
      q[4 * i] = w[i] & 0x000f000fu, q[4 * i + 1] = w[i] & 0x00f000f0u;
      q[4 * i + 2] = h & 0x000f000fu, q[4 * i + 3] = h & 0x00f000f0u;
    }
  } else if constexpr (BITS == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = w[i] >> 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) q[8 * i + j] = w[i] & (0x00030003u << (2 * j));
#pragma unroll
      for (int j = 0; j < 4; ++j) q[8 * i + 4 + j] = h & (0x00030003u << (2 * j));
    }
  } else {
    // the 96 bits as halves h0..h5: codes 0..15 are h0..h2, codes 16..31 are h3..h5; side by side, halves i and
    // i + 3 hold codes p and p + 16 at the same place. Codes 5 and 10 straddle two halves.
    const uint32_t a = __byte_perm(w[0], w[1], 0x7610), b = __byte_perm(w[0], w[2], 0x5432),
                   c = __byte_perm(w[1], w[2], 0x7610);
    const uint32_t ah = a >> 9, bh = b >> 8, ch = c >> 10;
    q[0] = a & 0x00070007u, q[1] = a & 0x00380038u, q[2] = a & 0x01c001c0u;
    q[3] = ah & 0x00070007u, q[4] = ah & 0x00380038u;
    q[5] = (ah & 0x00400040u) | ((b << 7) & 0x01800180u);
    q[6] = b & 0x001c001cu, q[7] = b & 0x00e000e0u;
    q[8] = bh & 0x00070007u, q[9] = bh & 0x00380038u;
    q[10] = (bh & 0x00c000c0u) | ((c << 8) & 0x01000100u);
    q[11] = c & 0x000e000eu, q[12] = c & 0x00700070u, q[13] = c & 0x03800380u;
    q[14] = ch & 0x00070007u, q[15] = ch & 0x00380038u;
  }
}

// (q - zero) 2^o of the sixteen pairs, from q at bit o of its half: 1024 + q 2^o
// by its bits, less 1024 + zero 2^o (a multiple of 2^o up to 1024 + 255 * 2^7:
// an f16 number). One addition for two codes, on another pipe than the
// unpacking. The codes as they are, f16 denormals, would be exact too, but the
// matrix unit aligns products by the operands' nominal exponents, so they cost
// the sums about eight bits; and zero * sum x taken off a sum of q x costs the
// bits of a large value that does not count (1e5 among ones, whose weight is 0:
// off by 0.13).
template <int BITS>
__device__ __forceinline__ void less_zero(uint32_t *q, uint32_t zero) {
  const uint32_t at0 = zero * 0x10001u + 0x64006400u, of1024 = 0x64006400u;
  const __half2 z = __hsub2(reinterpret_cast<const __half2 &>(at0), reinterpret_cast<const __half2 &>(of1024));
  __half2 off[8];
#pragma unroll
  for (int o = 0; o < 8; ++o) {
    const uint32_t by = (0x3c00u + (o << 10)) * 0x10001u;  // 2^o
    off[o] = o ? __hfma2(z, reinterpret_cast<const __half2 &>(by), reinterpret_cast<const __half2 &>(of1024))
               : reinterpret_cast<const __half2 &>(at0);
  }
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    q[p] |= of1024;
    const __half2 d = __hsub2(reinterpret_cast<const __half2 &>(q[p]), off[unit<BITS>(p)]);
    q[p] = reinterpret_cast<const uint32_t &>(d);
  }
}

// d = A B
__device__ __forceinline__ void mma0(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// c += A B
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.402823466e38f; }

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *v) {
#pragma unroll
  for (int u = 0; u < 8; u += io<T>::kVec) io<T>::unpack(*reinterpret_cast<const uint4 *>(p + u), v + u);
}

// sum of (q - z) x over a run of eight codes, in fp64, U of them unrolled.
template <int U, typename T>
__device__ __forceinline__ double run_dot(uint32_t w, int bits, int z, const T *x) {
  double sum = 0.;
#pragma unroll U
  for (int i = 0; i < 8; ++i, w >>= bits)
    sum = fma((double)((float)(w & ((1u << bits) - 1u)) - (float)z), (double)io<T>::load1(x + i), sum);
  return sum;
}

// One row and token by the definition in fp64, for results that the products
// leave infinite or NaN: a token with an infinity or a NaN has no pieces, and a
// sum of values near the type's largest may leave fp32's range before its scale
// brings it back. A thread by itself: slow, and rare.
static __device__ __noinline__ float plain_dot(const GemvArgs &a, int row, int tok) {
  const int ng = a.d_in / a.group;
  const uint8_t *qw = a.qw + (int64_t)row * (a.d_in / 8) * a.bits;
  double sum = 0.;
  for (int r = 0; r < a.d_in / 8; ++r) {
    uint32_t w = 0;
    for (int b = 0; b < a.bits; ++b) w |= (uint32_t)qw[(int64_t)r * a.bits + b] << (8 * b);
    const int64_t g = (int64_t)row * ng + r * 8 / a.group, at = (int64_t)tok * a.d_in + r * 8;
    const double part = a.f32 ? run_dot<8>(w, a.bits, a.zeros[g], static_cast<const float *>(a.x) + at)
                              : run_dot<8>(w, a.bits, a.zeros[g], static_cast<const __nv_bfloat16 *>(a.x) + at);
    sum = fma((double)a.scales[g], part, sum);
  }
  return (float)sum;
}

// Four consecutive values.
__device__ __forceinline__ void load4(const float *p, float *v) { io<float>::unpack(*reinterpret_cast<const uint4 *>(p), v); }
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *v) {
  const uint2 q = *reinterpret_cast<const uint2 *>(p);
  v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
}

__device__ __forceinline__ float exp2i(int k) { return __int_as_float((k + 127) << 23); }  // -126 <= k <= 127
__device__ __forceinline__ float exp2_far(int k) { return exp2i(k >> 1) * exp2i(k - (k >> 1)); }  // -149 <= k <= 127

// The tokens as operands: one thread per token, run of 32 columns and quarter
// of its pairs, the sixteen of a chunk on neighbouring lanes (i = run * 4 + j).
// The chunk's values are scaled by the power of two that brings the largest
// into [2^14, 2^15), then split into f16 pieces: the value rounded, and what
// that leaves, exact in fp32, times 2^11 for the next (the product's end takes
// the 2^-11 back). A pair's unit divides its values. factors gets, per group
// beside each column, the power of two that undoes the scaling: a denormal for
// a chunk whose largest is below 2^-112. A chunk with an infinity or a NaN gets
// the factor NaN, which sends its rows' sums to the plain path.
// In shared memory (OWN: one n-tile) a column's pieces lie together, `cols` being
// the stride between columns.
template <int BITS, bool OWN, typename T>
__device__ __forceinline__ void prepare_piece(const GemvArgs &a, int tok, int i, bool live, int cols, uint4 *pieces,
                                              float *factors) {
  const int run = i >> 2, j = i & 3, chunk = run >> 2, t = run & 3, k0 = run * 32;
  // the pairs' first halves and second halves are four consecutive values each
  const int at = first<BITS>(0) + (BITS == 4 ? 8 * j : BITS == 2 ? 16 * (j >> 1) + 4 * (j & 1) : 4 * j);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live && k0 < a.d_in) {
    const T *src = static_cast<const T *>(a.x) + (int64_t)tok * a.d_in + k0 + at;
    load4(src, v);
    load4(src + gap<BITS>(), v + 4);
  }
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) top = max(top, __float_as_uint(v[u]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 16; o *= 2) top = max(top, __shfl_xor_sync(~0u, top, o));
  const bool whole = top < 0x7f800000u;  // no infinity, no NaN
  const int e = max(1, (int)(top >> 23)), up = top && whole ? 141 - e : 0;  // top < 2^(e - 126)
  const float f0 = exp2i(up >> 1), f1 = exp2i(up - (up >> 1));
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = whole ? v[u] * f0 * f1 : 0.f;
  if (!live) return;
  const int G = a.group % 128 == 0 ? 1 : a.group % 64 == 0 ? 2 : 4;
  for (int p = 0; p < a.pieces; ++p) {
    const int col = tok * a.pieces + p, TPN = 8 / G;
    const int64_t tile = OWN ? chunk : (int64_t)chunk * x_tiles(cols, G) + col / TPN;
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // the unit of pair 4 j + k
      constexpr int A[4] = {unit<BITS>(0), unit<BITS>(1), unit<BITS>(2), unit<BITS>(3)},
                    B[4] = {unit<BITS>(4), unit<BITS>(5), unit<BITS>(6), unit<BITS>(7)},
                    C[4] = {unit<BITS>(8), unit<BITS>(9), unit<BITS>(10), unit<BITS>(11)},
                    D[4] = {unit<BITS>(12), unit<BITS>(13), unit<BITS>(14), unit<BITS>(15)};
      const int o = j == 0 ? A[k] : j == 1 ? B[k] : j == 2 ? C[k] : D[k];
      const float by = exp2i(-o), back = exp2i(o);
      const __half2 d = __floats2half2_rn(v[k] * by, v[4 + k] * by);
      r[k] = *reinterpret_cast<const uint32_t *>(&d);
      v[k] = (v[k] - __low2float(d) * back) * 2048.f, v[4 + k] = (v[4 + k] - __high2float(d) * back) * 2048.f;
    }
    pieces[OWN ? col * cols + chunk * 16 + j * 4 + t : tile * (16 * TPN) + j * (4 * TPN) + col % TPN * 4 + t] =
        make_uint4(r[0], r[1], r[2], r[3]);
    if (j == 0 && t % (4 / G) == 0)
      factors[tile * 8 + t * G / 4 * TPN + col % TPN] = whole ? exp2_far(-up) : __int_as_float(0x7fc00000);
  }
}

// What a lane holds of a chunk: its runs of 2 MT rows, with their scales and
// zero points where it has groups of its own (G > 1).
template <int BITS, int G, int MT>
struct Chunk {
  uint32_t w[2 * MT][BITS];
  float s[G > 1 ? 2 * MT : 1];
  uint32_t z[G > 1 ? 2 * MT : 1];
};

// Whether the word became 1 (in time); what was written before it is visible then.
__device__ __forceinline__ bool wait_ready(const unsigned int *word) {
  const uint64_t begin = bulk::now_ns();
  for (;;) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (v == 1) return true;
    if (bulk::now_ns() - begin > bulk::kWaitNs) return false;
  }
}

// A lane's operands of an n-tile, and the factors of its two columns.
struct XTile {
  uint4 x[4];
  float2 f;
};

template <int BITS>
__device__ __forceinline__ void f_zero(uint32_t *w) {
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0;
}

// f(0), f(1), ..., f(N - 1) with compile-time arguments.
template <int N, typename F>
__device__ __forceinline__ void each(F &&f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>());
  }
}

template <int BITS, int OFF>
__device__ __forceinline__ void load_run(const uint8_t *p, uint32_t *w) {
  if constexpr (BITS == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p), "n"(OFF));
  else if constexpr (BITS == 2)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2+%3];" : "=r"(w[0]), "=r"(w[1]) : "l"(p), "n"(OFF));
  else
    asm volatile(
        "ld.global.nc.u32 %0, [%3+%4];\n\tld.global.nc.u32 %1, [%3+%5];\n\tld.global.nc.u32 %2, [%3+%6];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2])
        : "l"(p), "n"(OFF), "n"(OFF + 4), "n"(OFF + 8));
}

// EXACT: the group is 128 / G columns, so a chunk's groups follow the chunk.
// OWN: no launch prepared the operands; every CTA makes its own in shared memory.
template <int BITS, int G, int NT, int MT, int DEPTH, bool EXACT, bool OWN>
__global__ void __launch_bounds__(kWarps * 32, NT <= 4 ? 2 : 1)
    gemv_mma_kernel(const __grid_constant__ GemvArgs a, int tokens_per_pass, int slices) {
  constexpr int TPN = 8 / G, ROWS = 16 * MT, ROW_CHUNK = 16 * BITS;
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int t0 = blockIdx.y * tokens_per_pass;
  const int np = a.T - t0 < tokens_per_pass ? a.T - t0 : tokens_per_pass;
  const int ng = a.d_in / a.group, chunks = (a.d_in + 127) / 128;
  const int tiles_here = kWarps / slices;
  const int row_first = blockIdx.x * tiles_here * ROWS;  // of the CTA
  const int row0 = row_first + warp / slices * ROWS;     // of the warp
  const int per = (chunks + slices - 1) / slices;
  const int c_begin = warp % slices * per;
  const int c_end = row0 < a.d_out ? (c_begin + per < chunks ? c_begin + per : chunks) : c_begin;

  const uint8_t *pw[2 * MT], *pz[2 * MT];
  const float *ps[2 * MT];
  {
    const int64_t row_bytes = (int64_t)(a.d_in / 32) * (4 * BITS);
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      int r = row0 + h * 8 + g;
      r = r < a.d_out ? r : a.d_out - 1;  // rows behind the last one repeat it and are not stored
      const int64_t grp = (int64_t)r * ng + (EXACT ? c_begin * G + t * G / 4 : 0);
      pw[h] = a.qw + r * row_bytes + (int64_t)c_begin * ROW_CHUNK + t * (4 * BITS);
      ps[h] = a.scales + grp;
      pz[h] = a.zeros + grp;
    }
  }
  // chunk c + I, I chunks behind the pointers
  auto fetch = [&](Chunk<BITS, G, MT> &f, int c, auto I) {
    constexpr int i = decltype(I)::value;
    const int k0 = c * 128 + t * 32;
    const bool on = c < c_end && (G == 1 || k0 < a.d_in);
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      if constexpr (G > 1) f.s[h] = 0.f;
      if (!on) continue;
      load_run<BITS, i * ROW_CHUNK>(pw[h], f.w[h]);
      if constexpr (G > 1) {
        const int gi = EXACT ? i * G : k0 / a.group;
        f.s[h] = __ldg(ps[h] + gi);
        f.z[h] = __ldg(pz[h] + gi);
      }
    }
  };
  // With one group to a chunk, the four lanes of a row load those of four chunks and hand them round: a quarter of
  // the requests (each touches eight rows), and half the registers of a ring of them.
  float sn[2 * MT], s4[2 * MT];
  uint32_t zn[2 * MT], z4[2 * MT];
  auto fetch_scales = [&](int c) {  // of chunks c .. c + 3
    const int ct = c + t;
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      sn[h] = 0.f, zn[h] = 0;
      if (ct < c_end) {
        const int gi = EXACT ? ct - c_begin : ct * 128 / a.group;
        sn[h] = __ldg(ps[h] + gi);
        zn[h] = __ldg(pz[h] + gi);
      }
    }
  };
  Chunk<BITS, G, MT> buf[DEPTH];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i)
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      f_zero<BITS>(buf[i].w[h]);
      if constexpr (G > 1) buf[i].z[h] = 0;
    }
  if constexpr (G == 1) fetch_scales(c_begin);
  each<DEPTH>([&](auto I) { fetch(buf[decltype(I)::value], c_begin + decltype(I)::value, I); });

  const int pieces = a.pieces, v_end = np * pieces, v_most = tokens_per_pass * pieces;
  const int n_tiles = x_tiles(a.T * pieces, G), nt0 = t0 * pieces / TPN;
  // this lane's column of an n-tile: a piece, live where the column's group is the lane's own
  const bool mine = g / TPN == t * G / 4;
  const uint4 *xp;
  const float2 *xs;
  if constexpr (OWN) {
    const int column = chunks * 16 + 4, parts = chunks * 16;  // padded: two columns' quarters in different banks
    uint4 *own = reinterpret_cast<uint4 *>(smem + kWarps * G * v_most * ROWS);
    float *factors = reinterpret_cast<float *>(own + v_most * column);
    for (int i = threadIdx.x; (i & ~31) < a.T * parts; i += kWarps * 32) {
      const bool live = i < a.T * parts;
      if (a.f32) prepare_piece<BITS, true, float>(a, i / parts, i % parts, live, column, own, factors);
      else prepare_piece<BITS, true, __nv_bfloat16>(a, i / parts, i % parts, live, column, own, factors);
    }
    __syncthreads();
    xp = own + g % TPN * column + c_begin * 16 + t;
    xs = reinterpret_cast<const float2 *>(factors) + c_begin * 4 + t;
  } else {
    // The values are the preparing launch's output: wait for it only here. With the entries' launch in between,
    // which runs beside this one, its word says so.
    if (a.y_ad) {
      if (lane == 0 && !wait_ready(a.ready)) atomicOr(a.err, kErrEntries);
      __syncwarp();
    } else {
      asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    xp = a.xpieces + ((int64_t)c_begin * n_tiles + nt0) * (16 * TPN) + g % TPN * 4 + t;
    xs = reinterpret_cast<const float2 *>(a.xfac) + ((int64_t)c_begin * n_tiles + nt0) * 4 + t;
  }
  // Tile n of the chunk `ahead` behind the pointers. The values are asked for as soon as the tile before in their
  // registers is used: they come from L2 as often as not. Columns of other groups and behind the last piece are
  // zero; runs behind the last column were prepared as zeros.
  constexpr int S = NT < 8 ? 1 : 2;
  const int tiles_of = NT == 1 ? 1 : n_tiles;  // a call with more n-tiles takes a wider variant
  XTile xt[S];
  const bool on1 = mine && g % TPN < v_end;
  auto load_x = [&](XTile &f, int ahead, int n) {
    if constexpr (OWN) {
      if (on1)
#pragma unroll
        for (int j = 0; j < 4; ++j) f.x[j] = xp[ahead * 16 + j * 4];
    } else if constexpr (NT == 1) {  // the registers hold nothing else: cleared once
      if (on1)
#pragma unroll
        for (int j = 0; j < 4; ++j) f.x[j] = xp[ahead * (16 * TPN) + j * (4 * TPN)];
    } else {
      const bool on = mine && n * TPN + g % TPN < v_end;
      const uint4 *p = xp + ((int64_t)ahead * tiles_of + n) * (16 * TPN);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.x[j] = make_uint4(0, 0, 0, 0);
        if (on) f.x[j] = p[j * (4 * TPN)];
      }
    }
    f.f = xs[(ahead * tiles_of + n) * 4];
  };
#pragma unroll
  for (int n = 0; n < S; ++n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) xt[n].x[j] = make_uint4(0, 0, 0, 0);
    if (c_begin < c_end && n * TPN < v_end) load_x(xt[n], 0, n);
  }

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

  for (int c = c_begin; c < c_end; c += DEPTH) {
#pragma unroll
    for (int h = 0; h < 2 * MT; ++h) {
      pw[h] += DEPTH * ROW_CHUNK;
      if (EXACT && G > 1) ps[h] += DEPTH * G, pz[h] += DEPTH * G;
    }
    each<DEPTH>([&](auto I) {
      constexpr int i = decltype(I)::value;
      if (c + i < c_end) {
        Chunk<BITS, G, MT> &f = buf[i];
        constexpr int at_chunk = i;
        uint32_t q[2 * MT][16];
        float s[2 * MT];
        [[maybe_unused]] const int of_four = DEPTH == 4 ? i : (c + i - c_begin) & 3;
        if constexpr (G == 1) {
          if (of_four == 0) {
#pragma unroll
            for (int h = 0; h < 2 * MT; ++h) s4[h] = sn[h], z4[h] = zn[h];
            fetch_scales(c + i + 4);
          }
        }
#pragma unroll
        for (int h = 0; h < 2 * MT; ++h) {
          uint32_t zero;
          if constexpr (G == 1) {
            s[h] = __shfl_sync(~0u, s4[h], of_four, 4), zero = __shfl_sync(~0u, z4[h], of_four, 4);
          } else {
            s[h] = f.s[h], zero = f.z[h];
          }
          unpack<BITS>(f.w[h], q[h]);
          less_zero<BITS>(q[h], zero);
        }
        fetch(f, c + i + DEPTH, I);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (NT > 1 && n * TPN >= v_end) break;
          const uint4 *x = xt[n % S].x;
          const float2 fx = xt[n % S].f;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t *q0 = q[2 * m], *q1 = q[2 * m + 1];
            float d[4];
            mma0(d, q0[0], q1[0], q0[1], q1[1], x[0].x, x[0].y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j) mma(d, q0[4 * j], q1[4 * j], q0[4 * j + 1], q1[4 * j + 1], x[j].x, x[j].y);
              mma(d, q0[4 * j + 2], q1[4 * j + 2], q0[4 * j + 3], q1[4 * j + 3], x[j].z, x[j].w);
            }
            // d[0], d[1]: row g, columns 2t and 2t + 1, whose group is this lane's; d[2], d[3]: row g + 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              acc[m][n][2 * h] = fmaf(s[2 * m + h], d[2 * h] * fx.x, acc[m][n][2 * h]);
              acc[m][n][2 * h + 1] = fmaf(s[2 * m + h], d[2 * h + 1] * fx.y, acc[m][n][2 * h + 1]);
            }
          }
          if (n + S < NT && (n + S) * TPN < v_end) load_x(xt[n % S], at_chunk, n + S);
          else if (c + i + 1 < c_end) load_x(xt[n % S], at_chunk + 1, n % S);
        }
      }
    });
    xp += OWN ? DEPTH * 16 : (int64_t)DEPTH * tiles_of * (16 * TPN);
    xs += DEPTH * tiles_of * 4;
  }

  float *red = smem;  // [kWarps][G][v_most][ROWS]: the warps' sums
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (NT > 1 && n * TPN >= v_end) break;
    const int v = n * TPN + 2 * t % TPN;
    float *dst = red + ((warp * G + 2 * t / TPN) * v_most + v) * ROWS + g;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (v + j < v_end) dst[j * ROWS + m * 16] = acc[m][n][j], dst[j * ROWS + m * 16 + 8] = acc[m][n][2 + j];
  }
  const int rows_here = tiles_here * ROWS < a.d_out - row_first ? tiles_here * ROWS : a.d_out - row_first;
  if (a.y_ad) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the entries' sums
  __syncthreads();
  for (int i = threadIdx.x; i < tiles_here * ROWS * np; i += blockDim.x) {
    const int r = i % (tiles_here * ROWS), tok = i / (tiles_here * ROWS);
    if (r >= rows_here) continue;
    const float *src = red + (r / ROWS) * slices * G * v_most * ROWS + r % ROWS;
    float sum = 0.f;
    float by = 1.f;  // of the piece
    for (int v = tok * pieces; v < (tok + 1) * pieces; ++v, by *= 0x1p-11f) {
      float part = 0.f;
      for (int w = 0; w < slices * G; ++w) part += src[(w * v_most + v) * ROWS];
      sum = fmaf(part, by, sum);
    }
    if (!finite(sum)) sum = plain_dot(a, row_first + r, t0 + tok);
    if (a.y_ad) sum += a.alpha * a.y_ad[(int64_t)(row_first + r) * a.tp + t0 + tok];
    const int64_t at = (int64_t)(t0 + tok) * a.d_out + row_first + r;
    if (a.f32) static_cast<float *>(a.y)[at] = sum;
    else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(sum);
  }
}

template <int BITS, int G, int NT, int MT, int DEPTH, bool EXACT, bool OWN = false>
cudaError_t launch_one(const GemvArgs &a, cudaStream_t s) {
  constexpr int TPN = 8 / G, cols = NT * TPN, ROWS = 16 * MT;
  int tpp = cols / a.pieces;
  if (tpp < a.T) tpp &= ~(TPN - 1);  // a further pass starts with an n-tile
  else tpp = a.T;
  // slices of the columns: as many as it takes to give every SM twelve warps, two chunks a warp at least (a target of
  // 24 or 48 warps took 3 and 4 us more for 14336 x 4096, 3 bits)
  const int64_t tiles = cdiv(a.d_out, ROWS), chunks = cdiv(a.d_in, 128);
  int slices = 1;
  while (slices < kWarps && tiles * slices < (int64_t)sm_count() * 12 && chunks >= 2 * slices) slices *= 2;
  size_t smem = sizeof(float) * (size_t)kWarps * G * tpp * a.pieces * ROWS;
  if (OWN) smem += (size_t)a.T * a.pieces * (chunks * 16 + 4) * sizeof(uint4) + chunks * 32;
  auto kernel = gemv_mma_kernel<BITS, G, NT, MT, DEPTH, EXACT, OWN>;
  static std::atomic<size_t> allowed[64];
  const cudaError_t e = allow_smem((const void *)kernel, smem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cdiv(tiles, kWarps / slices), (unsigned)cdiv(a.T, tpp));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.prepared ? 1 : 0;  // overlaps the launches of its call before it
  return cudaLaunchKernelEx(&cfg, kernel, a, tpp, slices);
}

// The n-tiles a warp keeps: more tiles leave fewer registers to codes in flight,
// and each is worth its operands' latency less.
template <int BITS, int G, bool EXACT>
cudaError_t launch_cols(const GemvArgs &a, cudaStream_t s) {
  const int tiles = x_tiles(a.T * a.pieces, G);
  if (!a.xpieces) return launch_one<BITS, G, 1, 1, 4, EXACT, true>(a, s);
  if (tiles <= 1) return launch_one<BITS, G, 1, 1, 4, EXACT>(a, s);
  if (tiles <= 2) return launch_one<BITS, G, 2, 1, 2, EXACT>(a, s);
  if (tiles <= 4) return launch_one<BITS, G, 4, 1, 1, EXACT>(a, s);
  return launch_one<BITS, G, 8, 2, 1, EXACT>(a, s);
}

template <int BITS>
cudaError_t launch_bits(const GemvArgs &a, cudaStream_t s) {
  if (a.group == 128) return launch_cols<BITS, 1, true>(a, s);
  if (a.group == 64) return launch_cols<BITS, 2, true>(a, s);
  if (a.group == 32) return launch_cols<BITS, 4, true>(a, s);
  if (a.group % 128 == 0) return launch_cols<BITS, 1, false>(a, s);
  if (a.group % 64 == 0) return launch_cols<BITS, 2, false>(a, s);
  return launch_cols<BITS, 4, false>(a, s);
}

}  // namespace gemv
}  // namespace qwha
