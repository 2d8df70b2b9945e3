// Attention over the quantized cache on tensor cores (mma.sync), for tiles of up
// to 32 rows of queries a cached head.
//
// Products are taken with the integers q - zero, exact in f16, and the scales
// stay outside, in fp32: a score is sum over groups of scale_g sum_d x_d (c_d -
// z_g), and a value enters as (p_t scale_tg) (c_td - z_tg). Cached tokens are the
// rows of the first product (S^T = C Q^T, 16 tokens, 8 queries a tile), channels
// the rows of the second (O^T = C^T P^T), so a lane unpacks codes straight into
// the operand's registers, whatever the number of queries, and P^T comes from S^T
// by one 8 x 8 transposition in registers. Rounded to f16 are the rotated query
// (11 bits of each value, scaled so that the row's largest is near 2^15) and p
// scale (11 bits, scaled to the largest scale met): 2^-12 each against the 2^-9
// of a bf16 output. fp32 calls carry both in two pieces, 22 bits.
//
// A warp has one cached head and 16 tokens of each stage, with its own running
// maximum and sums. The CTA's warps fill a ring of stages together with
// asynchronous copies: whole tokens, the rows of all the CTA's heads, so that the
// codes, the 4-byte scales and the single zero points of a token come in wide
// pieces, a thread always of the same token of the stage. With fewer heads than
// warps several warps share a head, and join their sums through shared memory at
// the end of a segment.
//
// The maximum is not kept exactly: a tile raises it only where a score passes it
// by 2^5, which a vote finds out; shuffles and the scaling of the sums are left
// to those tiles.
//
// Bound: instructions, not memory: 2.4 of 4 a clock, the ALU pipe, which unpacks,
// 47% busy, warps waiting for fixed latencies. 64 contexts of 4096 tokens, 8 heads of
// 128, 4 bits, one token each of 32 query heads take 98 us, 2.2 TB/s of the 6.5 that
// a copy moves; 8 contexts of 32768, keys of 4 and values of 2 bits, 120 us; one
// context of 700, 18 us, of which both launches' latencies are most.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attention.cuh"

namespace qwha {
namespace attn {

constexpr int kMmaWarps = 8;   // consumers of a CTA, at most
constexpr int kStages = 2;     // of the ring
constexpr int kTokens = 16;    // of a warp's tile
constexpr int kTilesPerStage = 2;  // of a warp
constexpr float kSlack = 5.f;  // by how much (base 2) a score may pass the maximum
constexpr float kTop = 1024.f;  // p scale stays below this times 2^kSlack in f16
constexpr float kNoScale = 1.329227995784916e36f;  // 2^120: no scale met yet

// A head of one group, of groups of whole 64-channel blocks, of any groups (keys and values of their own).
enum { kSingle, kBlocked, kMixed };

// An array of the cache in a stage: `bytes` of each token (`head` of each cached
// head), `stride` apart in memory, at `at` in the stage, `pitch` apart; fetched in
// `per` pieces of `wide` bytes. wide 0: a token's bytes begin anywhere in a word; the
// words that cover them are fetched, and where they begin in the first is kept per token.
struct Part {
  int head, bytes, stride, at, pitch, wide, per;
  // Pieces of a token's first `heads` heads. (The last block of cached heads may have
  // fewer than the others; what follows its last head is the next token, or behind the
  // last one nothing that may be read. `wide` divides both a block's bytes and a token's,
  // so what is left for the last block is whole pieces too.)
  __host__ __device__ int pieces(int heads) const { return wide ? heads * head / wide : (heads * head + 3 + 3) / 4; }
  __host__ __device__ void set(int head_, int hb, int heads, int step, int *end, int tokens) {
    head = head_, bytes = hb * head, stride = heads * head;
    wide = (bytes | stride) % 16 == 0 ? 16 : (bytes | stride) % 8 == 0 ? 8 : (bytes | stride) % 4 == 0 ? 4 : 0;
    per = pieces(hb);
    const int room = wide ? bytes : per * 4;
    // step: rows of a quarter warp on distinct banks (an odd number of steps apart)
    pitch = step ? ((room + step - 1) / step | 1) * step : room;
    at = *end;
    *end = (at + tokens * pitch + 15) / 16 * 16;
  }
};

constexpr int kMaxSmalls = 64;
// A piece of scales or zero points of the token in slot 0 and cached head 0.
struct alignas(16) Small {
  const char *from;
  uint32_t stride, to;  // of a slot; place of token 0 in a stage
  uint32_t head, pitch, wide;  // bytes of a head; from token to token in a stage
};

// A CTA's stages and shared memory, in bytes.
struct MmaShape {
  Part codes[2], scales[2], zeros[2];  // keys, values
  int row[2];                          // codes of a cached head's row
  int ng[2];                           // groups of a head
  int tokens;                          // of a stage
  int off_at, live_at, stage;          // off: 4 bytes a token, where its zero points and codes begin in their words
  int all_wide;                        // they begin at words in every token
  int smalls;                          // pieces of a token's scales and zero points
  int fast;                            // codes of a head in 16-byte pieces, scales and zero points in whole pieces
  int q_at, q_bytes;                   // queries as operands: after the ring; of a head
  int join_at, total;                  // where warps that share a head join
  __host__ __device__ MmaShape() {}
  __host__ __device__ MmaShape(int D, int dp, int bits_k, int bits_v, int group_k, int group_v, int nt, int pieces, int heads, int hb,
                               int per_head, int warps) {
    const int bits[2] = {bits_k, bits_v};
    ng[0] = D / group_k, ng[1] = D / group_v, tokens = kTokens * kTilesPerStage * per_head;
    int end = 0;
    for (int i = 0; i < 2; ++i) {
      row[i] = D / 8 * bits[i];
      codes[i].set(row[i], hb, heads, bits[i] == 8 ? 32 : 16, &end, tokens);
      end += 48;  // the last chunks of padded channels, and of 3 bits, are read past the row's end
      end = (end + dp / 8 * bits[i] - row[i] + 15) / 16 * 16;
    }
    for (int i = 0; i < 2; ++i) scales[i].set(ng[i] * 4, hb, heads, 0, &end, tokens);
    for (int i = 0; i < 2; ++i) zeros[i].set(ng[i], hb, heads, 0, &end, tokens);
    all_wide = codes[0].wide && codes[1].wide && zeros[0].wide && zeros[1].wide;
    smalls = scales[0].per + scales[1].per + zeros[0].per + zeros[1].per;
    fast = all_wide && row[0] % 16 == 0 && row[1] % 16 == 0 && smalls <= kMaxSmalls;
    off_at = end, live_at = off_at + tokens * 4;
    stage = (live_at + tokens + 15) / 16 * 16;
    q_at = kStages * stage;
    q_bytes = nt * pieces * (dp / 32) * 32 * 16;
    join_at = q_at + hb * q_bytes;
    total = join_at + (per_head > 1 ? warps * 8 * (dp + 4) * 4 : 0);
  }
};

__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 wide16(uint32_t v) { return __half22float2(reinterpret_cast<const __half2 &>(v)); }
__device__ __forceinline__ float exp2_fast(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// 1 / x of a power of two
__device__ __forceinline__ float inverse2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// Four bytes of which the last ones may lie outside the array: n are read, zeros follow.
__device__ __forceinline__ void copy_async_part(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Fetches a token's bytes of one array, n pieces: piece i and every `step`-th after it.
// src: where the token's bytes begin; dst: its place in the stage.
template <int N>
__device__ __forceinline__ void fetch_wide(int n, const char *src, uint32_t dst, int i, int step) {
  for (; i < n; i += step) copy_async<N>(dst + i * N, src + i * N);
}
__device__ __forceinline__ void fetch(const Part &p, int n, const char *src, const char *end, uint32_t dst, int i, int step) {
  if (p.wide == 16) return fetch_wide<16>(n, src, dst, i, step);
  if (p.wide == 8) return fetch_wide<8>(n, src, dst, i, step);
  if (p.wide == 4) return fetch_wide<4>(n, src, dst, i, step);
  src -= reinterpret_cast<uintptr_t>(src) & 3;
  for (; i < n; i += step)
    if (src + 4 * i < end) copy_async_part(dst + 4 * i, src + 4 * i, end - (src + 4 * i) < 4 ? (int)(end - (src + 4 * i)) : 4);
}
// All arrays of a token, whatever the format. Returns where zero points and codes
// begin in their words. (Not inlined: the kernel's usual path is short.)
static __device__ __noinline__ uint32_t fetch_any(const AttnArgs &a, const MmaShape &sh, uint32_t slot, int kv0, uint32_t to,
                                           int token, int piece, int step) {
  uint32_t off = 0;
  const int64_t slots = a.k.n_pages * a.k.page_size;
  const int here = a.k.heads - kv0;
  auto count = [&](const Part &p) { return here >= a.hb ? p.per : p.pieces(here); };
  for (int i = 0; i < 2; ++i) {
    const qwha_cache &c = i ? a.v : a.k;
    const char *codes = reinterpret_cast<const char *>(c.codes), *zeros = reinterpret_cast<const char *>(c.zeros);
    const char *code_end = codes + slots * sh.codes[i].stride, *zero_end = zeros + slots * sh.zeros[i].stride;
    codes += (int64_t)slot * sh.codes[i].stride + kv0 * sh.row[i];
    zeros += (int64_t)slot * sh.zeros[i].stride + kv0 * sh.ng[i];
    const char *scales = reinterpret_cast<const char *>(c.scales) + (int64_t)slot * sh.scales[i].stride + kv0 * sh.ng[i] * 4;
    fetch(sh.codes[i], count(sh.codes[i]), codes, code_end, to + sh.codes[i].at + token * sh.codes[i].pitch, piece, step);
    fetch(sh.scales[i], count(sh.scales[i]), scales, nullptr, to + sh.scales[i].at + token * sh.scales[i].pitch, piece, step);
    fetch(sh.zeros[i], count(sh.zeros[i]), zeros, zero_end, to + sh.zeros[i].at + token * sh.zeros[i].pitch, piece, step);
    if (!sh.zeros[i].wide) off |= (uint32_t)(reinterpret_cast<uintptr_t>(zeros) & 3) << (8 * i);
    if (!sh.codes[i].wide) off |= (uint32_t)(reinterpret_cast<uintptr_t>(codes) & 3) << (16 + 8 * i);
  }
  return off;
}

// Minus the zero points of a pair as the subtrahends of the forms that a field of
// a half-word takes without a shift: 1024 + c, and with the field 2, 4 or 6 bits
// up (3-bit codes: 3 or 6) 1024 + 2^u c, of which 2^-u times leaves 2^(10-u) + c.
template <int BITS>
struct Zero {
  uint32_t z[4];
  // zz: -(1024 + z), two f16
  __device__ __forceinline__ void set(uint32_t zz) {
    z[0] = zz;
    if constexpr (BITS == 4) z[1] = hadd2(z[0], 0x63806380u);  // - (64 + z): + 960
    if constexpr (BITS == 3) {
      z[1] = hadd2(z[0], 0x63006300u);  // - (128 + z): + 896
      z[2] = hadd2(z[0], 0x63e063e0u);  // - (16 + z): + 1008
    }
    if constexpr (BITS == 2) {
      z[1] = hadd2(z[0], 0x62006200u);  // - (256 + z): + 768
      z[2] = hadd2(z[0], 0x63806380u);  // - (64 + z)
      z[3] = hadd2(z[0], 0x63e063e0u);  // - (16 + z): + 1008
    }
  }
};

// Codes of eight channels as fields of two half-words, field i at bit BITS i: x.
// The pair i (c - z) of both halves.
template <int BITS>
__device__ __forceinline__ void unpack4(uint32_t x, const Zero<BITS> &z, uint32_t one, uint32_t *out) {
  // one: 0x64006400 in a register, so that mask and or are one instruction
  auto field = [&](uint32_t w, uint32_t mask) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(one));
    return d;
  };
  if constexpr (BITS == 4) {
    out[0] = hadd2(field(x, 0x000f000fu), z.z[0]);
    out[1] = hfma2(field(x, 0x00f000f0u), 0x2c002c00u, z.z[1]);
    x >>= 8;
    out[2] = hadd2(field(x, 0x000f000fu), z.z[0]);
    out[3] = hfma2(field(x, 0x00f000f0u), 0x2c002c00u, z.z[1]);
  } else if constexpr (BITS == 2) {
    out[0] = hadd2(field(x, 0x00030003u), z.z[0]);
    out[1] = hfma2(field(x, 0x000c000cu), 0x34003400u, z.z[1]);
    out[2] = hfma2(field(x, 0x00300030u), 0x2c002c00u, z.z[2]);
    out[3] = hfma2(field(x, 0x00c000c0u), 0x24002400u, z.z[3]);
  } else if constexpr (BITS == 3) {
    out[0] = hadd2(field(x, 0x00070007u), z.z[0]);
    out[1] = hfma2(field(x, 0x00380038u), 0x30003000u, z.z[1]);
    out[2] = hfma2(field(x, 0x01c001c0u), 0x24002400u, z.z[2]);
    out[3] = hadd2(field(x >> 9, 0x00070007u), z.z[0]);
  }
}
__device__ __forceinline__ uint32_t byte_pair(uint32_t a, uint32_t b, int i, uint32_t one) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(__byte_perm(a, b, 0x4400 + i * 0x1111)), "r"(0x00ff00ffu), "r"(one));
  return d;
}

// A group whose codes all equal its zero point is zeros whatever its scale (a row of zeros is stored with scale 1): idle.
// Byte i (word k) of codes that all are z; z above every code is no code.
template <int BITS>
__device__ __forceinline__ uint32_t idle_byte(uint32_t z, int i) {
  if constexpr (BITS == 8) return z;
  if constexpr (BITS == 4) return z * 0x11u;
  if constexpr (BITS == 2) return z * 0x55u;
  return z * 0x249249u >> (8 * (i % 3)) & 0xffu;
}
template <int BITS>
__device__ __forceinline__ uint32_t idle_word(uint32_t z, int k) {
  if constexpr (BITS == 8) return z * 0x01010101u;
  if constexpr (BITS == 4) return z * 0x11111111u;
  if constexpr (BITS == 2) return z * 0x55555555u;
  return k == 0 ? z * 0x49249249u : k == 1 ? z >> 2 | z * 0x92492492u : z >> 1 | z * 0x24924924u;
}
// Of `bytes` codes from `at` on, every `step`-th byte from i on.
template <int BITS, typename P>
__device__ __forceinline__ bool idle_bytes(const P *at, int bytes, uint32_t z, int i, int step) {
  bool same = z < 1u << BITS;
#pragma unroll 1
  for (; same && i < bytes; i += step) same = (uint8_t)at[i] == idle_byte<BITS>(z, i);
  return same;
}
// Eight codes of a row in shared memory: two words of which 8 bits use both.
template <int BITS>
__device__ __forceinline__ uint2 load_run(const char *row, int chunk, int mis) {
  if constexpr (BITS == 8) return *reinterpret_cast<const uint2 *>(row + 8 * chunk);
  if constexpr (BITS == 4) return make_uint2(*reinterpret_cast<const uint32_t *>(row + 4 * chunk), 0);
  if constexpr (BITS == 2) return make_uint2(*reinterpret_cast<const uint16_t *>(row + 2 * chunk), 0);
  const int at = 3 * chunk + mis;
  const uint32_t *w = reinterpret_cast<const uint32_t *>(row + (at & ~3));
  return make_uint2(__funnelshift_r(w[0], w[1], 8 * (at & 3)), 0);
}

// Channels of a row in the pairs (i, i + 4), i < 4: the first product's operand.
template <int BITS>
__device__ __forceinline__ void unpack_row(uint2 c, const Zero<BITS> &z, uint32_t one, uint32_t *out) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = hadd2(byte_pair(c.x, c.y, i, one), z.z[0]);
  } else {
    uint32_t x = c.x;
    if constexpr (BITS == 2) x = __byte_perm(x, 0, 0x4140);
    if constexpr (BITS == 3) x = (x & 0xfffu) | (x << 4 & 0x0fff0000u);
    unpack4<BITS>(x, z, one, out);
  }
}
// Tokens a and b side by side, channels 0..3 in out[0..3], 4..7 in out[4..7]: the
// second product's operand.
template <int BITS>
__device__ __forceinline__ void unpack_columns(uint2 a, uint2 b, const Zero<BITS> &z, uint32_t one, uint32_t *out) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = hadd2(byte_pair(a.x, b.x, i, one), z.z[0]);
      out[4 + i] = hadd2(byte_pair(a.y, b.y, i, one), z.z[0]);
    }
  } else if constexpr (BITS == 4) {
    unpack4<4>(__byte_perm(a.x, b.x, 0x5410), z, one, out);
    unpack4<4>(__byte_perm(a.x, b.x, 0x7632), z, one, out + 4);
  } else if constexpr (BITS == 2) {
    const uint32_t x = __byte_perm(a.x, b.x, 0x5410);
    unpack4<2>(x, z, one, out);
    unpack4<2>(x >> 8, z, one, out + 4);
  } else {
    unpack4<3>((a.x & 0xfffu) | (b.x << 16 & 0x0fff0000u), z, one, out);
    unpack4<3>((a.x >> 12 & 0xfffu) | (b.x << 4 & 0x0fff0000u), z, one, out + 4);
  }
}

// x H (blocks of had) for rows that lie over L lanes, eight consecutive channels
// each.
template <int L>
__device__ __forceinline__ void rotate_lanes(float *v, int had, float unit, int lane) {
  if (had < 2) return;
  auto inside = [&](int h) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & h)) {
        const float x = v[i], y = v[i + h];
        v[i] = x + y, v[i + h] = x - y;
      }
  };
  inside(1);
  if (had >= 4) inside(2);
  if (had >= 8) inside(4);
#pragma unroll
  for (int o = 1; o < L; o *= 2)
    if (had > 8 * o) {
      const float sign = lane & o ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], sign, __shfl_xor_sync(~0u, v[i], o));
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= unit;
}

// IDLE: idle groups have no say in the factor of the scales. Where a row may see less than
// another of its tile, such a scale (a row of zeros is stored with 1) would take bits
// from all of them, or have them done again in fp32; with one token to a sequence it
// is one of those that the row sees, and looking costs 2 to 8%.
template <int DP, int NT, int PIECES, int GROUPS, bool IDLE>
__global__ void __launch_bounds__(kMmaWarps * 32, NT == 1 && DP <= 128 ? 2 : 1)
    attention_mma_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ MmaShape sh, int per_head, uint32_t one) {
  extern __shared__ __align__(128) char smem[];
  constexpr int kSteps = DP / 32, kBlocks = DP / 64;
  constexpr bool MIXED = GROUPS == kMixed;
  __shared__ float c_s[kMmaWarps][32];                              // factor of the scales of each group
  __shared__ float m_s[kMmaWarps][8 * NT], l_s[kMmaWarps][8 * NT];  // of each warp's rows
  __shared__ float f_s[kMmaWarps][8 * NT];                          // by head: factor of a row's scores
  __shared__ Small small_s[kMaxSmalls];
  __shared__ Rows rows_s[kMmaWarps];                                // kept out of the loop's registers
  __shared__ uint8_t group_s[2][32];                                  // of a chunk of eight channels
  __shared__ int lim_s[kMmaWarps][8 * NT];
  __shared__ unsigned long long bits_s[kMmaWarps][8 * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5, D = a.k.head_dim;
  const int ng_k = sh.ng[0], group_k = a.k.group, ng_v = MIXED ? sh.ng[1] : ng_k, group_v = MIXED ? a.v.group : group_k;
  if (MIXED)
    for (int x = threadIdx.x; x < 64; x += blockDim.x)
      group_s[x >> 5][x & 31] = (uint8_t)min(8 * (x & 31) / (x >> 5 ? group_v : group_k), sh.ng[x >> 5] - 1);
  Place at;
  long long left = my_share(a, &at);
  __syncthreads();
  const int kt = 1 << a.kt_log2;
  const int hl = per_head == 1 ? warp : warp / per_head, sub = warp - hl * per_head;  // head of the block; place among its warps
  char *q_at = smem + sh.q_at + hl * sh.q_bytes;
  auto meet = [&] {  // the warps that share a head
    if (per_head > 1) __syncthreads();
    else __syncwarp();
  };
  if (threadIdx.x == 0) a.part_desc[2 * blockIdx.x] = a.part_desc[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  // what the thread fetches: of one token of each stage, every fetch_step-th piece
  const int fetch_step = a.hb, fetch_token = threadIdx.x / fetch_step, fetch_piece = threadIdx.x - fetch_token * fetch_step;
  const uint32_t slots = (uint32_t)(a.k.n_pages * a.k.page_size);
  const uint32_t smem_u = (uint32_t)__cvta_generic_to_shared(smem);
  if (sh.fast && threadIdx.x == 0) {
    int n = 0;
    for (int i = 0; i < 4; ++i) {
      const Part &x = i < 2 ? sh.scales[i] : sh.zeros[i - 2];
      const qwha_cache &c = i & 1 ? a.v : a.k;
      const char *from = i < 2 ? reinterpret_cast<const char *>(c.scales) : reinterpret_cast<const char *>(c.zeros);
      for (int p = 0; p < x.per; ++p)
        small_s[n++] = {from + p * x.wide, (uint32_t)x.stride, (uint32_t)(x.at + p * x.wide), (uint32_t)x.head, (uint32_t)x.pitch, (uint32_t)x.wide};
    }
  }
  __syncthreads();
  const uint32_t k_to = sh.codes[0].at + fetch_token * sh.codes[0].pitch + fetch_piece * 16;
  const uint32_t v_to = sh.codes[1].at + fetch_token * sh.codes[1].pitch + fetch_piece * 16;
  // the lane's tokens and head in a stage's parts
  const int k_row = sh.codes[0].at + (kTokens * kTilesPerStage * sub + g) * sh.codes[0].pitch + hl * sh.row[0];
  const int k_scale = sh.scales[0].at + (kTokens * kTilesPerStage * sub + g) * sh.scales[0].pitch + hl * ng_k * 4;
  const int v_scale = sh.scales[1].at + (kTokens * kTilesPerStage * sub + g) * sh.scales[1].pitch + hl * ng_v * 4;
  const int k_zero = sh.zeros[0].at + (kTokens * kTilesPerStage * sub + g) * sh.zeros[0].pitch + hl * ng_k;
  const int v_row = sh.codes[1].at + (kTokens * kTilesPerStage * sub + 2 * t) * sh.codes[1].pitch + hl * sh.row[1];
  const int v_zero = sh.zeros[1].at + (kTokens * kTilesPerStage * sub + 2 * t) * sh.zeros[1].pitch + hl * ng_v;
  while (left > 0) {
    const Seq s(a, at.b);
    if (s.rows == 0) {
      ++at.b;
      continue;
    }
    const int units = s.units(a, at.tile), past = s.past;
    if (threadIdx.x == 0 && (long long)s.past + (a.tree && s.rows > 64 ? 64 : s.rows) > a.cap) atomicOr(a.err, kErrPage);
    const int length = s.length(a, at.tile), block = block_of(a, at.block), kv0 = block * a.hb, kv = kv0 + hl;
    const bool mine = kv < a.k.heads;  // (the last block may have fewer heads)
    Rows rows = rows_of(a, s, mine ? kv : 0, at.block - block * a.parts, at.tile);
    const int run = left < units - at.unit ? (int)left : units - at.unit;

    // ---- the ring: stage j of the segment holds the tokens from (at.unit + j) kt on
    const int32_t *table = a.pages + (int64_t)at.b * a.max_pages;
    int fetch_t = at.unit * kt + fetch_token;
    const char *k_from = reinterpret_cast<const char *>(a.k.codes) + kv0 * sh.row[0] + fetch_piece * 16;
    const char *v_from = reinterpret_cast<const char *>(a.v.codes) + kv0 * sh.row[1] + fetch_piece * 16;
    // the page of token t, which is within the table, since lengths are cut there; and its place in the page
    auto page_at = [&](int t, int *in) -> int {
      const int pg = page_of(a, t);
      *in = t - pg * a.k.page_size;
      return t < length ? table[pg] : -2;
    };
    int fill_at = 0;
    auto fill = [&](int page, int in) {
      const bool on = (uint32_t)page < (uint32_t)a.k.n_pages;
      if (page != -2 && !on) atomicOr(a.err, kErrPage);
      const uint32_t slot = (uint32_t)page * (uint32_t)a.k.page_size + (uint32_t)in, to = smem_u + fill_at;
      uint32_t off = 0;
      if (on && sh.fast && kv0 + fetch_step <= a.k.heads) {
        // a block that has all its heads (one that has fewer goes by fetch_any, which costs it 6 to 9%: a count of pieces
        // here took 2 to 3% from all calls);
        // pieces p, p + fetch_step, ... of a token's codes; a row has whole pieces
        auto codes = [&](const char *src, uint32_t dst, int n) {
          const int step = 16 * fetch_step;
          for (; n >= 4; n -= 4, src += 4 * step, dst += 4 * step)
#pragma unroll
            for (int p = 0; p < 4; ++p) copy_async<16>(dst + p * step, src + p * step);
          if (n & 2) {
            copy_async<16>(dst, src), copy_async<16>(dst + step, src + step);
            src += 2 * step, dst += 2 * step;
          }
          if (n & 1) copy_async<16>(dst, src);
        };
        codes(k_from + (uint64_t)slot * (uint32_t)sh.codes[0].stride, to + k_to, sh.row[0] >> 4);
        codes(v_from + (uint64_t)slot * (uint32_t)sh.codes[1].stride, to + v_to, sh.row[1] >> 4);
        for (int q = fetch_piece; q < sh.smalls; q += fetch_step) {
          const Small &x = small_s[q];
          const char *src = x.from + (uint64_t)slot * x.stride + kv0 * x.head;
          const uint32_t dst = to + x.to + fetch_token * x.pitch;
          if (x.wide == 16) copy_async<16>(dst, src);
          else if (x.wide == 8) copy_async<8>(dst, src);
          else copy_async<4>(dst, src);
        }
      } else if (on) {
        off = fetch_any(a, sh, slot, kv0, to, fetch_token, fetch_piece, fetch_step);
      } else {  // codes and zero points are finite whatever they are; scales have to be
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int x = fetch_piece; x < a.hb * (i ? ng_v : ng_k); x += fetch_step)
            reinterpret_cast<float *>(smem + fill_at + sh.scales[i].at + fetch_token * sh.scales[i].pitch)[x] = 0.f;
      }
      if (fetch_piece == 0) {
        if (!sh.all_wide) *reinterpret_cast<uint32_t *>(smem + fill_at + sh.off_at + fetch_token * 4) = off;
        smem[fill_at + sh.live_at + fetch_token] = on;
      }
      fill_at = fill_at + sh.stage == kStages * sh.stage ? 0 : fill_at + sh.stage;
    };
    int pages[kStages], ins[kStages];  // of the token's next stages, on their way while the ones before are filled
#pragma unroll
    for (int i = 0; i < kStages; ++i) pages[i] = page_at(fetch_t + i * kt, &ins[i]);
    fetch_t += kStages * kt;  // of the stage after these
    __syncthreads();  // the last segment's stages are read
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < run) fill(pages[i], ins[i]);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int next_page = pages[kStages - 1], next_in = ins[kStages - 1];

    // ---- queries as operands: rows of a head by its warps in turn, 32 / L at once
    constexpr int L = DP / 8, kAtOnce = 32 / L;
    meet();  // the last segment's queries and masks are read
    constexpr int kPasses = 8 * NT / kAtOnce < 4 ? 8 * NT / kAtOnce : 4;  // whose loads are under way together
    const int c = lane % L;                                                // chunk of eight channels
#pragma unroll 1
    for (int p0 = 0; p0 * kAtOnce * per_head < 8 * NT; p0 += kPasses) {
    uint4 raw[kPasses][2];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = ((p0 + p) * per_head + sub) * kAtOnce + lane / L;
      raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
      if (r < rows.n && c * 8 < D) {
        const int64_t from = rows.q_row(r) * a.q_stride + (int64_t)rows.q_head(r) * D + c * 8;
        const uint4 *src = a.f32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) + from)
                                 : reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + from);
        raw[p][0] = __ldg(src);
        if (a.f32) raw[p][1] = __ldg(src + 1);
      }
    }
#pragma unroll 1
    for (int p = 0; p < kPasses; ++p) {
      const int r = ((p0 + p) * per_head + sub) * kAtOnce + lane / L;
      uint4 x = raw[0][0], y = raw[0][1];
#pragma unroll
      for (int i = 1; i < kPasses; ++i)
        if (p == i) x = raw[i][0], y = raw[i][1];
      const int r_first = ((p0 + p) * per_head + sub) * kAtOnce;
      if (r_first >= 8 * NT) break;
      uint4 *dst = reinterpret_cast<uint4 *>(q_at) + ((r >> 3) * kSteps + (c >> 2)) * PIECES * 32 + (r & 7) * 4 + (c & 3);
      if (r_first >= rows.n) {  // rows that the tile does not have
#pragma unroll
        for (int i = 0; i < PIECES; ++i) dst[32 * i] = make_uint4(0, 0, 0, 0);
        if (c == 0) f_s[hl][r] = 1.f, lim_s[hl][r] = 0, bits_s[hl][r] = 0;
        continue;
      }
      float v[8];
      if (a.f32) io<float>::unpack(x, v), io<float>::unpack(y, v + 4);
      else io<__nv_bfloat16>::unpack(x, v);
      rotate_lanes<L>(v, a.k.had_block, a.unit_k, lane);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= a.scale2, top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int o = 1; o < L; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      // 2^15 / 2^ceil: exact, the row's largest comes to lie in [2^14, 2^15]; infinities stay what they are
      const uint32_t bits = __float_as_uint(top);
      int e = (int)(bits >> 23) - 127 + 1;
      e = bits == 0 || bits >= 0x7f800000u ? 0 : e < -100 ? -100 : e;
      const float up = __uint_as_float((uint32_t)(127 + 15 - e) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= up;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pair16(v[i], v[i + 4]);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (PIECES == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 h = wide16(w[i]);
          w[i] = pair16(v[i] - h.x, v[i + 4] - h.y);
        }
        dst[32] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (c == 0) {
        f_s[hl][r] = __uint_as_float((uint32_t)(127 - 15 + e) << 23);  // 1 / up
        const int j = rows.j0 + (r < rows.n ? r / rows.heads : 0);
        lim_s[hl][r] = r >= rows.n ? 0 : a.tree ? s.past : s.past + j + 1;
        bits_s[hl][r] = r < rows.n && a.tree ? (unsigned long long)a.tree[s.row0 + j] : 0;
      }
    }
    }
    meet();

    float acc[kBlocks][4][NT][4], m[NT][2], l[NT][2], f[NT][2], thr[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[n][i] = -INFINITY, l[n][i] = 0.f, thr[n][i] = -INFINITY;
        f[n][i] = f_s[hl][8 * n + 2 * t + i];
      }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b][i][n][e] = 0.f;
    c_s[warp][lane] = kNoScale;
    __syncwarp();
    const uint4 *q_op = reinterpret_cast<const uint4 *>(q_at) + lane;
    const int safe = a.tree ? past : past + rows.j0 + 1;  // every row sees the tokens below
    int t_stage = at.unit * kt + kTokens * kTilesPerStage * sub, use_at = 0;
    __syncwarp();
    if (lane == 0) rows_s[warp] = rows;

#pragma unroll 1
    for (int u = 0; u < run; ++u, t_stage += kt) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();  // stage u has landed, and all have read stage u - 1
      const char *stage = smem + use_at;
      use_at = use_at + sh.stage == kStages * sh.stage ? 0 : use_at + sh.stage;
      if (u + kStages - 1 < run) {
        const int page = next_page, in = next_in;
        next_page = page_at(fetch_t, &next_in);
        fetch_t += kt;
        fill(page, in);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
      for (int h = 0; h < kTilesPerStage; ++h) {
        const int t0 = t_stage + kTokens * h;
        if (t0 >= length || !mine) break;
        // the tile in the stage's parts
        const char *st_k = stage + h * kTokens * sh.codes[0].pitch, *st_v = stage + h * kTokens * sh.codes[1].pitch;
        const char *st_ks = stage + h * kTokens * sh.scales[0].pitch, *st_vs = stage + h * kTokens * sh.scales[1].pitch;
        const char *st_kz = stage + h * kTokens * sh.zeros[0].pitch, *st_vz = stage + h * kTokens * sh.zeros[1].pitch;
        const int first_token = kTokens * (kTilesPerStage * sub + h);
        // a byte a token: whether it is there
        const uint32_t live = __ballot_sync(~0u, stage[sh.live_at + first_token + (lane & 15)]) & 0xffffu;
        const uint8_t *off = reinterpret_cast<const uint8_t *>(stage) + sh.off_at + 4 * first_token;  // of the tile's tokens

        // ---- scores of tokens g, g + 8 for queries 2 t, 2 t + 1 of each tile
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
        auto scores = [&](auto bits) {
          constexpr int B = decltype(bits)::value;
          float part[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[n][e] = 0.f;
          const char *r0 = st_k + k_row, *r1 = r0 + 8 * sh.codes[0].pitch;
          const uint8_t *z0 = reinterpret_cast<const uint8_t *>(st_kz) + k_zero, *z1 = z0 + 8 * sh.zeros[0].pitch;
          const float *s0 = reinterpret_cast<const float *>(st_ks + k_scale);
          const float *s1 = reinterpret_cast<const float *>(st_ks + k_scale + 8 * sh.scales[0].pitch);
          int mis0 = 0, mis1 = 0;
          if (!sh.zeros[0].wide) z0 += off[4 * g], z1 += off[4 * g + 32];
          if (B == 3 && !sh.codes[0].wide) {
            mis0 = (int)((off[4 * g + 2] + reinterpret_cast<uintptr_t>(r0)) & 3), r0 += off[4 * g + 2] - mis0;
            mis1 = (int)((off[4 * g + 34] + reinterpret_cast<uintptr_t>(r1)) & 3), r1 += off[4 * g + 34] - mis1;
          } else if (B == 3) {
            mis0 = (int)(reinterpret_cast<uintptr_t>(r0) & 3), r0 -= mis0;
            mis1 = (int)(reinterpret_cast<uintptr_t>(r1) & 3), r1 -= mis1;
          }
          int gr = 0, edge = group_k;  // the group of the running sums, and where it ends
          Zero<B> za, zb;
          auto zeros = [&](int x) {
            za.set((z0[x] | 0xe400u) * 0x10001u), zb.set((z1[x] | 0xe400u) * 0x10001u);
          };
          if (!MIXED) zeros(0);
#pragma unroll
          for (int step = 0; step < kSteps; ++step) {
            const int chunk = 4 * step + t;
            const int lane_group = MIXED ? group_s[0][chunk] : 0;
            if (MIXED) zeros(lane_group);
            uint32_t x[4], y[4];
            unpack_row<B>(load_run<B>(r0, chunk, mis0), za, one, x);
            unpack_row<B>(load_run<B>(r1, chunk, mis1), zb, one, y);
            const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
            for (;;) {  // once, where a step lies in one group
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                  uint4 q = q_op[((n * kSteps + step) * PIECES + p) * 32];
                  if (MIXED && lane_group != gr) q = make_uint4(0, 0, 0, 0);
                  mma16816(part[n], a0, q.x, q.y);
                  mma16816(part[n], a1, q.z, q.w);
                }
              const bool last = step + 1 == kSteps;
              if (GROUPS == kSingle ? !last : edge > 32 * (step + 1) && !last) break;
              const float f0 = s0[gr], f1 = s1[gr];
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                sc[n][0] = fmaf(part[n][0], f0, sc[n][0]), sc[n][1] = fmaf(part[n][1], f0, sc[n][1]);
                sc[n][2] = fmaf(part[n][2], f1, sc[n][2]), sc[n][3] = fmaf(part[n][3], f1, sc[n][3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) part[n][e] = 0.f;
              }
              if (GROUPS == kSingle || gr + 1 == ng_k) break;
              ++gr;
              const bool more = edge < 32 * (step + 1);
              edge += group_k;
              if (!MIXED) zeros(gr);
              if (!MIXED || !more) break;
            }
          }
        };
        switch (a.k.bits) {
          case 2: scores(std::integral_constant<int, 2>()); break;
          case 3: scores(std::integral_constant<int, 3>()); break;
          case 4: scores(std::integral_constant<int, 4>()); break;
          default: scores(std::integral_constant<int, 8>());
        }

        // ---- masks
        const bool masked = live != 0xffffu || t0 + kTokens > safe;
        bool any0 = true, any1 = true;  // whether any row sees token g, g + 8
        if (masked) {
          any0 = any1 = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 8 * n + 2 * t + (e & 1), tl = g + (e >> 1) * 8, tok = t0 + tl, w = tok - past;
              const bool on = (live >> tl & 1) && (tok < lim_s[hl][r] || (w >= 0 && w < 64 && (bits_s[hl][r] >> w & 1)));
              if (!on) sc[n][e] = -INFINITY;
              (e >> 1 ? any1 : any0) |= on;
            }
          const unsigned b0 = __ballot_sync(~0u, any0), b1 = __ballot_sync(~0u, any1);
          any0 = b0 >> (4 * g) & 15u, any1 = b1 >> (4 * g) & 15u;
        }

        // ---- the maximum, where a score has passed it by 2^kSlack
        bool passed = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) passed |= sc[n][e] > thr[n][e & 1];
        if (__any_sync(~0u, passed)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = fmaxf(sc[n][i], sc[n][i + 2]);
#pragma unroll
              for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
              const float now = fmaxf(m[n][i], top * f[n][i]);
              const float turn = now == -INFINITY ? 1.f : exp2_fast(m[n][i] - now);
              m[n][i] = now;
              thr[n][i] = (now + kSlack) * inverse2(f[n][i]);
              l[n][i] *= turn;
              if (u + h > 0)
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                  for (int k = 0; k < 4; ++k) acc[b][k][n][i] *= turn, acc[b][k][n][i + 2] *= turn;
            }
        }
        // ---- weights
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float base = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
            sc[n][e] = exp2_fast(fmaf(sc[n][e], f[n][e & 1], -base));
            l[n][e & 1] += sc[n][e];
          }

        // ---- values: channels 64 b + 8 g + i and + 4, tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        auto add_values = [&](auto bits) {
          constexpr int B = decltype(bits)::value;
          uint32_t w[NT][PIECES][2];  // weights times scales of the group, as operands
          auto weights = [&](int gr) {
            float s0 = reinterpret_cast<const float *>(st_vs + v_scale)[gr];
            float s1 = reinterpret_cast<const float *>(st_vs + v_scale + 8 * sh.scales[1].pitch)[gr];
            if (masked) s0 = any0 ? s0 : 0.f, s1 = any1 ? s1 : 0.f;
            float c = c_s[warp][gr];
            if (__any_sync(~0u, fabsf(s0) * c > kTop || fabsf(s1) * c > kTop)) {
              if constexpr (IDLE) {  // four lanes look at a group's codes
                auto idle = [&](int tk) {
                  const int back = g - 2 * t + tk;  // v_row, v_zero: of token 2 t
                  const char *row = st_v + v_row + back * sh.codes[1].pitch + gr * (group_v / 8 * B);
                  const uint8_t *zero = reinterpret_cast<const uint8_t *>(st_vz) + v_zero + back * sh.zeros[1].pitch + gr;
                  const uint8_t *o = off + 4 * (g + tk);
                  if (!sh.codes[1].wide) row += o[3];
                  if (!sh.zeros[1].wide) zero += o[1];
                  bool same = idle_bytes<B>(row, group_v / 8 * B, *zero, t, 4);
                  same &= __shfl_xor_sync(~0u, same, 1);
                  return same & __shfl_xor_sync(~0u, same, 2);
                };
                const bool idle0 = idle(0), idle1 = idle(8);
                if (idle0 && fabsf(s0) < INFINITY) s0 = 0.f;
                if (idle1 && fabsf(s1) < INFINITY) s1 = 0.f;
              }
              // a scale above all before it: twice its power of two. Infinities stay what they are
              const float x0 = fabsf(s0), x1 = fabsf(s1);
              const uint32_t top = __reduce_max_sync(~0u, max(x0 < INFINITY ? __float_as_uint(x0) : 0u, x1 < INFINITY ? __float_as_uint(x1) : 0u));
              int e = 127 + 10 - ((int)(top >> 23) - 127 + 2);
              e = e < 1 ? 1 : e > 247 ? 247 : e;
              const float now = fminf(c, __uint_as_float((uint32_t)e << 23)), turn = now * inverse2(c);
              c = now;
              __syncwarp();
              if (lane == 0) c_s[warp][gr] = now;
              __syncwarp();
              if (u + h > 0)
#pragma unroll
              for (int b = 0; b < kBlocks; ++b)
                if (GROUPS == kSingle || min(8 * (8 * b + g) / group_v, ng_v - 1) == gr)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                      for (int x = 0; x < 4; ++x) acc[b][k][n][x] *= turn;
            }
            s0 *= c, s1 *= c;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float v[4] = {sc[n][0] * s0, sc[n][1] * s0, sc[n][2] * s1, sc[n][3] * s1};
              if (masked)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = sc[n][e] == 0.f ? 0.f : v[e];  // the scale may be a NaN
#pragma unroll
              for (int p = 0; p < PIECES; ++p) {
                const uint32_t lo = pair16(v[0], v[1]), hi = pair16(v[2], v[3]);
                w[n][p][0] = turn8x8(lo), w[n][p][1] = turn8x8(hi);
                if (p + 1 < PIECES) {
                  const float2 h0 = wide16(lo), h1 = wide16(hi);
                  v[0] -= h0.x, v[1] -= h0.y, v[2] -= h1.x, v[3] -= h1.y;
                }
              }
            }
          };
          const char *r[4];
          const uint8_t *z[4];
          int mis[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tk = (k & 1) + (k >> 1) * 8;
            r[k] = st_v + v_row + tk * sh.codes[1].pitch;
            z[k] = reinterpret_cast<const uint8_t *>(st_vz) + v_zero + tk * sh.zeros[1].pitch;
            const uint8_t *o = off + 4 * (2 * t + tk);
            if (!sh.zeros[1].wide) z[k] += o[1];
            mis[k] = 0;
            if (B == 3) {
              if (!sh.codes[1].wide) r[k] += o[3];
              mis[k] = (int)(reinterpret_cast<uintptr_t>(r[k]) & 3), r[k] -= mis[k];
            }
          }
          int have = -1, v_group = 0, v_edge = group_v;
          Zero<B> za, zb;
          auto zeros = [&](int x) {
            za.set(z[0][x] | (uint32_t)z[1][x] << 16 | 0xe400e400u);
            zb.set(z[2][x] | (uint32_t)z[3][x] << 16 | 0xe400e400u);
          };
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int chunk = 8 * b + g;
            if (GROUPS == kBlocked && b > 0 && 64 * b == v_edge) ++v_group, v_edge += group_v;
            const int lane_group = MIXED ? group_s[1][chunk] : v_group;
            if (MIXED || (GROUPS == kSingle ? b == 0 : lane_group != have)) zeros(lane_group);
            uint32_t x[8], y[8];
            unpack_columns<B>(load_run<B>(r[0], chunk, mis[0]), load_run<B>(r[1], chunk, mis[1]), za, one, x);
            unpack_columns<B>(load_run<B>(r[2], chunk, mis[2]), load_run<B>(r[3], chunk, mis[3]), zb, one, y);
            const int g0 = MIXED ? group_s[1][8 * b] : lane_group, g1 = MIXED ? group_s[1][8 * b + 7] : lane_group;
            for (int gr = g0; gr <= g1; ++gr) {
              if (MIXED || (GROUPS == kSingle ? b == 0 : gr != have)) weights(gr), have = gr;
              const uint32_t keep = !MIXED || lane_group == gr ? ~0u : 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t op[4] = {x[k] & keep, x[k + 4] & keep, y[k] & keep, y[k + 4] & keep};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int p = 0; p < PIECES; ++p) mma16816(acc[b][k][n], op, w[n][p][0], w[n][p][1]);
              }
            }
          }
        };
        switch (a.v.bits) {
          case 2: add_values(std::integral_constant<int, 2>()); break;
          case 3: add_values(std::integral_constant<int, 3>()); break;
          case 4: add_values(std::integral_constant<int, 4>()); break;
          default: add_values(std::integral_constant<int, 8>());
        }
      }
    }

    // ---- the rows' sums: of the warp, then of the warps that share the head
    __syncwarp();
    rows = rows_s[warp];
    const bool starts = at.unit == 0, ends = at.unit + run == units;
    const int slot_out = 2 * blockIdx.x + (starts ? 1 : 0);
    float back[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) back[b] = inverse2(c_s[warp][GROUPS == kSingle ? 0 : min(8 * (8 * b + g) / group_v, ng_v - 1)]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 4; o < 32; o *= 2) l[n][i] += __shfl_xor_sync(~0u, l[n][i], o);
    // eight channels 64 b + 8 g .. of query 2 t + i
    auto chunk_of = [&](int b, int n, int i, float *v) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[b][k][n][i] * back[b], v[k + 4] = acc[b][k][n][i + 2] * back[b];
    };
    auto store_piece = [&](int r, int c0, const float *v, float mm, float ll) {
      const int rr = hl * a.tq * a.gh + r;
      if (c0 < D) {
        float4 *dst = reinterpret_cast<float4 *>(piece_values(a, slot_out, rr) + c0);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]), dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      if (c0 == 0) piece_stats(a, slot_out, rr)[0] = mm, piece_stats(a, slot_out, rr)[1] = ll;
    };
    if (per_head == 1) {
      if (mine) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * n + 2 * t + i;
            float v[kBlocks][8];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) chunk_of(b, n, i, v[b]);
            if (starts && ends) {
              const float inv = l[n][i] == 0.f ? 0.f : 1.f / l[n][i];
              // H: channels' bits 0..2 within a chunk, 3..5 over the lanes g, 6 and 7 over the blocks
              const int had = a.v.had_block;
#pragma unroll
              for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[b][k] *= inv;
                rotate_lanes<1>(v[b], had, a.unit_v, 0);
#pragma unroll
                for (int o = 1; o < 8; o *= 2)
                  if (had > 8 * o) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                      v[b][k] = fmaf(v[b][k], g & o ? -1.f : 1.f, __shfl_xor_sync(~0u, v[b][k], 4 * o));
                  }
              }
#pragma unroll
              for (int o = 1; o < kBlocks; o *= 2)
                if (had > 64 * o)
#pragma unroll
                  for (int b = 0; b < kBlocks; ++b)
                    if (!(b & o))
#pragma unroll
                      for (int k = 0; k < 8; ++k) {
                        const float x = v[b][k], y = v[b + o][k];
                        v[b][k] = x + y, v[b + o][k] = x - y;
                      }
              if (r < rows.n) {
                const int64_t row = rows.q_row(r), head = rows.q_head(r);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                  const int c0 = 64 * b + 8 * g;
                  if (c0 >= D) continue;
                  const int64_t to = (row * a.q_heads + head) * D + c0;
                  if (a.f32) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + to);
                    dst[0] = io<float>::pack(v[b]), dst[1] = io<float>::pack(v[b] + 4);
                  } else {
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to) = io<__nv_bfloat16>::pack(v[b]);
                  }
                }
                if (a.lse && g == 0) a.lse[row * a.q_heads + head] = l[n][i] == 0.f ? -INFINITY : (m[n][i] + log2f(l[n][i])) * kLn2;
              }
            } else if (r < rows.n) {
#pragma unroll
              for (int b = 0; b < kBlocks; ++b) store_piece(r, 64 * b + 8 * g, v[b], m[n][i], l[n][i]);
            }
          }
      }
    } else {
      constexpr int kPitch = DP + 4;
      float *x = reinterpret_cast<float *>(smem + sh.join_at) + warp * 8 * kPitch;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        meet();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (g == 0) m_s[warp][8 * n + 2 * t + i] = m[n][i], l_s[warp][8 * n + 2 * t + i] = l[n][i];
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            float v[8];
            chunk_of(b, n, i, v);
            float4 *dst = reinterpret_cast<float4 *>(x + (2 * t + i) * kPitch + 64 * b + 8 * g);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]), dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        meet();
        for (int i = sub; i < 8; i += per_head) {
          const int r = 8 * n + i;
          if (!mine || r >= rows.n) break;
          float mm = -INFINITY, ll = 0.f;
          for (int w = hl * per_head; w < (hl + 1) * per_head; ++w) mm = fmaxf(mm, m_s[w][r]);
          const float base = mm == -INFINITY ? 0.f : mm;
          float v[DP / 32];
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) v[d] = 0.f;
          for (int w = 0; w < per_head; ++w) {
            const float turn = exp2_fast(m_s[hl * per_head + w][r] - base);
            const float *o = x + ((w - sub) * 8 + i) * kPitch;
            ll += l_s[hl * per_head + w][r] * turn;
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) v[d] += o[lane + 32 * d] * turn;
          }
          if (starts && ends) {
            float *own = x + i * kPitch;  // row i is read by this warp alone
            __syncwarp();
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) own[lane + 32 * d] = v[d];
            __syncwarp();
            warp_finish(a, own, mm, ll, rows.q_row(r), rows.q_head(r));
          } else {
            const int rr = hl * a.tq * a.gh + r;
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
              if (lane + 32 * d < D) piece_values(a, slot_out, rr)[lane + 32 * d] = v[d];
            if (lane == 0) piece_stats(a, slot_out, rr)[0] = mm, piece_stats(a, slot_out, rr)[1] = ll;
          }
        }
      }
    }
    if (threadIdx.x == 0 && !(starts && ends)) a.part_desc[slot_out] = make_int4(at.b, at.block, at.tile, ends ? kPieceThere | kPieceEnds : kPieceThere);
    left -= run;
    at.unit = 0;
    if (rows.j0 + a.tq >= rows.all) {  // the sequence's last tile
      at.tile = 0;
      if (++at.block == a.blocks) at.block = 0, ++at.b;
    } else {
      ++at.tile;
    }
  }
}

template <int DP, int NT, int PIECES, int GROUPS, bool IDLE>
cudaError_t launch_mma(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  static std::atomic<size_t> allowed[64];
  auto kernel = attention_mma_kernel<DP, NT, PIECES, GROUPS, IDLE>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), l.smem, allowed);
  if (e != cudaSuccess) return e;
  const MmaShape sh(a.k.head_dim, DP, a.k.bits, a.v.bits, a.k.group, a.v.group, NT, PIECES, a.k.heads, a.hb, l.per_head, l.warps);
  kernel<<<l.ctas, l.warps * 32, l.smem, s>>>(a, sh, l.per_head, 0x64006400u);
  return cudaGetLastError();
}
template <int DP, int NT, int PIECES, bool IDLE>
cudaError_t launch_mma_groups(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  const bool alike = a.k.group == a.v.group;
  if (alike && a.k.group == a.k.head_dim) return launch_mma<DP, NT, PIECES, kSingle, IDLE>(a, l, s);
  if (alike && a.k.group % 64 == 0) return launch_mma<DP, NT, PIECES, kBlocked, IDLE>(a, l, s);
  return launch_mma<DP, NT, PIECES, kMixed, IDLE>(a, l, s);
}
template <int DP, int NT, int PIECES>
cudaError_t launch_mma_pieces(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  // one token to a sequence is the rule only with few rows: no other copies of the kernel
  if (NT == 1 && a.tq == 1) return launch_mma_groups<DP, NT, PIECES, NT != 1>(a, l, s);
  return launch_mma_groups<DP, NT, PIECES, true>(a, l, s);
}
template <int DP, int NT>
cudaError_t launch_mma_nt(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  return a.f32 ? launch_mma_pieces<DP, NT, 2>(a, l, s) : launch_mma_pieces<DP, NT, 1>(a, l, s);
}

}  // namespace attn
}  // namespace qwha
