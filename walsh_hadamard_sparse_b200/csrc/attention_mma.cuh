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
// A warp has one cached head and every so-manieth run of 16 tokens, by itself: a
// ring of stages that its own asynchronous copies fill, its own running maximum
// and sums; warps of a CTA meet only at the ends of segments. With as many warps
// as heads a CTA reads whole tokens, all heads of them, so the codes' 64-byte
// rows and the 4-byte scales and single zero points of a token come from the same
// sectors at about the same time.
//
// The maximum is not kept exactly: a tile raises it only where a score passes it
// by 2^5, which a vote finds out; shuffles and the scaling of the sums are left
// to those tiles.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attention.cuh"

namespace qwha {
namespace attn {

constexpr int kMmaWarps = 8;   // of a CTA, at most
constexpr int kStages = 3;     // of a warp's ring
constexpr int kTokens = 16;    // of a stage
constexpr float kSlack = 5.f;  // by how much (base 2) a score may pass the maximum
constexpr float kTop = 1024.f;  // p scale stays below this times 2^kSlack in f16
constexpr float kNoScale = 1.329227995784916e36f;  // 2^120: no scale met yet

// Sizes of a warp's stage and of a CTA's shared memory, in bytes.
struct MmaShape {
  int row_k, row_v;      // codes of a cached row
  int pitch_k, pitch_v;  // of a token in a stage
  int ng, words;         // groups of a head; words that cover their zero points
  int k_at, v_at, ks_at, vs_at, kz_at, vz_at, off_at, live_at, stage;
  int ring;              // of a warp: its stages, or a tile of its values
  int q_bytes;           // of a head: the queries as operands
  int fixed;             // zero points (and codes) begin at the same place of a word in every token
  __host__ __device__ MmaShape() {}
  __host__ __device__ static int pitch(int bytes, int bits) {
    // rows of a quarter warp on distinct banks: 16-byte (8 bits: 32-byte) steps, an odd number of them
    const int step = bits == 8 ? 32 : 16;
    return ((bytes + step - 1) / step | 1) * step;
  }
  __host__ __device__ MmaShape(int D, int dp, int bits_k, int bits_v, int group, int nt, int pieces, int heads) {
    row_k = D / 8 * bits_k, row_v = D / 8 * bits_v;
    // (the words that cover a row of 3-bit codes may be one more than it fills)
    pitch_k = pitch(dp / 8 * bits_k + (bits_k == 3 ? 4 : 0), bits_k);
    pitch_v = pitch(dp / 8 * bits_v + (bits_v == 3 ? 4 : 0), bits_v);
    ng = D / group, words = (ng + 3 + 3) / 4;
    fixed = heads * ng % 4 == 0 && row_k % 4 == 0 && row_v % 4 == 0;
    k_at = 0, v_at = k_at + kTokens * pitch_k;
    ks_at = v_at + kTokens * pitch_v, vs_at = ks_at + kTokens * ng * 4;
    kz_at = vs_at + kTokens * ng * 4, vz_at = kz_at + kTokens * words * 4;
    off_at = vz_at + kTokens * words * 4;  // bytes: where zero points (and codes of 3 bits) begin in their first word
    live_at = off_at + 2 * kTokens * 2;
    stage = (live_at + 4 + 15) / 16 * 16;
    const int values = 8 * (dp + 4) * 4;
    ring = kStages * stage > values ? kStages * stage : values;
    ring = (ring + 127) / 128 * 128;
    q_bytes = nt * pieces * (dp / 32) * 32 * 16;
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
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How the lanes of a warp fetch the rows of a stage's 16 tokens: pieces of 16, 8
// or 4 bytes, dealt to the lanes in order. (3-bit rows that are no multiple of
// four bytes: the words that cover them.)
struct Pieces {
  int tk, p, per, wide, step_t, step_p;
  __device__ __forceinline__ Pieces(int bytes, int bits) {
    wide = bits == 3 && bytes % 4 ? 0 : bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : 4;
    per = wide ? bytes / wide : bytes / 4 + 2;
    const int lane = threadIdx.x & 31;
    tk = lane / per, p = lane - tk * per;
    step_t = 32 / per, step_p = 32 - step_t * per;
  }
  template <int N>
  __device__ __forceinline__ void copy_wide(const uint8_t *row, uint32_t live, int from, uint32_t to, int pitch) const {
    int k = tk, q = p;
    for (int x = 0; x < kTokens * per; x += 32) {
      const uint8_t *r = reinterpret_cast<const uint8_t *>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(row), from + (k & 15)));
      if (k < kTokens && live >> k & 1) copy_async<N>(to + k * pitch + q * N, r + q * N);
      k += step_t, q += step_p;
      if (q >= per) q -= per, ++k;
    }
  }
  // row: the lane's token's codes; those of token 0 in lane `from`.
  __device__ __forceinline__ void copy(const uint8_t *row, uint32_t live, int from, uint32_t to, int bytes, int pitch,
                                       const qwha_cache &c) const {
    if (wide == 16) return copy_wide<16>(row, live, from, to, pitch);
    if (wide == 8) return copy_wide<8>(row, live, from, to, pitch);
    if (wide == 4) return copy_wide<4>(row, live, from, to, pitch);
    const uint8_t *end = c.codes + c.n_pages * c.page_size * c.heads * bytes;
    int k = tk, q = p;
    for (int x = 0; x < kTokens * per; x += 32) {
      const uint8_t *r = reinterpret_cast<const uint8_t *>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(row), from + (k & 15)));
      r = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(r) & ~(uintptr_t)3) + 4 * q;
      if (k < kTokens && live >> k & 1 && r < end) copy_async_part(to + k * pitch + 4 * q, r, end - r < 4 ? (int)(end - r) : 4);
      k += step_t, q += step_p;
      if (q >= per) q -= per, ++k;
    }
  }
};

// Minus the zero points of a pair as the subtrahends of the forms that a field of
// a half-word takes without a shift: 1024 + c, and with the field 2, 4 or 6 bits
// up (3-bit codes: 3 or 6) 1024 + 2^u c, of which 2^-u times leaves 2^(10-u) + c.
template <int BITS>
struct Zero {
  uint32_t z[4];
  // zz: 1024 + z, two f16
  __device__ __forceinline__ void set(uint32_t zz) {
    z[0] = zz ^ 0x80008000u;
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
__device__ __forceinline__ void unpack4(uint32_t x, const Zero<BITS> &z, uint32_t *out) {
  constexpr uint32_t kOne = 0x64006400u;
  auto field = [&](uint32_t w, uint32_t mask) { return (w & mask) | kOne; };
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
__device__ __forceinline__ uint32_t byte_pair(uint32_t a, uint32_t b, int i) {
  return (__byte_perm(a, b, 0x4000 + 0x0400 + i * 0x1111) & 0x00ff00ffu) | 0x64006400u;
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
__device__ __forceinline__ void unpack_row(uint2 c, const Zero<BITS> &z, uint32_t *out) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = hadd2(byte_pair(c.x, c.y, i), z.z[0]);
  } else {
    uint32_t x = c.x;
    if constexpr (BITS == 2) x = __byte_perm(x, 0, 0x4140);
    if constexpr (BITS == 3) x = (x & 0xfffu) | (x << 4 & 0x0fff0000u);
    unpack4<BITS>(x, z, out);
  }
}
// Tokens a and b side by side, channels 0..3 in out[0..3], 4..7 in out[4..7]: the
// second product's operand.
template <int BITS>
__device__ __forceinline__ void unpack_columns(uint2 a, uint2 b, const Zero<BITS> &z, uint32_t *out) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = hadd2(byte_pair(a.x, b.x, i), z.z[0]);
      out[4 + i] = hadd2(byte_pair(a.y, b.y, i), z.z[0]);
    }
  } else if constexpr (BITS == 4) {
    unpack4<4>(__byte_perm(a.x, b.x, 0x5410), z, out);
    unpack4<4>(__byte_perm(a.x, b.x, 0x7632), z, out + 4);
  } else if constexpr (BITS == 2) {
    const uint32_t x = __byte_perm(a.x, b.x, 0x5410);
    unpack4<2>(x, z, out);
    unpack4<2>(x >> 8, z, out + 4);
  } else {
    unpack4<3>((a.x & 0xfffu) | (b.x << 16 & 0x0fff0000u), z, out);
    unpack4<3>((a.x >> 12 & 0xfffu) | (b.x << 4 & 0x0fff0000u), z, out + 4);
  }
}

// The largest |s| of the warp as bits (finite ones; zero if none).
__device__ __forceinline__ uint32_t warp_max_bits(uint32_t v) { return __reduce_max_sync(~0u, v); }

template <int DP, int NT, int PIECES, bool MIXED>
__global__ void __launch_bounds__(kMmaWarps * 32, NT == 1 && DP <= 128 ? 2 : 1)
    attention_mma_kernel(const AttnArgs a, const MmaShape sh, int per_head) {
  extern __shared__ __align__(128) char smem[];
  constexpr int kSteps = DP / 32, kBlocks = DP / 64;
  constexpr bool kKeepQ = NT == 1 && kSteps * PIECES <= 8;
  __shared__ float c_s[kMmaWarps][32];                       // factor of the scales of each group
  __shared__ float m_s[kMmaWarps][8 * NT], l_s[kMmaWarps][8 * NT];  // of each warp's rows
  __shared__ float f_s[kMmaWarps][8 * NT];                   // by head: factor of a row's scores
  __shared__ uint8_t group_s[32];                            // of a chunk of eight channels
  __shared__ int lim_s[kMmaWarps][8 * NT];
  __shared__ unsigned long long bits_s[kMmaWarps][8 * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5;
  const int hl = warp / per_head, sub = warp - hl * per_head;  // head of the block; place among its warps
  char *ring = smem + warp * sh.ring;
  char *q_at = smem + warps * sh.ring + hl * sh.q_bytes;
  const int D = a.k.head_dim, ng = sh.ng, group = a.k.group;
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);

  Place at;
  long long left = my_share(a, &at);
  int4 begun = make_int4(0, 0, 0, 0), gone_on = begun;
  bool first = true;
  const bool upper = lane >> 4;
  const qwha_cache own = upper ? a.v : a.k;
  const int own_bytes = upper ? sh.row_v : sh.row_k;
  const int64_t slots = a.k.n_pages * a.k.page_size, zeros_end = slots * a.k.heads * ng;
  const Pieces pieces_k(sh.row_k, a.k.bits), pieces_v(sh.row_v, a.v.bits);
  if (MIXED && threadIdx.x < 32) group_s[threadIdx.x] = (uint8_t)min(8 * (int)threadIdx.x / group, ng - 1);
  while (left > 0) {
    const Seq s(a, at.b);
    if (s.rows == 0) {
      ++at.b;
      continue;
    }
    if (threadIdx.x == 0 && (long long)s.past + (a.tree && s.rows > 64 ? 64 : s.rows) > a.cap) atomicOr(a.err, kErrPage);
    const int units = s.units(a, at.tile), length = s.length(a, at.tile);
    const int block = at.block / a.parts, kv = block * a.hb + hl;
    const bool mine = kv < a.k.heads;  // (the last block may have fewer heads)
    const Rows rows = rows_of(a, s, kv, at.block % a.parts, at.tile);
    const int run = left < units - at.unit ? (int)left : units - at.unit;
    const int t_lo = at.unit * a.kt, t_hi = min(length, (at.unit + run) * a.kt);

    // ---- queries as operands: row r of the head by the warps of the head in turn
    __syncthreads();  // the last segment's values are read
    if (mine) {
      float *x = reinterpret_cast<float *>(ring);
      for (int r = sub; r < 8 * NT; r += per_head) {
        __syncwarp();
        float top = 0.f;
        for (int d = lane; d < DP; d += 32) x[d] = 0.f;
        __syncwarp();
        if (r < rows.n) {
          warp_query(a, x, rows.q_row(r), rows.q_head(r));
          for (int d = lane; d < D; d += 32) top = fmaxf(top, fabsf(x[d]));
        }
        const uint32_t bits = warp_max_bits(__float_as_uint(top));
        // 2^15 / 2^ceil: exact, the row's largest comes to lie in [2^14, 2^15]; infinities stay what they are
        int e = (int)(bits >> 23) - 127 + 1;
        e = bits == 0 || bits >= 0x7f800000u ? 0 : e < -100 ? -100 : e;
        const float up = __uint_as_float((uint32_t)(127 + 15 - e) << 23);
        uint4 *dst = reinterpret_cast<uint4 *>(q_at);
        if (lane < DP / 8) {  // chunk lane = 4 step + t of row r: operand lane (r & 7, t)
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = x[lane * 8 + i] * up;
          const int to = ((r >> 3) * kSteps + (lane >> 2)) * PIECES * 32 + (r & 7) * 4 + (lane & 3);
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pair16(v[i], v[i + 4]);
          dst[to] = make_uint4(w[0], w[1], w[2], w[3]);
          if constexpr (PIECES == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 h = wide16(w[i]);
              w[i] = pair16(v[i] - h.x, v[i + 4] - h.y);
            }
            dst[to + 32] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (lane == 0) {
          f_s[hl][r] = 1.f / up;
          const int j = rows.j0 + (r < rows.n ? r / rows.heads : 0);
          lim_s[hl][r] = r >= rows.n ? 0 : a.tree ? s.past : s.past + j + 1;
          bits_s[hl][r] = r < rows.n && a.tree ? (unsigned long long)a.tree[s.row0 + j] : 0;
        }
      }
    }
    __syncthreads();

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
    const uint4 *q_op = reinterpret_cast<const uint4 *>(q_at) + lane;
    uint4 q_keep[kKeepQ ? kSteps * PIECES : 1];
    if constexpr (kKeepQ) {
#pragma unroll
      for (int i = 0; i < kSteps * PIECES; ++i) q_keep[i] = q_op[i * 32];
    }
    const int z_in = kv * ng & 3;  // where a token's zero points begin in their first word, if it is the same for all
    const int safe = a.tree ? s.past : s.past + rows.j0 + 1;  // every row sees the tokens below

    // ---- the warp's runs of 16 tokens
    const int stride = per_head * kTokens, t_first = t_lo + sub * kTokens;
    const int tiles = mine && t_first < t_hi ? (t_hi - t_first + stride - 1) / stride : 0;
    const int32_t *table = a.pages + (int64_t)at.b * a.max_pages;
    auto look_up = [&](int i) -> int64_t {  // slot of the lane's token (lanes 16.. again) of tile i
      const int tok = t_first + i * stride + (lane & 15);
      if (i >= tiles || tok >= t_hi) return -1;
      const int pg = page_of(a, tok);  // within the table, since lengths are cut there
      return (int64_t)table[pg] * a.k.page_size + (tok - pg * a.k.page_size);  // pages outside: sorted out when used
    };
    int fill = 0;  // the stage that is filled next
    auto issue = [&](int i, int64_t slot) {
      const uint32_t st = ring_u + fill;
      fill = fill + sh.stage == kStages * sh.stage ? 0 : fill + sh.stage;
      if (i < tiles) {
        const int tok = t_first + i * stride + (lane & 15);
        bool on = tok < t_hi;
        if (on && (slot < 0 || slot >= slots)) {
          atomicOr(a.err, kErrPage);
          on = false;
        }
        const int64_t row = slot * a.k.heads + kv;
        const uint32_t live = __ballot_sync(~0u, on) & 0xffffu;
        // keys by the lower lanes, values by the upper: each has its token's row
        const uint8_t *mine_codes = own.codes + row * own_bytes;
        pieces_k.copy(mine_codes, live, 0, st + sh.k_at, sh.row_k, sh.pitch_k, a.k);
        pieces_v.copy(mine_codes, live, 16, st + sh.v_at, sh.row_v, sh.pitch_v, a.v);
        const uint32_t s_to = st + (upper ? sh.vs_at : sh.ks_at) + (lane & 15) * 4;
        char *off = ring + (st - ring_u) + sh.off_at + lane * 2;
        if (on) {
          const int64_t z = row * ng;
          for (int x = 0; x < ng; ++x) copy_async<4>(s_to + x * kTokens * 4, own.scales + z + x);
          const uint32_t z_to = st + (upper ? sh.vz_at : sh.kz_at) + (lane & 15) * sh.words * 4;
          const int in = (int)z & 3;
          for (int w = -in; w < ng; w += 4) {
            const int64_t rest = zeros_end - (z + w);
            copy_async_part(z_to + w + in, own.zeros + z + w, rest < 4 ? (int)rest : 4);
          }
          if (!sh.fixed) off[0] = (char)in, off[1] = (char)(own.bits == 3 ? row * own_bytes & 3 : 0);
        } else {
          for (int x = 0; x < ng; ++x) *reinterpret_cast<float *>(ring + (s_to - ring_u) + x * kTokens * 4) = 0.f;
          if (!sh.fixed) off[0] = off[1] = 0;
        }
        if (lane == 0) *reinterpret_cast<uint32_t *>(ring + (st - ring_u) + sh.live_at) = live;
      }
      copy_commit();
    };
    int use = 0;  // the stage that is used next
    int64_t slot = look_up(0);
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
      const int64_t next = look_up(i + 1);
      issue(i, slot);
      slot = next;
    }
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      copy_wait<kStages - 2>();
      __syncwarp();
      const int64_t next = look_up(i + kStages);
      issue(i + kStages - 1, slot);
      slot = next;
      const char *st = ring + use;
      use = use + sh.stage == kStages * sh.stage ? 0 : use + sh.stage;
      const int t0 = t_first + i * stride;
      const uint32_t live = *reinterpret_cast<const uint32_t *>(st + sh.live_at);
      const uint8_t *off = reinterpret_cast<const uint8_t *>(st) + sh.off_at;
      const float *ks = reinterpret_cast<const float *>(st + sh.ks_at);
      const float *vs = reinterpret_cast<const float *>(st + sh.vs_at);

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
        const uint8_t *z0 = reinterpret_cast<const uint8_t *>(st + sh.kz_at) + g * sh.words * 4, *z1 = z0 + 8 * sh.words * 4;
        int mis0 = 0, mis1 = 0;
        if (sh.fixed) {
          z0 += z_in, z1 += z_in;
        } else {
          z0 += off[2 * g], z1 += off[2 * (g + 8)];
          if (B == 3) mis0 = off[2 * g + 1], mis1 = off[2 * (g + 8) + 1];
        }
        const char *r0 = st + sh.k_at + g * sh.pitch_k, *r1 = r0 + 8 * sh.pitch_k;
        int gr = 0, edge = group;  // the group of the running sums, and where it ends
        Zero<B> za, zb;
        auto zeros = [&](int x) {
          za.set((z0[x] | 0x6400u) * 0x10001u), zb.set((z1[x] | 0x6400u) * 0x10001u);
        };
        if (!MIXED) zeros(0);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
          const int chunk = 4 * step + t;
          const int lane_group = MIXED ? group_s[chunk] : 0;
          if (MIXED) zeros(lane_group);
          uint32_t x[4], y[4];
          unpack_row<B>(load_run<B>(r0, chunk, mis0), za, x);
          unpack_row<B>(load_run<B>(r1, chunk, mis1), zb, y);
          const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
          for (;;) {  // once, where a step lies in one group
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < PIECES; ++p) {
                uint4 q;
                if constexpr (kKeepQ) q = q_keep[step * PIECES + p];
                else q = q_op[((n * kSteps + step) * PIECES + p) * 32];
                if (MIXED && lane_group != gr) q = make_uint4(0, 0, 0, 0);
                mma16816(part[n], a0, q.x, q.y);
                mma16816(part[n], a1, q.z, q.w);
              }
            const bool last = step + 1 == kSteps;
            if (edge > 32 * (step + 1) && !last) break;
            const float s0 = ks[gr * kTokens + g], s1 = ks[gr * kTokens + g + 8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              sc[n][0] = fmaf(part[n][0], s0, sc[n][0]), sc[n][1] = fmaf(part[n][1], s0, sc[n][1]);
              sc[n][2] = fmaf(part[n][2], s1, sc[n][2]), sc[n][3] = fmaf(part[n][3], s1, sc[n][3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) part[n][e] = 0.f;
            }
            if (gr + 1 == ng) break;
            ++gr;
            const bool more = edge < 32 * (step + 1);
            edge += group;
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
            const int r = 8 * n + 2 * t + (e & 1), tl = g + (e >> 1) * 8, tok = t0 + tl, u = tok - s.past;
            const bool on = (live >> tl & 1) && (tok < lim_s[hl][r] || (u >= 0 && u < 64 && (bits_s[hl][r] >> u & 1)));
            if (!on) sc[n][e] = -INFINITY;
            (e >> 1 ? any1 : any0) |= on;
          }
        unsigned b0 = __ballot_sync(~0u, any0), b1 = __ballot_sync(~0u, any1);
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
            thr[n][i] = (now + kSlack) / f[n][i];
            l[n][i] *= turn;
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
          float s0 = vs[gr * kTokens + g], s1 = vs[gr * kTokens + g + 8];
          if (masked) s0 = any0 ? s0 : 0.f, s1 = any1 ? s1 : 0.f;
          float c = c_s[warp][gr];
          const float x0 = fabsf(s0), x1 = fabsf(s1);
          const bool far0 = x0 * c > kTop && x0 < INFINITY, far1 = x1 * c > kTop && x1 < INFINITY;
          if (__any_sync(~0u, far0 || far1)) {  // a scale above all before it: twice its power of two
            const uint32_t top = warp_max_bits(max(far0 ? __float_as_uint(x0) : 0u, far1 ? __float_as_uint(x1) : 0u));
            int e = 127 + 10 - ((int)(top >> 23) - 127 + 2);
            e = e < 1 ? 1 : e > 247 ? 247 : e;
            const float now = __uint_as_float((uint32_t)e << 23), turn = now / c;
            c = now;
            __syncwarp();
            if (lane == 0) c_s[warp][gr] = now;
            __syncwarp();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
              if (min(8 * (8 * b + g) / group, ng - 1) == gr)
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
                const float2 a0 = wide16(lo), a1 = wide16(hi);
                v[0] -= a0.x, v[1] -= a0.y, v[2] -= a1.x, v[3] -= a1.y;
              }
            }
          }
        };
        const char *r[4];
        const uint8_t *z[4];
        int mis[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tk = 2 * t + (k & 1) + (k >> 1) * 8;
          r[k] = st + sh.v_at + tk * sh.pitch_v;
          z[k] = reinterpret_cast<const uint8_t *>(st + sh.vz_at) + tk * sh.words * 4 + (sh.fixed ? z_in : off[2 * (16 + tk)]);
          mis[k] = B == 3 && !sh.fixed ? off[2 * (16 + tk) + 1] : 0;
        }
        int have = -1, v_group = 0, v_edge = group;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const int chunk = 8 * b + g;
          if (b > 0 && 64 * b == v_edge && v_group + 1 < ng) ++v_group, v_edge += group;
          const int lane_group = MIXED ? group_s[chunk] : v_group;
          Zero<B> za, zb;
          za.set(z[0][lane_group] | (uint32_t)z[1][lane_group] << 16 | 0x64006400u);
          zb.set(z[2][lane_group] | (uint32_t)z[3][lane_group] << 16 | 0x64006400u);
          uint32_t x[8], y[8];
          unpack_columns<B>(load_run<B>(r[0], chunk, mis[0]), load_run<B>(r[1], chunk, mis[1]), za, x);
          unpack_columns<B>(load_run<B>(r[2], chunk, mis[2]), load_run<B>(r[3], chunk, mis[3]), zb, y);
          const int g0 = MIXED ? group_s[8 * b] : lane_group, g1 = MIXED ? group_s[8 * b + 7] : lane_group;
          for (int gr = g0; gr <= g1; ++gr) {
            if (MIXED || gr != have) weights(gr), have = gr;
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
      __syncwarp();  // the stage is read
    }
    copy_wait<0>();

    // ---- the warp's sums, and those of a head's warps together
    const bool starts = at.unit == 0, ends = at.unit + run == units;
    const int slot_out = 2 * blockIdx.x + (starts ? 1 : 0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) l[n][i] += __shfl_xor_sync(~0u, l[n][i], o);
        if (g == 0) m_s[warp][8 * n + 2 * t + i] = m[n][i], l_s[warp][8 * n + 2 * t + i] = l[n][i];
      }
    float *x = reinterpret_cast<float *>(ring);
    constexpr int kPitch = DP + 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      __syncthreads();
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const int c0 = 64 * b + 8 * g;
        const float back = 1.f / c_s[warp][min(c0 / group, ng - 1)];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[(2 * t + (e & 1)) * kPitch + c0 + k + 4 * (e >> 1)] = acc[b][k][n][e] * back;
      }
      __syncthreads();
      if (!mine) continue;
      for (int i = sub; i < 8; i += per_head) {
        const int r = 8 * n + i;
        if (r >= rows.n) break;
        float mm = -INFINITY, ll = 0.f;
        for (int w = hl * per_head; w < (hl + 1) * per_head; ++w) mm = fmaxf(mm, m_s[w][r]);
        const float base = mm == -INFINITY ? 0.f : mm;
        float v[DP / 32];
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) v[d] = 0.f;
        for (int w = hl * per_head; w < (hl + 1) * per_head; ++w) {
          const float turn = exp2_fast(m_s[w][r] - base);
          const float *o = reinterpret_cast<const float *>(smem + w * sh.ring) + i * kPitch;
          ll += l_s[w][r] * turn;
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) v[d] += o[lane + 32 * d] * turn;
        }
        if (starts && ends) {
          float *mine_row = x + i * kPitch;  // row i is read by this warp alone
          __syncwarp();
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) mine_row[lane + 32 * d] = v[d];
          __syncwarp();
          warp_finish(a, mine_row, mm, ll, rows.q_row(r), rows.q_head(r));
        } else {
          const int rr = hl * a.tq * a.gh + r;
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
            if (lane + 32 * d < D) piece_values(a, slot_out, rr)[lane + 32 * d] = v[d];
          if (lane == 0) piece_stats(a, slot_out, rr)[0] = mm, piece_stats(a, slot_out, rr)[1] = ll;
        }
      }
    }
    if (starts && !ends) begun = make_int4(at.b, at.block, at.tile, 1);
    if (!starts && first) gone_on = make_int4(at.b, at.block, at.tile, ends ? 3 : 1);
    first = false;
    left -= run;
    at.unit = 0;
    if (++at.tile == s.tiles) {
      at.tile = 0;
      if (++at.block == a.blocks) at.block = 0, ++at.b;
    }
  }
  if (threadIdx.x == 0) a.part_desc[2 * blockIdx.x] = gone_on, a.part_desc[2 * blockIdx.x + 1] = begun;
}

template <int DP, int NT, int PIECES, bool MIXED>
cudaError_t launch_mma(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  static std::atomic<size_t> allowed[64];
  auto kernel = attention_mma_kernel<DP, NT, PIECES, MIXED>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), l.smem, allowed);
  if (e != cudaSuccess) return e;
  const MmaShape sh(a.k.head_dim, DP, a.k.bits, a.v.bits, a.k.group, NT, PIECES, a.k.heads);
  kernel<<<l.ctas, l.warps * 32, l.smem, s>>>(a, sh, l.per_head);
  return cudaGetLastError();
}
template <int DP, int NT>
cudaError_t launch_mma_nt(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s) {
  const bool mixed = a.k.group != a.k.head_dim && a.k.group % 64;
  if (a.f32) return mixed ? launch_mma<DP, NT, 2, true>(a, l, s) : launch_mma<DP, NT, 2, false>(a, l, s);
  return mixed ? launch_mma<DP, NT, 1, true>(a, l, s) : launch_mma<DP, NT, 1, false>(a, l, s);
}

}  // namespace attn
}  // namespace qwha
