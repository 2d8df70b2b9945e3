// Attention over the quantized cache: the kernel for every format, the joining of
// tiles that were cut between CTAs, and the choice of the kernels.

#include <algorithm>

#include "attention_mma.cuh"

namespace qwha {
namespace {

using namespace attn;

// ---------------------------------------------------------------- every format

constexpr int kAnyThreads = 128, kAnyRows = 8, kAnyTokens = 32;

__device__ __forceinline__ void unpack_run(const uint8_t *p, float *q, int bits) {
  const uint32_t mask = (1u << bits) - 1u;
  uint32_t w = 0, hi = 0;
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
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = (float)((w >> (bits * i)) & mask);
}

// scale (code - zero) of eight codes of a row.
__device__ __forceinline__ void load_values(const qwha_cache &c, int64_t row, int run, float *v) {
  unpack_run(c.codes + row * (c.head_dim / 8 * c.bits) + run * c.bits, v, c.bits);
  const int64_t group = row * (c.head_dim / c.group) + run * 8 / c.group;
  const float s = c.scales[group], z = (float)c.zeros[group];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s * (v[i] - z);
}

// One cached head and up to eight rows of queries a tile: 32 tokens at a time go
// to shared memory as fp32 values; lane t of a warp holds the scores of token t
// for the warp's two rows, a thread the values of one or two channels. Bound by
// its shared-memory reads: 64 contexts of 4096 tokens, 8 heads of 128, take 2.9 ms
// where the kernels below take 0.1. It has what those leave: heads whose 2-bit codes
// are no whole words, and caches of 2^31 slots.
__global__ void __launch_bounds__(kAnyThreads) attention_any_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) float smem[];
  const int D = a.k.head_dim, pitch = D + 4;
  float *q_s = smem;                          // [8][D]
  float *k_s = q_s + kAnyRows * D;            // [32][D + 4]
  float *v_s = k_s + kAnyTokens * pitch;      // [32][D]
  float *p_s = v_s + kAnyTokens * D;          // [8][32]
  __shared__ float m_s[kAnyRows], l_s[kAnyRows], turn_s[kAnyRows];
  __shared__ int64_t slot_s[kAnyTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Place at;
  long long left = my_share(a, &at);
  int4 begun = make_int4(0, 0, 0, 0), gone_on = begun;
  bool first = true;
  while (left > 0) {
    const Seq s(a, at.b);
    if (s.rows == 0) {
      ++at.b;
      continue;
    }
    if (threadIdx.x == 0 && (long long)s.past + (a.tree && s.rows > 64 ? 64 : s.rows) > a.cap) atomicOr(a.err, kErrPage);
    const int kv = block_of(a, at.block), units = s.units(a, at.tile), length = s.length(a, at.tile);
    const Rows rows = rows_of(a, s, kv, at.block - block_of(a, at.block) * a.parts, at.tile);
    const int run = left < units - at.unit ? (int)left : units - at.unit;
    __syncthreads();
    for (int r = warp; r < kAnyRows; r += kAnyThreads / 32) {
      if (r < rows.n) warp_query(a, q_s + r * D, rows.q_row(r), rows.q_head(r));
      if (lane == 0) m_s[r] = -INFINITY, l_s[r] = 0.f;
    }
    float acc[2][kAnyRows];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < kAnyRows; ++r) acc[i][r] = 0.f;
    for (int u = at.unit; u < at.unit + run; ++u) {
      const int t0 = u * kAnyTokens;
      __syncthreads();
      if (threadIdx.x < kAnyTokens) slot_s[threadIdx.x] = t0 + (int)threadIdx.x < length ? slot_of(a, at.b, t0 + threadIdx.x) : -1;
      __syncthreads();
      for (int i = threadIdx.x; i < kAnyTokens * (D / 8); i += kAnyThreads) {
        const int t = i / (D / 8), c = i - t * (D / 8);
        float k[8], v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
        if (slot_s[t] >= 0) {
          load_values(a.k, slot_s[t] * a.k.heads + kv, c, k);
          load_values(a.v, slot_s[t] * a.k.heads + kv, c, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) k_s[t * pitch + c * 8 + e] = k[e], v_s[t * D + c * 8 + e] = v[e];
      }
      __syncthreads();
      for (int r = warp * 2; r < warp * 2 + 2; ++r) {
        float x = 0.f;
        for (int d = 0; d < D; ++d) x = fmaf(q_s[r * D + d], k_s[lane * pitch + d], x);
        bool on = r < rows.n && slot_s[lane] >= 0;
        if (on) {
          const int j = rows.j0 + r / rows.heads;
          on = s.sees(a, j, a.tree ? (unsigned long long)a.tree[s.row0 + j] : 0, t0 + lane);
        }
        // a score that is not a number stays one; a masked one counts nothing
        float top = on ? x : -INFINITY;
#pragma unroll
        for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float old = m_s[r], m = fmaxf(old, top), base = m == -INFINITY ? 0.f : m;
        const float p = on ? exp2f(x - base) : 0.f;
        float sum = p;
#pragma unroll
        for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
        p_s[r * kAnyTokens + lane] = p;
        __syncwarp();
        if (lane == 0) {
          const float f = exp2f(old - base);
          turn_s[r] = f, m_s[r] = m, l_s[r] = l_s[r] * f + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = threadIdx.x + i * kAnyThreads;
        if (d >= D) break;
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) acc[i][r] *= turn_s[r];
        for (int t = 0; t < kAnyTokens; ++t) {
          if (slot_s[t] < 0) continue;
          const float v = v_s[t * D + d];
#pragma unroll
          for (int r = 0; r < kAnyRows; ++r) {
            const float p = p_s[r * kAnyTokens + t];
            if (p != 0.f) acc[i][r] = fmaf(p, v, acc[i][r]);  // a masked value may be a NaN
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = threadIdx.x + i * kAnyThreads;
      if (d < D)
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) q_s[r * D + d] = acc[i][r];
    }
    __syncthreads();
    const bool starts = at.unit == 0, ends = at.unit + run == units;
    const int slot = 2 * blockIdx.x + (starts ? 1 : 0);
    for (int r = warp; r < rows.n; r += kAnyThreads / 32) {
      if (starts && ends) {
        warp_finish(a, q_s + r * D, m_s[r], l_s[r], rows.q_row(r), rows.q_head(r));
      } else {
        for (int d = lane; d < D; d += 32) piece_values(a, slot, r)[d] = q_s[r * D + d];
        if (lane == 0) piece_stats(a, slot, r)[0] = m_s[r], piece_stats(a, slot, r)[1] = l_s[r];
      }
    }
    if (starts && !ends) begun = make_int4(at.b, at.block, at.tile, 1);
    if (!starts && first) gone_on = make_int4(at.b, at.block, at.tile, ends ? kPieceThere | kPieceEnds : kPieceThere);
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

// ---------------------------------------------------------------- joining

// The tile that CTA blockIdx.x of the kernel before began and left: its piece and
// those of the CTAs that went on with it, in order. L lanes have a row, eight
// channels each; they look at L pieces' maxima and sums at once and read the values
// of four pieces ahead. Bound by the latency of those loads: 15 us of the 343 that 4
// chunks of 1021 tokens behind 2048 take.
constexpr int kJoinThreads = 256, kJoinRows = 32, kJoinAhead = 4;
template <int L>
__global__ void __launch_bounds__(kJoinThreads, 4) attention_join_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ Rows rows_s;
  __shared__ int count_s;
  extern __shared__ int slots_s[];  // the pieces
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (it waits for this launch before it writes)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int4 begun = a.part_desc[2 * c + 1];
  if (!(begun.w & kPieceThere)) return;
  const int part = begun.y - block_of(a, begun.y) * a.parts, kv0 = block_of(a, begun.y) * a.hb, each = a.tq * a.gh;
  if (threadIdx.x < 32) {
    int n = 1;
    if (lane == 0) slots_s[0] = 2 * c + 1;
    for (int p0 = c + 1; p0 < a.ctas; p0 += 32) {
      const int p = p0 + lane, flags = p < a.ctas ? a.part_desc[2 * p].w : 0;  // 0: a CTA without units
      const unsigned ends = __ballot_sync(~0u, flags & kPieceEnds), upto = ends ? (ends & -ends) * 2 - 1 : ~0u;
      const unsigned on = __ballot_sync(~0u, flags & kPieceThere) & upto;
      if (on >> lane & 1) slots_s[n + __popc(on & ((1u << lane) - 1))] = 2 * p;
      n += __popc(on);
      if (ends) break;
    }
    if (lane == 0) count_s = n;
  } else if (threadIdx.x == 32) {
    const Seq s(a, begun.x);
    rows_s = rows_of(a, s, 0, part, begun.z);
  }
  __syncthreads();
  const Rows rows = rows_s;
  const int count = count_s, at = threadIdx.x % L, c0 = 8 * at, D = a.v.head_dim;
#pragma unroll 1
  for (int i = threadIdx.x / L; i < kJoinRows; i += kJoinThreads / L) {
    const int rr = blockIdx.y * kJoinRows + i, hl = rr / each, r = rr - hl * each;
    const bool real = rr < a.part_rows && kv0 + hl < a.k.heads && r < rows.n;
    float m = -INFINITY, l = 0.f, v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    if (__any_sync(~0u, real)) {
      for (int p0 = 0; p0 < count; p0 += L) {
        const int n = count - p0 < L ? count - p0 : L;
        const int slot = slots_s[p0 + (at < n ? at : 0)];
        const bool mine = real && at < n;
        const float2 st = mine ? *reinterpret_cast<const float2 *>(piece_stats(a, slot, rr)) : make_float2(-INFINITY, 0.f);
        float top = fmaxf(m, st.x);
#pragma unroll
        for (int o = 1; o < L; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // a NaN is dropped from the maximum, but the sums carry it
        const float base = top == -INFINITY ? 0.f : top, turn = exp2f(m - base), w = mine ? exp2f(st.x - base) : 0.f;
        float sum = mine ? st.y * w : 0.f;
#pragma unroll
        for (int o = 1; o < L; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
        l = l * turn + sum, m = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= turn;
        for (int p = 0; p < n; p += kJoinAhead) {
          float4 x[kJoinAhead][2];
#pragma unroll
          for (int u = 0; u < kJoinAhead; ++u)
            if (p + u < n && real && c0 < D) {
              const float4 *src = reinterpret_cast<const float4 *>(piece_values(a, slots_s[p0 + p + u], rr) + c0);
              x[u][0] = src[0], x[u][1] = src[1];
            }
#pragma unroll
          for (int u = 0; u < kJoinAhead; ++u) {
            const float f = __shfl_sync(~0u, w, (p + u) % L, L);
            if (p + u < n && real && c0 < D && f != 0.f) {
              const float4 y = x[u][0], z = x[u][1];
              v[0] = fmaf(y.x, f, v[0]), v[1] = fmaf(y.y, f, v[1]), v[2] = fmaf(y.z, f, v[2]), v[3] = fmaf(y.w, f, v[3]);
              v[4] = fmaf(z.x, f, v[4]), v[5] = fmaf(z.y, f, v[5]), v[6] = fmaf(z.z, f, v[6]), v[7] = fmaf(z.w, f, v[7]);
            }
          }
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
      rotate_lanes<L>(v, a.v.had_block, a.unit_v, lane);
    }
    if (!real || c0 >= D) continue;
    const int64_t row = rows.q_row(r), head = rows.q_head(r) + (kv0 + hl) * a.grp, to = (row * a.q_heads + head) * D + c0;
    if (a.f32) {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + to);
      dst[0] = io<float>::pack(v), dst[1] = io<float>::pack(v + 4);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to) = io<__nv_bfloat16>::pack(v);
    }
    if (a.lse && at == 0) a.lse[row * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// ---------------------------------------------------------------- repairing

// The tensor-core kernels keep scales in f16, relative to the largest met.
// attention_mma.cuh has p scale, of which 2^-33 of the largest is a step. A row that does
// not see the token of the largest scale has the less room for its own: tiles where
// tokens that not all rows see have scales 2^8 times the others' are done again in fp32,
// so that a token costs 2^-25 of a row's own at most.
// attention_tc.cu has the scales of keys and values themselves, which lose bits from 2^-13
// of the largest on, whoever sees it. It tells where it met such; tiles with scales that far
// apart are done again.
// Caches of values of ordinary spread have none of these. A third launch looks while the
// second runs (on mma.sync, which cannot tell: 2 us for 2 trees of 2 behind 1024, 4 for 64
// behind 4096).
// (The same in the kernels themselves took registers and instruction cache from them:
// 325 to 375 us for 304 where four chunks of 1021 tokens are answered behind 2048.)
constexpr float kRoomMma = 256.f;

// Rows of a tile again, in fp32, right whatever the scales are: of one cached head, up to
// four rows a warp and 32 cached tokens at a time, which go to shared memory as values.
// With a later token in eight of values 2^20 times the others', which makes nearly every
// tile one of those, 4 chunks of 1021 behind 2048 take 22.5 ms for 0.36, 16 trees of 64
// behind 4096 8.4 for 0.16, one behind 32768 8.5 for 0.1, 64 trees of 4 3.4 for 0.17; bound by
// the latency of a step's loads, sums and barriers. (A warp a row and a token at a time,
// and a third of the chunks' tiles: 88, 208 and, for the last, 101 ms.) 80 registers, so that a CTA starts beside the joining ones: with
// 128 the ordinary call of 2 trees waited 2 us longer.
constexpr int kRepairThreads = 256, kRepairWarps = kRepairThreads / 32, kRepairRows = 4, kRepairTokens = 32;
__host__ __device__ __forceinline__ size_t repair_smem(int D) {
  return (size_t)(kRepairTokens * (2 * D + 4) + kRepairWarps * kRepairRows * (D + kRepairTokens)) * 4;
}
// Rows first, first + 1, ... of the tile's rows of head hl of the block, `each` to a warp; C channels a lane.
template <int C>
__device__ __forceinline__ void repair(const AttnArgs &a, const Seq &s, int b, int block, int tile, int hl, int first, int each,
                                       float *smem, int64_t *slot_s) {
  const int head_block = block_of(a, block), part = block - head_block * a.parts, kv = head_block * a.hb + hl;
  const int length = s.length(a, tile), D = a.k.head_dim, pitch = D + 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Rows rows = rows_of(a, s, kv, part, tile);
  float *k_s = smem, *v_s = k_s + kRepairTokens * pitch;                       // [32][D + 4], [32][D]
  float *q_s = v_s + kRepairTokens * D + warp * kRepairRows * (D + kRepairTokens);  // of the warp: [4][D], [4][32]
  float *p_s = q_s + kRepairRows * D;
  const int r0 = first + warp * each, mine = min(each, rows.n - r0);  // (below 1: none)
  float m[kRepairRows], l[kRepairRows], acc[kRepairRows][C];
  int token[kRepairRows];
  unsigned long long bits[kRepairRows];
#pragma unroll
  for (int i = 0; i < kRepairRows; ++i) {
    m[i] = -INFINITY, l[i] = 0.f, token[i] = 0, bits[i] = 0;
#pragma unroll
    for (int k = 0; k < C; ++k) acc[i][k] = 0.f;
    if (i >= mine) continue;
    warp_query(a, q_s + i * D, rows.q_row(r0 + i), rows.q_head(r0 + i));
    token[i] = rows.j0 + rows.token(r0 + i);
    if (a.tree) bits[i] = (unsigned long long)a.tree[s.row0 + token[i]];
  }
#pragma unroll 1
  for (int t0 = 0; t0 < length; t0 += kRepairTokens) {
    __syncthreads();  // the tokens before are used
    if (threadIdx.x < kRepairTokens) slot_s[threadIdx.x] = t0 + (int)threadIdx.x < length ? slot_of(a, b, t0 + threadIdx.x) : -1;
    __syncthreads();
    for (int x = threadIdx.x; x < kRepairTokens * (D / 8); x += kRepairThreads) {
      const int t = x / (D / 8), c = x - t * (D / 8);
      float k[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
      if (slot_s[t] >= 0) {
        load_values(a.k, slot_s[t] * a.k.heads + kv, c, k);
        load_values(a.v, slot_s[t] * a.k.heads + kv, c, v);
      }
      float4 *to_k = reinterpret_cast<float4 *>(k_s + t * pitch + c * 8), *to_v = reinterpret_cast<float4 *>(v_s + t * D + c * 8);
      to_k[0] = make_float4(k[0], k[1], k[2], k[3]), to_k[1] = make_float4(k[4], k[5], k[6], k[7]);
      to_v[0] = make_float4(v[0], v[1], v[2], v[3]), to_v[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
    if (mine < 1) continue;
    float x[kRepairRows] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(k_s + lane * pitch + d);
#pragma unroll
      for (int i = 0; i < kRepairRows; ++i)
        if (i < mine) {
          const float4 q = *reinterpret_cast<const float4 *>(q_s + i * D + d);
          x[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, x[i]))));
        }
    }
    const bool there = slot_s[lane] >= 0;
#pragma unroll
    for (int i = 0; i < kRepairRows; ++i)
      if (i < mine) {
        // a score that is not a number stays one; a masked one counts nothing
        const bool on = there && s.sees(a, token[i], bits[i], t0 + lane);
        float top = on ? x[i] : -INFINITY;
#pragma unroll
        for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float now = fmaxf(m[i], top), base = now == -INFINITY ? 0.f : now, turn = exp2f(m[i] - base);
        const float p = on ? exp2f(x[i] - base) : 0.f;
        float sum = p;
#pragma unroll
        for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
        p_s[i * kRepairTokens + lane] = p;
        m[i] = now, l[i] = l[i] * turn + sum;
#pragma unroll
        for (int k = 0; k < C; ++k) acc[i][k] *= turn;
      }
    __syncwarp();
#pragma unroll 1
    for (int t = 0; t < kRepairTokens; t += 4) {
      float v[4][C];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < C; ++k) v[u][k] = lane + 32 * k < D ? v_s[(t + u) * D + lane + 32 * k] : 0.f;
#pragma unroll
      for (int i = 0; i < kRepairRows; ++i) {
        if (i >= mine) break;
        const float4 p = *reinterpret_cast<const float4 *>(p_s + i * kRepairTokens + t);
        auto add = [&](float w, int u) {
          if (w != 0.f)  // a masked value may be a NaN
#pragma unroll
            for (int k = 0; k < C; ++k) acc[i][k] = fmaf(w, v[u][k], acc[i][k]);
        };
        add(p.x, 0), add(p.y, 1), add(p.z, 2), add(p.w, 3);
      }
    }
    __syncwarp();
  }
  for (int i = 0; i < kRepairRows; ++i)
    if (i < mine) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float y = acc[0][k];
#pragma unroll
        for (int j = 1; j < kRepairRows; ++j)
          if (i == j) y = acc[j][k];
        if (lane + 32 * k < D) q_s[i * D + lane + 32 * k] = y;
      }
      float mm = m[0], ll = l[0];
#pragma unroll
      for (int j = 1; j < kRepairRows; ++j)
        if (i == j) mm = m[j], ll = l[j];
      __syncwarp();
      warp_finish(a, q_s + i * D, mm, ll, rows.q_row(r0 + i), rows.q_head(r0 + i));
      __syncwarp();
    }
}
// The scale of a group of a row, without its sign; 0 where it is no number or the group is idle. (Its first byte of codes
// is loaded beside it: nearly always that one tells.)
__device__ __forceinline__ float live_scale(const qwha_cache &c, int64_t row, int g, int groups) {
  const int bytes = c.group / 8 * c.bits;
  const uint8_t *at = c.codes + row * (c.head_dim / 8 * c.bits) + g * bytes;
  const float x = fabsf(__ldg(c.scales + row * groups + g));
  const uint32_t z = __ldg(c.zeros + row * groups + g), first = __ldg(at), mask = (1u << c.bits) - 1u;
  if (!(x < INFINITY)) return 0.f;
  if ((first & mask) != z) return x;
  bool idle;
  switch (c.bits) {
    case 2: idle = idle_bytes<2>(at, bytes, z, 0, 1); break;
    case 3: idle = idle_bytes<3>(at, bytes, z, 0, 1); break;
    case 4: idle = idle_bytes<4>(at, bytes, z, 0, 1); break;
    default: idle = idle_bytes<8>(at, bytes, z, 0, 1);
  }
  return idle ? 0.f : x;
}
// Looking at the scales of a tile's tokens: a warp has a cached head of the block, or, where
// there are fewer heads, a share of it.
struct Look {
  const AttnArgs &a;
  const int b, kv, hl, sub, per_head, lane;
  __device__ __forceinline__ Look(const AttnArgs &a_, int b_, int head_block)
      : a(a_), b(b_), kv(head_block * a_.hb + (int)(threadIdx.x >> 5) % a_.hb), hl((int)(threadIdx.x >> 5) % a_.hb),
        sub((int)(threadIdx.x >> 5) / a_.hb), per_head(kRepairWarps / a_.hb), lane(threadIdx.x & 31) {}
  __device__ __forceinline__ bool here() const { return sub < per_head && kv < a.k.heads; }
  __device__ __forceinline__ int64_t row(int t) const {  // of the token's scales; -1: none
    const int pg = page_of(a, t), page = __ldg(a.pages + (int64_t)b * a.max_pages + pg);
    return (uint32_t)page < (uint32_t)a.v.n_pages ? (((int64_t)page * a.v.page_size + t - pg * a.v.page_size) * a.v.heads + kv) : -1;
  }
};
// What is known of a group: bits of fp32, which order like the numbers.
struct Scales {
  uint32_t top, all, some;
};
constexpr uint32_t kInf = 0x7f800000u;
__device__ __forceinline__ float as_float(uint32_t x) { return __uint_as_float(x); }
// Which heads of the block (bits) `is` finds in the table.
template <typename F>
__device__ __forceinline__ unsigned heads_where(const AttnArgs &a, Scales (*of)[33], F is) {
  __shared__ unsigned heads_s;
  if (threadIdx.x == 0) heads_s = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.hb * 33; i += kRepairThreads)
    if (is(of[i / 33][i % 33])) atomicOr(&heads_s, 1u << (i / 33));
  __syncthreads();
  return heads_s;
}
__device__ __forceinline__ void clear(const AttnArgs &a, Scales (*of)[33]) {
  __syncthreads();
  for (int i = threadIdx.x; i < a.hb * 33; i += kRepairThreads) of[i / 33][i % 33] = {0u, 0u, kInf};
  __syncthreads();
}

// mma.sync: which heads have a group where tokens that not all rows see have scales (top)
// far above the least that a row may have: the largest of the tokens that all rows see
// (all), of which the newest 32 are looked at (every one, where these have none), or, where
// there are none, the least of the others (some). Idle groups do not count.
__device__ __forceinline__ unsigned far_for_some(const AttnArgs &a, const Seq &s, int b, int block, int tile, Scales (*of)[33]) {
  const int ng = a.v.head_dim / a.v.group, length = s.length(a, tile);
  const int safe = a.tree ? s.past : s.past + tile * a.tq + 1, near = max(safe - 32, 0);  // every row sees the tokens below safe
  if (s.rows - tile * a.tq == 1 || a.tq == 1 || length <= safe) return 0;  // (one token: its rows see the same)
  const Look l(a, b, block_of(a, block));
  // First without the codes: hardly any tile has scales so far apart, idle groups and all, as long as the newest token that
  // all rows see is not idle, whose scale the rows have.
  bool maybe = false;
  for (int g = l.sub; l.here() && g < ng; g += l.per_head) {
    float top = 0.f, least = INFINITY;
#pragma unroll 4
    for (int t = near + l.lane; t < length; t += 32) {
      const int64_t row = l.row(t);
      const float x = row >= 0 ? fabsf(__ldg(a.v.scales + row * ng + g)) : 0.f;
      if (t == safe - 1) maybe |= row < 0 || live_scale(a.v, row, g, ng) == 0.f;
      if (x > 0.f && x < INFINITY) {
        least = fminf(least, x);
        if (t >= safe) top = fmaxf(top, x);
      }
    }
    maybe |= as_float(__reduce_max_sync(~0u, __float_as_uint(top))) > kRoomMma * as_float(__reduce_min_sync(~0u, __float_as_uint(least)));
  }
  if (!__syncthreads_or(maybe)) return 0;
  clear(a, of);
  auto look = [&](int lo, int hi) {  // the scales of tokens [lo, hi)
    for (int t0 = lo + 32 * l.sub; l.here() && t0 < hi; t0 += 32 * l.per_head) {
      const int t = t0 + l.lane;
      const int64_t row = t < hi ? l.row(t) : -1;
      for (int g = 0; g < ng; ++g) {
        const uint32_t x = row >= 0 ? __float_as_uint(live_scale(a.v, row, g, ng)) : 0u;
        const uint32_t top = __reduce_max_sync(~0u, t < safe ? 0u : x), all = __reduce_max_sync(~0u, t < safe ? x : 0u);
        const uint32_t some = __reduce_min_sync(~0u, t < safe || !x ? kInf : x);
        Scales &y = of[l.hl][g];
        if (l.lane == 0) atomicMax(&y.top, top), atomicMax(&y.all, all), atomicMin(&y.some, some);
      }
    }
    __syncthreads();
  };
  look(near, length);
  if (near > 0 && heads_where(a, of, [](const Scales &x) { return x.top && !x.all; })) look(0, near);
  return heads_where(a, of, [](const Scales &x) { return as_float(x.top) > kRoomMma * as_float(x.all ? x.all : x.some); });
}
// tcgen05: which heads have scales far apart, of the values of a group (top, some) or of the keys (in the last place). Idle
// groups do not count.
__device__ __forceinline__ unsigned far_apart(const AttnArgs &a, const Seq &s, int b, int block, int tile, Scales (*of)[33]) {
  const int ng = a.v.head_dim / a.v.group, ng_k = a.k.head_dim / a.k.group, length = s.length(a, tile);
  const Look l(a, b, block_of(a, block));
  clear(a, of);
  for (int t0 = 32 * l.sub; l.here() && t0 < length; t0 += 32 * l.per_head) {
    const int64_t row = t0 + l.lane < length ? l.row(t0 + l.lane) : -1;
    auto put = [&](int at, float scale) {
      const uint32_t x = __float_as_uint(scale), top = __reduce_max_sync(~0u, x), some = __reduce_min_sync(~0u, x ? x : kInf);
      if (l.lane == 0) atomicMax(&of[l.hl][at].top, top), atomicMin(&of[l.hl][at].some, some);
    };
    for (int g = 0; g < ng; ++g) put(g, row >= 0 ? live_scale(a.v, row, g, ng) : 0.f);
    for (int g = 0; g < ng_k; ++g) put(32, row >= 0 ? live_scale(a.k, row, g, ng_k) : 0.f);
  }
  __syncthreads();
  return heads_where(a, of, [](const Scales &x) { return as_float(x.top) > kSpreadTc * as_float(x.some); });
}
// CTA (x, y): of sequences x, x + gridDim.x, ... the tiles y, y + gridDim.y, ..., or, where there are fewer tiles than
// that, a share of a tile's rows.
template <bool TC, int C>
__global__ void __launch_bounds__(kRepairThreads, C <= 4 ? 3 : 2) attention_repair_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(16) float repair_s[];
  __shared__ Scales of[kMmaWarps][33];
  __shared__ int64_t slot_s[kRepairTokens];
  if (TC) {  // only where some CTA of the kernel before says so
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool coarse = false;
    for (int i = threadIdx.x; i < a.ctas; i += kRepairThreads) coarse |= a.part_desc[2 * i].w & kPieceCoarse;
    if (!__syncthreads_or(coarse)) return;
  }
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const Seq s(a, b);
    const long long tiles = (long long)s.tiles * a.blocks;
    const int share = tiles < gridDim.y && tiles ? (int)(gridDim.y / tiles) : 1, step = (int)(gridDim.y / share);
    if ((int)blockIdx.y >= step * share) continue;
    for (long long i = blockIdx.y / share; i < tiles; i += step) {
      const int block = (int)(i / s.tiles), tile = (int)(i - (long long)block * s.tiles);
      const unsigned heads = TC ? far_apart(a, s, b, block, tile, of) : far_for_some(a, s, b, block, tile, of);
      if (!heads) continue;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      // pieces of `each` rows a warp, in turn to the CTAs that share the tile
      const int rows = min(a.tq, s.rows - tile * a.tq) * a.gh;  // (the last part of a group may have fewer)
      const int each = min(max((rows * __popc(heads) + share * kRepairWarps - 1) / (share * kRepairWarps), 1), kRepairRows);
      int turn = blockIdx.y % share;
      for (int hl = 0; hl < a.hb; ++hl)
        if (heads >> hl & 1)
          for (int first = 0; first < rows; first += each * kRepairWarps, turn = turn ? turn - 1 : share - 1)
            if (turn == 0) repair<C>(a, s, b, block, tile, hl, first, each, repair_s, slot_s);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

size_t any_smem(int D) {
  return (size_t)(kAnyRows * D + kAnyTokens * (D + 4) + kAnyTokens * D + kAnyRows * kAnyTokens) * 4;
}

}  // namespace

namespace {

// Rows of a cached head above which tiles of 128 on tcgen05 are taken instead of 32 on
// mma.sync, which does as many rows as there are (64 contexts of 4096, 8 heads, us on
// tcgen05 and mma.sync: 370 and 206 with 16 rows, 373 and 298 with 28, 376 and 299 with 32;
// even near 44); and those above which it is where the call is small: its tiles are a
// head's, not all heads', and are cut into fewer pieces (2 contexts of 1024: 25 and 38
// with 12 rows, 27 and 55 with 36; 16 of 4096: 101 and 71 with 12, 102 and 111 with 20; 4 of
// 32768: 169 and 152 with 16, 170 and 178 with 24). Small: up to 2^14 tokens of a cached
// head for each row, which over 1 to 64 contexts of 256 to 32768 tokens and 2 or 8 heads
// takes the better or is within 25%, but for one long context (of 32768: 61 and 116 with
// 16 rows, where it takes the latter). What the caller knows of the longest sequence, or
// the table's room, stands for the tokens, which only the device knows.
constexpr int kTcAbove = 44, kTcAboveIfSmall = 8, kTcSmallLog2 = 14;

// Shared memory of an SM, and what a CTA has of it besides the dynamic part: the kernels' arrays (more with more rows)
// and 1 KB of the system's.
constexpr size_t kSmemLimit = 228 * 1024;
constexpr size_t smem_besides(int nt) { return nt == 1 ? 6400 : 11 * 1024; }

// How a call is cut and launched.
struct Cut {
  int tq, gh, parts, hb, kt_log2, ctas;
  MmaLaunch mma;
  int part_rows() const { return hb * tq * gh; }
};
Cut cut_rows(int grp, int rows, int64_t n) {
  Cut c = {};
  c.parts = (int)cdiv(grp, rows), c.gh = (int)cdiv(grp, c.parts);
  c.tq = (int)std::clamp<int64_t>(rows / c.gh, 1, n);
  return c;
}
Cut any_cut(int grp, int64_t n) {
  Cut c = cut_rows(grp, kAnyRows, n);
  c.hb = 1, c.kt_log2 = ilog2(kAnyTokens), c.ctas = sm_count() * 3;
  return c;
}
Cut tc_cut(int grp, int64_t n) {
  Cut c = cut_rows(grp, kTcRows, n);
  c.hb = 1, c.kt_log2 = kTcKeysLog2, c.ctas = sm_count();
  return c;
}
int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Of a CTA of up to `warps` warps, as many CTAs as registers allow: two of eight
// warps to an SM for tiles of one n-tile, else one.
Cut cut_warps(int D, int heads, int grp, int64_t n, int nt, int warps) {
  Cut c = cut_rows(grp, 8 * nt, n);
  c.hb = (int)cdiv(heads, cdiv(heads, warps));
  c.mma.per_head = std::max(1, warps / c.hb), c.mma.warps = c.hb * c.mma.per_head, c.mma.nt = nt;
  c.ctas = sm_count() * std::max(1, (nt == 1 && padded(D) <= 128 ? 2 : 1) * kMmaWarps / c.mma.warps);
  c.kt_log2 = ilog2(kTokens * kTilesPerStage * c.mma.per_head);
  return c;
}
Cut mma_cut(int D, int heads, int grp, int64_t n, int nt, int pieces, int bits_k, int bits_v, int group_k, int group_v) {
  for (int warps = kMmaWarps;; warps /= 2) {
    Cut c = cut_warps(D, heads, grp, n, nt, warps);
    c.mma.smem = MmaShape(D, padded(D), bits_k, bits_v, group_k, group_v, nt, pieces, heads, c.hb, c.mma.per_head, c.mma.warps).total;
    const size_t fit = kSmemLimit / (c.mma.smem + smem_besides(nt));
    if (fit == 0 && warps > 1) continue;
    c.ctas = std::min(c.ctas, sm_count() * (int)std::max<size_t>(1, fit));
    c.mma.ctas = c.ctas;
    return c;
  }
}
size_t cut_bytes(const Cut &c, int D) {
  return align_up((size_t)c.ctas * 2 * sizeof(int4), 256) + align_up((size_t)c.ctas * 2 * c.part_rows() * 8, 256) +
         align_up((size_t)c.ctas * 2 * c.part_rows() * D * 4, 256);
}

// Whether the tensor-core kernels take a cache's codes: rows of whole words (3-bit
// ones lie as they may).
bool takes_codes(const qwha_cache &c) { return c.bits != 2 || c.head_dim % 16 == 0; }
// (slots in 32 bits: a cache of more has rows of a few bytes)
bool mma_takes(const AttnArgs &a) {
  return takes_codes(a.k) && takes_codes(a.v) && a.k.n_pages * a.k.page_size < (1LL << 31);
}
bool tc_takes(const AttnArgs &a) {
  const int64_t rows = cdiv(a.n, a.n_seqs) * a.grp, tokens = (int64_t)a.n_seqs * a.k.heads * a.longest;
  return (rows > kTcAbove || (rows > kTcAboveIfSmall && tokens <= rows << kTcSmallLog2)) && attention_tc_takes(a);
}
// Whether rows may have to be done again: on mma.sync not where a tile has one token, whose rows all see the same.
bool repairs(const AttnArgs &a) { return tc_takes(a) || (mma_takes(a) && a.n > a.n_seqs); }

}  // namespace

// Enough for any formats of the caches: their sizes decide how many warps a CTA
// gets and how many CTAs fit, of which cut_warps's are the most.
size_t attention_workspace(int32_t q_heads, int32_t head_dim, int32_t heads, int64_t n, bool f32) {
  if (heads <= 0 || q_heads % heads || n <= 0) return 0;
  const int grp = q_heads / heads;
  size_t most = cut_bytes(any_cut(grp, n), head_dim);
  if (!f32) most = std::max(most, cut_bytes(tc_cut(grp, n), head_dim));
  for (int nt = 1; nt <= 4; nt *= 2)
    for (int warps = kMmaWarps; warps; warps /= 2)
      most = std::max(most, cut_bytes(cut_warps(head_dim, heads, grp, n, nt, warps), head_dim));
  return most;
}

int attention_launches(const AttnArgs &a) { return repairs(a) ? 3 : 2; }

cudaError_t launch_attention(AttnArgs a, void *ws, cudaStream_t s) {
  static std::atomic<size_t> allowed[64];
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidDevicePointer;
  const int D = a.k.head_dim;
  const int64_t rows = cdiv(a.n, a.n_seqs) * a.grp;  // of a cached head, on average
  const bool tc = tc_takes(a), mma = mma_takes(a);
  const int64_t most = a.n <= a.n_seqs ? 1 : a.n;  // tokens of a tile
  Cut c;
  if (tc) {
    c = tc_cut(a.grp, most);
  } else if (mma) {
    const int nt = rows <= 8 ? 1 : rows <= 16 || D > 128 ? 2 : 4;
    c = mma_cut(D, a.k.heads, a.grp, most, nt, a.f32 ? 2 : 1, a.k.bits, a.v.bits, a.k.group, a.v.group);
  } else {
    c = any_cut(a.grp, a.n);
  }
  a.tq = c.tq, a.gh = c.gh, a.parts = c.parts, a.hb = c.hb, a.kt_log2 = c.kt_log2, a.ctas = c.ctas;
  a.blocks = (int)cdiv(a.k.heads, a.hb) * a.parts, a.part_rows = c.part_rows();
  char *p = static_cast<char *>(ws);
  a.part_desc = reinterpret_cast<int4 *>(p), p += align_up((size_t)a.ctas * 2 * sizeof(int4), 256);
  a.part_stats = reinterpret_cast<float *>(p), p += align_up((size_t)a.ctas * 2 * a.part_rows * 8, 256);
  a.part = reinterpret_cast<float *>(p);
  cudaError_t e;
  if (tc) {
    e = launch_attention_tc(a, s);
  } else if (mma) {
    e = D <= 64 ? launch_attention_d64(a, c.mma, s) : D <= 128 ? launch_attention_d128(a, c.mma, s) : launch_attention_d256(a, c.mma, s);
  } else {
    const size_t smem = any_smem(D);
    e = allow_smem(reinterpret_cast<const void *>(attention_any_kernel), smem, allowed);
    if (e != cudaSuccess) return e;
    attention_any_kernel<<<a.ctas, kAnyThreads, smem, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas, (unsigned)cdiv(a.part_rows, kJoinRows)), cfg.blockDim = dim3(kJoinThreads), cfg.stream = s;
  cfg.dynamicSmemBytes = a.ctas * sizeof(int);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, D <= 64 ? attention_join_kernel<8> : D <= 128 ? attention_join_kernel<16> : attention_join_kernel<32>, a);
  if (e != cudaSuccess || !repairs(a)) return e;
  static std::atomic<size_t> repair_allowed[3][64];
  auto kernel = tc ? attention_repair_kernel<true, 4> : D <= 128 ? attention_repair_kernel<false, 4> : attention_repair_kernel<false, 8>;
  const size_t smem = repair_smem(D);
  e = allow_smem(reinterpret_cast<const void *>(kernel), smem, repair_allowed[tc ? 0 : D <= 128 ? 1 : 2]);
  if (e != cudaSuccess) return e;
  const int ctas = 2 * sm_count(), seqs = std::min(a.n_seqs, ctas);
  cfg.gridDim = dim3(seqs, ctas / seqs), cfg.blockDim = dim3(kRepairThreads), cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace qwha
