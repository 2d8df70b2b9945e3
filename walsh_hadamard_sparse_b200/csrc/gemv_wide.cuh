// The packed product for many columns (tokens times their pieces) on the
// 5th-generation tensor cores: one definition for the three code widths.
//
//   Y[t, r] = sum over groups g of scales[r, g] * (sum_{k in g} (q - zero)[r, k] x[t, k])
//
// q - zero is an integer of at most eight bits and a sign, exact in bf16, and
// so is a bf16 value; an fp32 value is three bf16 pieces (wide_prepare), each a
// column. So the inner sums are tcgen05 products of exact operands with fp32
// accumulators, and the scales stay outside: an accumulator per group, read
// back once and added with its scale in fp32. No weight is rounded.
//
// A CTA takes 128 rows and a slice of the columns (a cluster of slices shares
// its rows and adds its sums through distributed shared memory in rank order).
//   12 or 8   unpack, teams of four in turn: a lane holds runs of 32 codes of
//             four rows, kAhead chunks of its team in flight from memory; a code
//             ORed into the mantissa of 128 minus 128 + zero is q - zero; stored
//             as a K-major tile with 128-byte swizzle.
//   8 warps   scale: thread = row (TMEM lane), the two halves of the warps take
//             alternate blocks of 16 columns.
//   1 warp    copies the values' tile, laid out by the preparing launch as
//             shared memory holds it: one bulk copy a chunk.
//   1 warp    issues the products.
// The order of the columns inside a run is the one the codes' masks yield, in
// both operands. Unpacking sets the pace: 14336 x 4096, 4 bits, 64 bf16 tokens
// take 27.6 us on 112 SMs, 0.7 us for a CTA's chunk of 128 x 128 codes, of which
// the products need 0.5; the bytes alone 5 us. Every wait is bounded; a thread that gives up sets the error
// word and leaves its loop, and TMEM is freed after the products issued so far.

#pragma once

#include "gemv_mma.cuh"

namespace qwha {
namespace wide {

constexpr int kRows = 128, kScaleWarps = 8, kAhead = 1, kMaxSlots = 8;
// With NB blocks of 16 columns to a scaling warp: the stages that fit, and the
// teams that the registers of the sums leave room for (64 bf16 tokens of
// 14336 x 4096, when three teams took 30 us: two 36; 32 tokens: three 27, four
// with five stages 29). A second chunk in flight to a team needs its loop
// unrolled once more: 39 instead of 36 us with two teams, for the instructions'
// own fetches.
template <int NB>
constexpr int stages() { return NB <= 2 ? 4 : 3; }
template <int NB>
constexpr int teams() { return NB <= 2 ? 3 : 2; }
template <int NB>
constexpr int threads() { return (4 * teams<NB>() + kScaleWarps + 2) * 32; }
constexpr uint32_t kABytes = kRows * 256, kTmemCols = 512;

__device__ __forceinline__ uint64_t sw128(uint32_t saddr) {  // K-major rows of 128 bytes, eight to an atom
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One thread of a converged warp, in the form that tells the compiler so.
__device__ __forceinline__ bool elected() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one;
}
// bulk::wait with a hint that lets the thread be suspended for up to 2 us at a
// time: most warps of the CTA wait for another at any moment.
__device__ __forceinline__ bool calm_wait(uint32_t bar, uint32_t parity) {
  uint64_t begin = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(2000u)
        : "memory");
    if (ok) return true;
    const uint64_t now = bulk::now_ns();
    if (begin == 0) begin = now;
    else if (now - begin > bulk::kWaitNs) return false;
  }
}
// One lane waits for its warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = calm_wait(bar, parity);
  return __all_sync(~0u, ok);
}
__device__ __forceinline__ void load16(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// The loads of v and w have arrived; nothing that reads them moves before this.
__device__ __forceinline__ void wait_loads(float *v, float *w) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
  asm volatile(""
               : "+f"(w[0]), "+f"(w[1]), "+f"(w[2]), "+f"(w[3]), "+f"(w[4]), "+f"(w[5]), "+f"(w[6]), "+f"(w[7]),
                 "+f"(w[8]), "+f"(w[9]), "+f"(w[10]), "+f"(w[11]), "+f"(w[12]), "+f"(w[13]), "+f"(w[14]), "+f"(w[15])
               :
               : "memory");
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d =
      __hsub2(reinterpret_cast<const __nv_bfloat162 &>(a), reinterpret_cast<const __nv_bfloat162 &>(b));
  return reinterpret_cast<const uint32_t &>(d);
}
__device__ __forceinline__ uint32_t bf16x2_of(float v) {  // v in both halves
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v)) * 0x10001u;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float peer_float(uint32_t saddr, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}

// The sixteen pairs of a run (gemv::first, gemv::gap) as bf16 128 + q.
template <int BITS>
__device__ __forceinline__ void unpack(const uint32_t *w, uint32_t *q) {
  constexpr uint32_t mask = 0x00010001u * ((1u << BITS) - 1u), of128 = 0x43004300u;
  if constexpr (BITS == 3) {
    gemv::unpack<3>(w, q);
#pragma unroll
    for (int p = 0; p < 16; ++p) q[p] = (q[p] >> gemv::unit<3>(p)) | of128;
  } else {
#pragma unroll
    for (int p = 0; p < 16; ++p) q[p] = (w[p * BITS / 16] >> (p * BITS % 16) & mask) | of128;
  }
}

// The values of one token as columns of the products' second operand, by one
// CTA: per chunk of 128 columns, the tile as shared memory holds it, [2 slabs
// of 64][npad][128 bytes, 16-byte units swizzled by the column]. An fp32 token
// is scaled by a power of two that brings its largest value into [1, 2) (undone
// by fac), so that the third piece of all but negligible values is a normal
// number. Slots of the last pass without a token, and pieces that fill npad,
// are zeros.
template <int BITS, typename T>
__device__ __forceinline__ void wide_prepare(const GemvArgs &a, int slot, int slots) {
  constexpr bool f32 = sizeof(T) == 4;
  constexpr int P = f32 ? 3 : 1;
  const int pass = slot / slots, at = slot % slots, tok = pass * a.tpp + at;
  const bool live = at < a.tpp && tok < a.T;
  const int chunks = (a.d_in + 127) / 128;
  const T *src = static_cast<const T *>(a.x) + (int64_t)tok * a.d_in;
  float up = 1.f;
  if constexpr (f32) {
    __shared__ uint32_t top_s;
    if (threadIdx.x == 0) top_s = 0;
    __syncthreads();
    uint32_t top = 0;
    for (int k = threadIdx.x * 4; live && k < a.d_in; k += blockDim.x * 4) {
      float v[4];
      gemv::load4(src + k, v);
#pragma unroll
      for (int u = 0; u < 4; ++u) top = max(top, __float_as_uint(v[u]) & 0x7fffffffu);
    }
    atomicMax(&top_s, __reduce_max_sync(~0u, top));
    __syncthreads();
    top = top_s;
    const int e = (int)(top >> 23);
    // 2^(127 - e), kept within normal numbers; nothing to scale for 0, infinities and NaN
    const int k = top == 0 || e == 255 ? 0 : min(126, max(-126, 127 - e));
    up = gemv::exp2i(k);
    if (threadIdx.x == 0 && live) a.fac[tok] = gemv::exp2i(-k);
  }
  uint8_t *tiles = reinterpret_cast<uint8_t *>(a.xpieces) + (int64_t)pass * chunks * a.npad * 256;
  for (int i = threadIdx.x; i < chunks * 16; i += blockDim.x) {
    const int run = i >> 2, u = i & 3, k0 = run * 32;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live && k0 < a.d_in) {
      const int k = k0 + (BITS == 4 ? 8 * u : BITS == 2 ? 16 * (u >> 1) + 4 * (u & 1) : 4 * u);
      gemv::load4(src + k, v);
      gemv::load4(src + k + gemv::gap<BITS>(), v + 4);
    }
    const int unit = (run & 1) * 4 + u;
    uint8_t *slab = tiles + ((int64_t)(run >> 2) * 2 + ((run >> 1) & 1)) * a.npad * 128;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = at * P + p;
      if (col >= a.npad) break;
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = p ? v[j] : v[j] * up, hi = p ? v[4 + j] : v[4 + j] * up;
        r[j] = pack_bf16x2(lo, hi);
        v[j] = lo - bf16_lo(r[j]), v[4 + j] = hi - bf16_hi(r[j]);
      }
      *reinterpret_cast<uint4 *>(slab + col * 128 + ((unit ^ (col & 7)) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

// NB blocks of 16 columns to each half of the scaling warps.
template <int BITS, int NB>
__global__ void __launch_bounds__(threads<NB>(), 1) gemv_wide_kernel(const __grid_constant__ GemvArgs a, int slices) {
  constexpr int kStages = stages<NB>(), kTeams = teams<NB>(), kUnpackWarps = 4 * kTeams;
  constexpr int kCopyWarp = kUnpackWarps + kScaleWarps, kIssueWarp = kCopyWarp + 1;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (bulk::saddr(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (base - bulk::saddr(raw));
  const uint32_t b_bytes = a.npad * 256, b_base = base + kStages * kABytes;
  __shared__ uint64_t bars[2 * kStages + 2 * kMaxSlots + 1];
  __shared__ uint32_t tmem_s;
  const uint32_t bar0 = bulk::saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto sum_full = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
  auto sum_empty = [&](int s) { return bar0 + 8u * (2 * kStages + kMaxSlots + s); };
  const uint32_t done = bar0 + 8u * (2 * kStages + 2 * kMaxSlots);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % slices, row0 = blockIdx.x / slices * kRows;  // the cluster lies along x
  const int ng = a.d_in / a.group, chunks = (a.d_in + 127) / 128, runs = a.group / 32;
  const int G = a.group % 128 == 0 ? 1 : a.group % 64 == 0 ? 2 : 4;
  const int per = (chunks + slices - 1) / slices, c_begin = rank * per < chunks ? rank * per : chunks;
  const int c_end = c_begin + per < chunks ? c_begin + per : chunks;
  const int stride = a.npad <= 32 ? 32 : a.npad <= 64 ? 64 : 128;  // TMEM columns from one accumulator to the next
  const int slots = (int)kTmemCols / stride < kMaxSlots ? (int)kTmemCols / stride : kMaxSlots;
  auto give_up = [&]() { atomicOr(a.err, kErrEntries); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) bulk::init(full(s), 4 * 32 + 1), bulk::init(empty(s), 1);
    for (int s = 0; s < kMaxSlots; ++s) bulk::init(sum_full(s), 1), bulk::init(sum_empty(s), kScaleWarps);
    bulk::init(done, 1);
    bulk::fence_init();
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bulk::saddr(&tmem_s)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_s;
  const int out_stride = a.npad + 1;
  float *out = reinterpret_cast<float *>(smem);  // [kRows][out_stride], over the stages once they are used up

  if (warp < kUnpackWarps) {
    // Teams of four warps take the chunks in turn, so that some wait while others compute.
    const int team = warp / 4, g = lane >> 2, t = lane & 3;
    const uint8_t *next[4], *pz[4];
    const int c_first = c_begin + team;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int r = warp % 4 * 32 + h * 8 + g;
      const int row = row0 + r < a.d_out ? row0 + r : a.d_out - 1;  // rows behind the last repeat it, not stored
      next[h] = a.qw + ((int64_t)row * (a.d_in / 32) + c_first * 4 + t) * (4 * BITS);
      pz[h] = a.zeros + (int64_t)row * ng;
    }
    // the run's units in a stage are (4 (t % 2) + u) ^ (row % 8); the upper slab's lanes hold u ^ 2 in place of u, so
    // that the eight lanes of a store's quarter meet eight different bank groups (3-bit runs: four, twice)
    const bool swap = BITS != 3 && (t & 2);
    uint8_t *dst0 = smem + (t >> 1) * (kRows * 128) + (warp % 4 * 32 + g) * 128;
    uint32_t w[kAhead][4][BITS], z[kAhead][4];
    // the group of the lane's run in the chunk to fetch next: run / runs, by steps of a round of the teams
    int group = (c_first * 4 + t) / runs, in_group = (c_first * 4 + t) % runs;
    const int group_step = 4 * kTeams / runs, in_step = 4 * kTeams % runs;
    auto fetch = [&](auto I, int c) {
      constexpr int i = decltype(I)::value;
      const bool in = c < c_end && c * 4 + t < a.d_in / 32;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        gemv::f_zero<BITS>(w[i][h]);
        z[i][h] = 0;
        if (in) {
          gemv::load_run<BITS, 0>(next[h], w[i][h]);
          z[i][h] = __ldg(pz[h] + group);
        }
        next[h] += kTeams * 16 * BITS;
      }
      group += group_step, in_group += in_step;
      if (in_group >= runs) in_group -= runs, ++group;
    };
    gemv::each<kAhead>([&](auto I) { fetch(I, c_first + kTeams * decltype(I)::value); });
    bool ok = true;
    for (int c0 = c_first, it = team; ok && c0 < c_end; c0 += kTeams * kAhead) {
      gemv::each<kAhead>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if (!ok || c0 + kTeams * i >= c_end) return;
        const int s = it % kStages;
        if (!warp_wait(empty(s), (it / kStages & 1) ^ 1)) {
          give_up();
          ok = false;
          return;
        }
        const bool any_far = __any_sync(~0u, max(max(z[i][0], z[i][1]), max(z[i][2], z[i][3])) > 127);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if constexpr (BITS != 3) {
#pragma unroll
            for (int j = 0; j < BITS / 2; ++j) {
              const uint32_t x = w[i][h][j], y = w[i][h][j + BITS / 2];
              w[i][h][j] = swap ? y : x, w[i][h][j + BITS / 2] = swap ? x : y;
            }
          }
          uint32_t q[16];
          unpack<BITS>(w[i][h], q);
          // 128 + zero is exact for a zero below 128; a larger one is taken off in two exact steps
          const bool far = z[i][h] > 127;
          const uint32_t first = (0x4300u | (far ? 0u : z[i][h])) * 0x10001u;
#pragma unroll
          for (int p = 0; p < 16; ++p) q[p] = sub_bf16x2(q[p], first);
          if (any_far) {
            const uint32_t rest = far ? bf16x2_of((float)z[i][h]) : 0u;
#pragma unroll
            for (int p = 0; p < 16; ++p) q[p] = sub_bf16x2(q[p], rest);
          }
          uint8_t *dst = dst0 + s * kABytes + h * 8 * 128;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4 *>(dst + (((4 * (t & 1) + (u ^ (swap ? 2 : 0))) ^ g) << 4)) =
                make_uint4(q[4 * u], q[4 * u + 1], q[4 * u + 2], q[4 * u + 3]);
        }
        fetch(I, c0 + kTeams * (i + kAhead));
        bulk::fence_proxy();
        arrive(full(s));
        it += kTeams;
      });
    }
  } else if (warp < kUnpackWarps + kScaleWarps) {
    const int half = (warp - kUnpackWarps) / 4, r = warp % 4 * 32 + lane;
    const int row = row0 + r < a.d_out ? row0 + r : a.d_out - 1;
    const float *ps = a.scales + (int64_t)row * ng;
    float acc[NB][16];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[b][i] = 0.f;
    const int units = (c_end - c_begin) * G, runs_of = 4 / G;  // runs of a unit
    // the unit to load next: its first run, and the group of that by steps
    int run = c_begin * 4, in_group = run % runs;
    const float *next = ps + run / runs;
    auto next_scale = [&]() {
      const float v = run < c_end * 4 && run < a.d_in / 32 ? __ldg(next) : 0.f;
      run += runs_of, in_group += runs_of;
      if (in_group >= runs) in_group -= runs, ++next;
      return v;
    };
    float s_next = next_scale(), s_then = next_scale();
    uint32_t parity = 0;
    for (int u = 0, slot = 0; u < units; ++u) {
      const float s = s_next;
      s_next = s_then, s_then = next_scale();
      if (!warp_wait(sum_full(slot), parity)) {
        give_up();
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t at = tmem + ((uint32_t)(warp % 4) << 21) + slot * stride;  // lanes 32 (warp % 4) on
      // columns behind npad are read (they lie within the stride) and not stored
#pragma unroll
      for (int b = 0; b < NB; b += 2) {
        float v[2][16];
        load16(at + (2 * b + half) * 16, v[0]);
        if constexpr (NB > 1) {
          load16(at + (2 * b + 2 + half) * 16, v[1]);
          wait_loads(v[0], v[1]);
        } else {
          wait_loads(v[0], v[0]);
        }
#pragma unroll
        for (int j = 0; j < (NB > 1 ? 2 : 1); ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[b + j][i] = fmaf(s, v[j][i], acc[b + j][i]);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(sum_empty(slot));
      if (++slot == slots) slot = 0, parity ^= 1;
    }
    // the last accumulator's products were the last readers of the stages
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if ((2 * b + half) * 16 < a.npad)
#pragma unroll
        for (int i = 0; i < 16; ++i) out[r * out_stride + (2 * b + half) * 16 + i] = acc[b][i];
  } else if (warp == kCopyWarp) {
    if (lane == 0) {
      // the values are the preparing launch's output (see gemv_mma_kernel)
      if (a.y_ad) {
        if (!gemv::wait_ready(a.ready)) give_up();
      } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      const uint8_t *src = reinterpret_cast<const uint8_t *>(a.xpieces) + (int64_t)blockIdx.y * chunks * b_bytes;
      for (int c = c_begin, it = 0; c < c_end; ++c, ++it) {
        const int s = it % kStages;
        if (!calm_wait(empty(s), (it / kStages & 1) ^ 1)) {
          give_up();
          break;
        }
        bulk::load(b_base + s * b_bytes, src + (int64_t)c * b_bytes, b_bytes, full(s));
      }
    }
    __syncwarp();
  } else {
    if (elected()) {
      // D fp32, A and B bf16, both K-major, N / 8, M / 16
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(a.npad >> 3) << 17) | (8u << 24);
      // a thread by itself: every instruction costs its latency, so nothing is divided or tested per product
      auto issue = [&](auto groups) {
        constexpr int n = decltype(groups)::value;
        uint64_t da = sw128(base), db = sw128(b_base);
        const uint32_t slab = a.npad * 128 >> 4;
        uint32_t parity = 0, turn = 1;  // of the stages; of the accumulators
        for (int c = c_begin, s = 0, slot = 0; c < c_end; ++c) {
          if (!calm_wait(full(s), parity)) return false;
#pragma unroll
          for (int gi = 0; gi < n; ++gi) {
            if (!calm_wait(sum_empty(slot), turn)) return false;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + slot * stride;
#pragma unroll
            for (int k = gi * 8 / n; k < (gi + 1) * 8 / n; ++k)
              product(d, da + (k >> 2) * (kRows * 128 >> 4) + (k & 3) * 2, db + (k >> 2) * slab + (k & 3) * 2, idesc,
                      k != gi * 8 / n);
            commit(sum_full(slot));
            if (++slot == slots) slot = 0, turn ^= 1;
          }
          commit(empty(s));
          da += kABytes >> 4, db += b_bytes >> 4;
          if (++s == kStages) s = 0, parity ^= 1, da = sw128(base), db = sw128(b_base);
        }
        return true;
      };
      const bool ok = G == 1   ? issue(std::integral_constant<int, 1>())
                      : G == 2 ? issue(std::integral_constant<int, 2>())
                               : issue(std::integral_constant<int, 4>());
      if (!ok) give_up();
      commit(done);  // TMEM must not be freed under a product
      if (!calm_wait(done, 0)) give_up();
    }
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // before the cluster's barrier: another cluster's CTA may be waiting for these columns
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
  if (a.y_ad) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the entries' sums
  if (slices > 1) cluster_sync();
  // a thread takes one row and every step-th token
  const int rows = kRows / slices, t0 = blockIdx.y * a.tpp, np = a.T - t0 < a.tpp ? a.T - t0 : a.tpp;
  const int step = 512 / rows, r = rank * rows + (threadIdx.x & (rows - 1)), row = row0 + r;
  if (threadIdx.x < 512 && row < a.d_out) {
    const int first = threadIdx.x >> (31 - __clz(rows));
    auto sum_of = [&](int tok) {
      const float *mine = out + r * out_stride + tok * a.pieces;
      float sum = 0.f;
      for (int p = 0; p < a.pieces; ++p) {
        if (slices == 1) {
          sum += mine[p];
        } else {
          for (int w = 0; w < slices; ++w) sum += peer_float(bulk::saddr(mine + p), w);
        }
      }
      return a.f32 ? sum * a.fac[t0 + tok] : sum;
    };
    auto put = [&](int tok, float sum) {
      if (a.y_ad) sum += a.alpha * a.y_ad[(int64_t)row * a.tp + t0 + tok];
      const int64_t at = (int64_t)(t0 + tok) * a.d_out + row;
      if (a.f32) static_cast<float *>(a.y)[at] = sum;
      else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(sum);
    };
    bool again = false;
#pragma unroll 4
    for (int tok = first; tok < np; tok += step) {
      const float sum = sum_of(tok);
      again |= !gemv::finite(sum);
      put(tok, sum);
    }
    if (again)
      for (int tok = first; tok < np; tok += step) {
        const float sum = sum_of(tok);
        if (!gemv::finite(sum)) put(tok, gemv::plain_dot(a, row, t0 + tok));
      }
  }
  if (slices > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

template <int BITS, int NB>
cudaError_t launch_one(const GemvArgs &a, cudaStream_t s) {
  const int64_t tiles = cdiv(a.d_out, kRows), chunks = cdiv(a.d_in, 128);
  // slices: as many as leave a CTA on every SM at most, two chunks each at least
  int slices = 1;
  while (slices < 8 && tiles * slices * 2 <= sm_count() && chunks >= 4 * slices) slices *= 2;
  const size_t smem = stages<NB>() * (size_t)(kABytes + a.npad * 256) + 1024;
  auto kernel = gemv_wide_kernel<BITS, NB>;
  static std::atomic<size_t> allowed[64];
  const cudaError_t e = allow_smem((const void *)kernel, smem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * slices), (unsigned)cdiv(a.T, a.tpp));
  cfg.blockDim = dim3(threads<NB>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = slices, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;  // overlaps the launches of its call before it
  return cudaLaunchKernelEx(&cfg, kernel, a, slices);
}

template <int BITS>
cudaError_t launch_bits(const GemvArgs &a, cudaStream_t s) {
  if (a.npad <= 32) return launch_one<BITS, 1>(a, s);
  if (a.npad <= 64) return launch_one<BITS, 2>(a, s);
  return launch_one<BITS, 4>(a, s);
}

}  // namespace wide
}  // namespace qwha
