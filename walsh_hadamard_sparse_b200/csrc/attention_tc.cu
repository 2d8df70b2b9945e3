// Attention over the quantized cache on the 5th-generation tensor cores: bf16
// calls with more rows to a cached head than the kernel of attention_mma.cuh
// likes (drafted trees, chunks of prompts).
//
// A CTA takes one cached head and up to 256 rows of queries (tokens times the
// query heads that share the head), two tiles of 128, and walks 128 cached tokens
// at a time:
//   S_w = Q_w C_k^T    tcgen05, operands in shared memory, fp32 in TMEM, 64 tokens
//                      at a time: one half is multiplied while the other is read
//   P_w = 2^(S_w - m)  by the 128 threads of the tile, a row each; f16 over S_w
//   O_w += P_w C_v     tcgen05, P from TMEM, C_v in shared memory
// C holds (code - zero) times scale in f16, rounded once (the difference is exact, the
// scale, times a power of two that follows the largest of its group, comes in two
// pieces): 2^-11 at the most beside the 2^-9 of a bf16 output, and different for each
// channel, so that a score's errors average out. (A scale of one piece errs alike in all
// channels of a token: 0.0023 against 0.0019 of error for a tree of 64, 0.0017 of it
// the output's own rounding.) Scales left to the columns of S and P in fp32 were two
// multiplications and 16 loads more for 16 scores: 384 us for 4 chunks of 1021 tokens
// behind 2048, where this took 350. The query (rotated, its largest value near 2^15)
// and P are rounded to 11 bits as in attention_mma.cuh; the maximum is kept to within
// what f16 leaves room for: half a tile whose weights sum to more than 2^7 has its
// maximum taken and is done again, others need none.
//   8 warps  unpack, four the keys and four the values: a lane's 32 codes of a
//            token, fetched a tile ahead, to swizzled tiles of f16 (two of each). They
//            notice scales that lie 2^13 below the largest, which would lose bits in
//            f16: tiles that have such are done again (attention.cu). By the comparison
//            that finds growing scales; a minimum kept beside it cost 3%.
//   8 warps  softmax: four for each tile of rows.
//   1 warp   issues the products: S_w of the next tile's half behind O_w of this
//            one's.
// Bound: the 16384 exponentials and about 80 thousand other operations of a tile of 128
// rows and tokens, and 1024 clocks of products. 4 chunks of 1021 tokens behind 2048 (32
// and 8 heads of 128, 8 bits): 343 us, 388 TFLOP/s; trees of 64 tokens on 16 contexts of
// 4096, 4 bits: 149 us. Of a CTA's clocks in the first the softmax warps spend 38% on
// weights, 14% on writing rows out, 11% on queries, 11% waiting for scores. Every wait is
// bounded; a thread that gives up sets the error word and goes on without waiting.

#include <cuda_fp16.h>

#include <type_traits>

#include "attention_mma.cuh"
#include "gemv_wide.cuh"

namespace qwha {
namespace {

using namespace attn;
using bulk::saddr;
using wide::arrive;
using wide::commit;
using wide::sw128;

constexpr int kRowsTile = 128, kKeys = 128, kUnpackWarps = 8, kSoftWarps = 8;  // (unpacking: half for the keys)
constexpr int kUnpackers = kUnpackWarps * 16, kRounds = 128 / kUnpackers * 2, kTcThreads = (kUnpackWarps + kSoftWarps + 1) * 32;
constexpr int kScaleSlots = 4;      // tiles whose scales are kept: a tile's are read until its weights are made
constexpr float kTcTop = 64.f;      // of a scale in f16, times 255 of a code below the largest
constexpr float kTcLeast = 0.001953125f;  // what scales are to be at least: 2^4, where the largest lies, over kSpreadTc
constexpr float kTcShift = 8.f;     // weights are kept 2^8 times as large: f16 holds them to 2^-33 of the maximum's
constexpr float kTcSum = 32768.f;   // of the weights of half a tile, before its maximum is taken again
constexpr uint32_t kTcCols = 512;   // TMEM: S_0, S_1, O_0, O_1
constexpr unsigned int kErrTc = 0x10000u;  // a wait gave up

__device__ __forceinline__ uint64_t sw128_mn(uint32_t at) {  // slabs of 64 channels x 128 tokens, rows of 128 bytes
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)(kKeys * 128 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D += A B with A in TMEM
__device__ __forceinline__ void product_t(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
#define QWHA_R32(x)                                                                                              \
  x(0), x(1), x(2), x(3), x(4), x(5), x(6), x(7), x(8), x(9), x(10), x(11), x(12), x(13), x(14), x(15), x(16), x(17), \
      x(18), x(19), x(20), x(21), x(22), x(23), x(24), x(25), x(26), x(27), x(28), x(29), x(30), x(31)
__device__ __forceinline__ void load32(uint32_t at, uint32_t *r) {
#define X(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : QWHA_R32(X)
      : "r"(at)
      : "memory");
#undef X
}
__device__ __forceinline__ void store32(uint32_t at, const uint32_t *r) {
#define X(i) "r"(r[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::QWHA_R32(X),
      "r"(at)
      : "memory");
#undef X
}
__device__ __forceinline__ void load8(uint32_t at, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void loads_done(uint32_t *r) {  // (32 registers that the loads wrote)
#define X(i) "+r"(r[i])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : QWHA_R32(X)::"memory");
#undef X
}
__device__ __forceinline__ void stores_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void store8(uint32_t at, const float *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "r"(at)
               : "memory");
}
// Eight columns from `at` on of every 32 of a row.
template <int DP>
__device__ __forceinline__ void load_across(uint32_t at, float *v) {
  uint32_t u[32];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (x < DP / 32) load8(at + 32 * x, u + 8 * x);
    else
#pragma unroll
      for (int k = 0; k < 8; ++k) u[8 * x + k] = 0;
  }
  loads_done(u);
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(u[k]);
}
// Sixteen columns, and the wait for them: no memory but TMEM, so that the compiler may move other loads past them.
__device__ __forceinline__ void columns16(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at));
}
__device__ __forceinline__ void columns_done(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 both(float a, float b) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void split(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Butterflies of the places H, 2 H, ... below N H of 32 values, those below had.
template <int H, int N>
__device__ __forceinline__ void rotate32(float *v, int had) {
#pragma unroll
  for (int h = H; h < H * N; h *= 2)
    if (had > h) {
      if (h == 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float x = v[i], y = v[i + 1];
          v[i] = x + y, v[i + 1] = x - y;
        }
      } else {  // two at once
        const f32x2 minus = both(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          if (!(i & h)) {
            const f32x2 x = both(v[i], v[i + 1]), y = both(v[i + h], v[i + h + 1]);
            split(add2(x, y), v[i], v[i + 1]);
            split(fma2(y, minus, x), v[i + h], v[i + h + 1]);
          }
      }
    }
}

// What the softmax threads know of a tile of tokens.
struct alignas(16) TileScales {
  uint32_t live[4];       // a bit a token
  float values[4];        // what the values' scales were multiplied by, of each 32 channels: powers of two
  float grow[4];          // these against the last tile's, where grown
  float keys;             // the keys'
  int grown;
  int bad;                // some token's values have a group that is no number
  int pad;
  uint8_t groups[kKeys];  // which groups, where bad
};

template <int DP>
struct TcSmem {
  static constexpr int kTile = kKeys * DP * 2;  // bytes of a tile of 128 rows or tokens
  static constexpr int kQ = 0, kK = 2 * kTile, kV = kK + 2 * kTile, kScales = kV + 2 * kTile;
  static constexpr int kBars = kScales + kScaleSlots * (int)sizeof(TileScales), kTotal = kBars + 256 + 1024;
};
// barriers
enum { kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kSFull = 8, kPReady = 12, kPDone = 16, kOFull = 18, kQReady = 20, kScFull = 22, kBarCount = 26 };  // kSFull, kPReady: 2 w + half

// Waits for a phase of a barrier, suspended for up to a microsecond at a time; false after two seconds.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
  uint64_t begin = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity), "r"(1000u)
          : "memory");
      if (ok) return true;
    }
    const uint64_t now = bulk::now_ns();
    if (begin == 0) begin = now;
    else if (now - begin > bulk::kWaitNs) return false;
  }
}

// A segment's geometry, as every role works it out.
struct Segment {
  Seq s;
  int units, length, run, kv, starts, ends;
  Rows rows;
  __device__ __forceinline__ Segment(const AttnArgs &a, const Place &at, long long left) : s(a, at.b) {
    if (s.rows == 0) return;
    units = s.units(a, at.tile), length = s.length(a, at.tile);
    run = left < units - at.unit ? (int)left : units - at.unit;
    kv = block_of(a, at.block);
    rows = rows_of(a, s, kv, at.block - kv * a.parts, at.tile);
    starts = at.unit == 0, ends = at.unit + run == units;
  }
  __device__ __forceinline__ void next(const AttnArgs &a, Place *at, long long *left) const {
    *left -= run;
    at->unit = 0;
    if (++at->tile == s.tiles) {
      at->tile = 0;
      if (++at->block == a.blocks) at->block = 0, ++at->b;
    }
  }
};

// What one unpacking thread fetches of a tile: per round (two) and slab (DP / 64)
// 32 codes of a token, its scales and zero point.
template <int BITS>
__device__ __forceinline__ void fetch_codes(const uint8_t *p, uint32_t *w) {
  if constexpr (BITS == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x, w[1] = v.y;
  } else if constexpr (BITS == 3) {
    const uint32_t *s = reinterpret_cast<const uint32_t *>(p);
    w[0] = __ldg(s), w[1] = __ldg(s + 1), w[2] = __ldg(s + 2);
  } else {
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}
// Codes 8 x .. 8 x + 7 of 32 as unpack_row takes them.
template <int BITS>
__device__ __forceinline__ uint2 chunk_of(const uint32_t *w, int x) {
  if constexpr (BITS == 8) return make_uint2(w[2 * x], w[2 * x + 1]);
  if constexpr (BITS == 4) return make_uint2(w[x], 0);
  if constexpr (BITS == 2) return make_uint2(x & 1 ? w[x >> 1] >> 16 : w[x >> 1] & 0xffffu, 0);
  const uint32_t v = x == 0 ? w[0] : x == 1 ? __funnelshift_r(w[0], w[1], 24) : x == 2 ? __funnelshift_r(w[1], w[2], 16) : w[2] >> 8;
  return make_uint2(v & 0xffffffu, 0);
}

// The unpacking warps of the keys or of the values: a segment's tokens to tiles of
// f16. Two lanes have a token, 32 channels each of a slab of 64; a lane has a token
// in each of kRounds runs of 16.
template <int DP, int B>
struct Unpacker {
  static constexpr int kSlabs = DP / 64;
  using S = TcSmem<DP>;
  const AttnArgs &a;
  const qwha_cache &c;
  const bool values;
  uint8_t *smem;
  uint32_t bars, one;
  bool ok = true;
  bool coarse = false;       // scales far apart were met
  uint32_t it = 0;           // tiles so far
  uint32_t w[kRounds][kSlabs][B];  // raw codes of the next tile's tokens
  float scale[kRounds][kSlabs];  // of the lane's groups
  float factor[kSlabs];      // of the scales of the lane's channels (the keys: of all): follows the largest met by any of the warps
  uint8_t zero[kRounds][kSlabs], bad[kRounds];
  bool on[kRounds];

  __device__ __forceinline__ Unpacker(const AttnArgs &a_, bool values_, uint8_t *smem_, uint32_t bars_, uint32_t one_)
      : a(a_), c(values_ ? a_.v : a_.k), values(values_), smem(smem_), bars(bars_), one(one_) {}

  // The scales and zero points of the lane's groups, and which of them are no numbers. Values of such a group stay out of
  // the products, where they would meet weights of zero; keys go in as they are.
  __device__ __forceinline__ void scales(int64_t row, int ng, int r) {
    int b = 0;
#pragma unroll
    for (int i = 0; i < kSlabs; ++i) {
      const int d = 64 * i + 32 * (threadIdx.x & 1), g = ng > 1 && d < c.head_dim ? d / c.group : 0;
      float x = __ldg(c.scales + row * ng + g);
      zero[r][i] = __ldg(c.zeros + row * ng + g);
      if (values && !(fabsf(x) < INFINITY)) b |= 1 << g, x = 0.f;
      scale[r][i] = d < c.head_dim ? x : none(i);
    }
    bad[r] = (uint8_t)b;
  }
  // A scale that changes no factor, for what is not there.
  __device__ __forceinline__ float none(int i) const { return 16.f * inverse2(factor[i]); }

  // (code - zero) times the scale, which comes as the sum of two f16 numbers: the product is rounded once.
  __device__ __forceinline__ void write(uint8_t *row, int token, int r, int i, float factor, bool live) {
    Zero<B> z;
    z.set((zero[r][i] | 0xe400u) * 0x10001u);
    const int half = threadIdx.x & 1;
    const float full = scale[r][i] * factor;
    const __half2 share = __float2half2_rn(full), rest = __float2half2_rn(full - __low2float(share));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t v[4] = {0, 0, 0, 0};
      if (live) {
        unpack_row<B>(chunk_of<B>(w[r][i], x), z, one, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 d = reinterpret_cast<const __half2 &>(v[k]), p = __hfma2(d, share, __hmul2(d, rest));
          v[k] = reinterpret_cast<const uint32_t &>(p);
        }
      }
      *reinterpret_cast<uint4 *>(row + (((4 * half + x) ^ (token & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }

  __device__ __forceinline__ void wait(int bar, uint32_t parity) { ok = ok && wait_for(bars + 8 * bar, parity); }

  // Whether the lane's 32 codes all equal their zero point.
  __device__ __forceinline__ bool idle(int r, int i) const {
    bool same = zero[r][i] < 1u << B;
#pragma unroll
    for (int k = 0; k < B; ++k) same &= w[r][i][k] == idle_word<B>(zero[r][i], k);
    return same;
  }

  __device__ __forceinline__ void run(const Segment &g, const Place &at) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % (kUnpackWarps / 2), half = lane & 1, D = c.head_dim, ng = D / c.group;
    const int32_t *table = a.pages + (int64_t)at.b * a.max_pages;
    // which new tokens of a tree any row of the tile sees
    unsigned long long seen = ~0ull;
    if (a.tree) {
      seen = 0;
      for (int j = lane; j < g.rows.tokens; j += 32) seen |= (unsigned long long)a.tree[g.s.row0 + g.rows.j0 + j];
#pragma unroll
      for (int o = 1; o < 32; o *= 2) seen |= __shfl_xor_sync(~0u, seen, o);
    }
    const int past = g.s.past, mine = warp * (16 * kRounds) + (lane >> 1);
    int t0 = at.unit * kKeys + mine;
    int page[kRounds];
    // the pages of the lane's tokens, which are within the table, since lengths are cut there; -2 where there is none to
    // fetch. They are used a tile later.
    auto ask = [&](bool any) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int t = t0 + 16 * r;
        page[r] = !any || t >= g.length || (a.tree && t >= past && !(seen >> (t - past) & 1)) ? -2 : __ldg(table + page_of(a, t));
      }
    };
    auto fetch = [&] {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        on[r] = (uint32_t)page[r] < (uint32_t)a.k.n_pages;
        bad[r] = 0;
        if (!on[r]) {
#pragma unroll
          for (int i = 0; i < kSlabs; ++i) scale[r][i] = none(i);
          if (page[r] != -2) atomicOr(a.err, kErrPage);
          continue;
        }
        const int t = t0 + 16 * r;
        const int64_t row = ((int64_t)page[r] * a.k.page_size + (t - page_of(a, t) * a.k.page_size)) * c.heads + g.kv;
        const uint8_t *src = c.codes + row * (D / 8 * B) + half * (4 * B);
#pragma unroll
        for (int i = 0; i < kSlabs; ++i)
          if (32 * (2 * i + half) < D) fetch_codes<B>(src + i * (8 * B), w[r][i]);
        scales(row, ng, r);
      }
    };
#pragma unroll
    for (int i = 0; i < kSlabs; ++i) factor[i] = kNoScale;
    ask(true);
    fetch();
    t0 += kKeys;
    ask(g.run > 1);
    uint8_t *tiles = smem + (values ? S::kV : S::kK);
    for (int u = 0; u < g.run; ++u, ++it) {
      const int st = it & 1;
      TileScales &sc = *reinterpret_cast<TileScales *>(smem + S::kScales + (it % kScaleSlots) * sizeof(TileScales));
      float grow[kSlabs];
      int any_bad = 0;
      // Scales that times the factor lie outside kTcLeast .. kTcTop: a distance in bits, of which one comparison takes both
      // ends (0 too), since the factor is a power of two.
      uint32_t far = 0;
#pragma unroll
      for (int i = 0; i < kSlabs; ++i) {
        grow[i] = 1.f;
        const uint32_t shift = __float_as_uint(factor[i]) - (__float_as_uint(kTcLeast) + __float_as_uint(1.f));
#pragma unroll
        for (int r = 0; r < kRounds; ++r) far = max(far, __float_as_uint(fabsf(scale[r][i])) + shift);
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) any_bad |= bad[r];
      const int grown = any_of(far > __float_as_uint(kTcTop) - __float_as_uint(kTcLeast));
      if (grown) {
        uint32_t *top_s = reinterpret_cast<uint32_t *>(smem + S::kBars + 8 * kBarCount + 16) + (values ? 4 : 0);
        if (threadIdx.x % kUnpackers < 4) top_s[threadIdx.x % kUnpackers] = 0;
        meet();
        // codes that all equal their zero point have no say, whatever their scale
        float top[kSlabs];
#pragma unroll
        for (int i = 0; i < kSlabs; ++i) {
          top[i] = 0.f;
#pragma unroll
          for (int r = 0; r < kRounds; ++r) {
            const float x = fabsf(scale[r][i]);
            if (!on[r] || 32 * (2 * i + half) >= D || !(x < INFINITY)) continue;
            if (x * factor[i] > kTcTop && idle(r, i)) scale[r][i] = 0.f;
            else top[i] = fmaxf(top[i], x);
          }
        }
#pragma unroll
        for (int i = 0; i < kSlabs; ++i) atomicMax(top_s + (values ? 2 * i + half : 0), __float_as_uint(top[i]));
        meet();
#pragma unroll
        for (int i = 0; i < kSlabs; ++i) {
          int e = 127 + 6 - ((int)(top_s[values ? 2 * i + half : 0] >> 23) - 127 + 2);
          e = e < 1 ? 1 : e > 247 ? 247 : e;
          const float now = fminf(factor[i], __uint_as_float((uint32_t)e << 23));
          grow[i] = now * inverse2(factor[i]), factor[i] = now;
#pragma unroll
          for (int r = 0; r < kRounds; ++r)
            coarse |= on[r] && 32 * (2 * i + half) < D && scale[r][i] != 0.f && fabsf(scale[r][i]) * now < kTcLeast;
        }
        meet();
      }
      if (values) {
        any_bad = any_of(any_bad);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
          if (const int other = __shfl_xor_sync(~0u, bad[r], 1); half == 0) sc.groups[mine + 16 * r] = (uint8_t)(bad[r] | other);
        if (threadIdx.x % kUnpackers < 2) {
#pragma unroll
          for (int i = 0; i < kSlabs; ++i) sc.values[2 * i + half] = factor[i], sc.grow[2 * i + half] = grow[i];
          sc.bad = any_bad, sc.grown = grown;
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          unsigned x = __ballot_sync(~0u, on[r]) & 0x55555555u;  // two lanes a token: the even bits together
          x = (x | x >> 1) & 0x33333333u, x = (x | x >> 2) & 0x0f0f0f0fu, x = (x | x >> 4) & 0x00ff00ffu, x = (x | x >> 8) & 0xffffu;
          if (lane == 0) reinterpret_cast<uint16_t *>(sc.live)[warp * kRounds + r] = (uint16_t)x;
        }
        if (threadIdx.x % kUnpackers == 0) sc.keys = factor[0];
      }
      arrive(bars + 8 * (kScFull + it % kScaleSlots));
      wait((values ? kVEmpty : kKEmpty) + st, (it >> 1 & 1) ^ 1);
      uint8_t *tile = tiles + st * S::kTile + mine * 128;
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
#pragma unroll
        for (int i = 0; i < kSlabs; ++i)
          write(tile + i * (kKeys * 128) + r * (16 * 128), mine, r, i, factor[i], on[r] && 32 * (2 * i + half) < D);
      bulk::fence_proxy();
      arrive(bars + 8 * ((values ? kVFull : kKFull) + st));
      if (u + 1 < g.run) {  // the next tile's codes are on their way while this one is multiplied
        fetch();
        t0 += kKeys;
        ask(u + 2 < g.run);
      }
    }
  }
  // the unpacking threads of the keys, or of the values
  __device__ __forceinline__ void meet() const { asm volatile("bar.sync %0, %1;" ::"r"(values ? 3 : 2), "n"(kUnpackers) : "memory"); }
  __device__ __forceinline__ int any_of(int x) const {  // whether it is true of any of them
    int any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.or.pred q, %3, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(x), "n"(kUnpackers), "r"(values ? 3 : 2)
                 : "memory");
    return any;
  }
};

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) attention_tc_kernel(const __grid_constant__ AttnArgs a, uint32_t one) {
  using S = TcSmem<DP>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024u - (saddr(raw) & 1023u)) & 1023u);
  const uint32_t base = saddr(smem), bars = base + S::kBars;
  uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + S::kBars + 8 * kBarCount);
  volatile int *coarse_s = reinterpret_cast<int *>(tmem_s + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kIssue = kUnpackWarps + kSoftWarps;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bulk::init(bars + 8 * (kKFull + i), kUnpackers), bulk::init(bars + 8 * (kVFull + i), kUnpackers);
      bulk::init(bars + 8 * (kKEmpty + i), 1), bulk::init(bars + 8 * (kVEmpty + i), 1);
      bulk::init(bars + 8 * (kPDone + i), 1), bulk::init(bars + 8 * (kOFull + i), 1), bulk::init(bars + 8 * (kQReady + i), 128);
    }
    for (int i = 0; i < 4; ++i) bulk::init(bars + 8 * (kSFull + i), 1), bulk::init(bars + 8 * (kPReady + i), 128);
    for (int i = 0; i < kScaleSlots; ++i) bulk::init(bars + 8 * (kScFull + i), kUnpackWarps * 32);
    bulk::fence_init();
  }
  if (warp == kIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_s)), "r"(kTcCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  if (threadIdx.x == 0) {
    a.part_desc[2 * blockIdx.x] = a.part_desc[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    *coarse_s = 0;
  }
  Place at;
  long long left = my_share(a, &at);
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_s;

  if (warp < kUnpackWarps) {
    // ------------------------------------------------------------ unpacking
    const bool values = warp >= kUnpackWarps / 2;
    auto work = [&](auto bits) {
      Unpacker<DP, decltype(bits)::value> unpack(a, values, smem, bars, one);
      while (left > 0) {
        const Segment g(a, at, left);
        if (g.s.rows == 0) {
          ++at.b;
          continue;
        }
        if (threadIdx.x == 0 && (long long)g.s.past + (a.tree && g.s.rows > 64 ? 64 : g.s.rows) > a.cap) atomicOr(a.err, kErrPage);
        unpack.run(g, at);
        g.next(a, &at, &left);
      }
      if (!unpack.ok) atomicOr(a.err, kErrTc);
      if (unpack.coarse) *coarse_s = kPieceCoarse;
    };
    switch (values ? a.v.bits : a.k.bits) {
      case 2: work(std::integral_constant<int, 2>()); break;
      case 3: work(std::integral_constant<int, 3>()); break;
      case 4: work(std::integral_constant<int, 4>()); break;
      default: work(std::integral_constant<int, 8>());
    }
  } else if (warp < kIssue) {
    // ------------------------------------------------------------ softmax: a row a thread
    const int w = (warp - kUnpackWarps) / 4, r = (warp & 3) * 32 + lane;  // tile of rows; row of it (TMEM lane)
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // (unpacking takes whole groups of four warps: warp % 4 is the quarter)
    const uint32_t s_at = tmem + lanes + 128 * w, o_at = tmem + lanes + 256 + 128 * w;
    uint8_t *q_tile = smem + S::kQ + w * S::kTile;
    bool ok = true;
    uint32_t it = 0, halves = 0, slot = 0, segment = 0;  // tiles (and halves) of this tile of rows, tiles of the CTA; segments with rows in it
    auto wait = [&](int bar, uint32_t parity) { ok = ok && wait_for(bars + 8 * bar, parity); };
    while (left > 0) {
      const Segment g(a, at, left);
      if (g.s.rows == 0) {
        ++at.b;
        continue;
      }
      const int n = g.rows.n - 128 * w;  // rows of this tile
      const int out_slot = 2 * blockIdx.x + (g.starts ? 1 : 0);
      if (n > 0) {
        // ---- queries: 2^15 near the row's largest, rotated; S's columns keep what registers do not
        const int rr = 128 * w + r, D = a.k.head_dim, had = a.k.had_block;
        const bool real = r < n;
        const __nv_bfloat16 *q_row = static_cast<const __nv_bfloat16 *>(a.q) +
                                     (real ? g.rows.q_row(rr) * a.q_stride + (int64_t)g.rows.q_head(rr) * D : 0);
        float top = 0.f;
#pragma unroll 1
        for (int x = 0; x < DP / 32; ++x) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = real && 32 * x < D;  // (whole runs of 32)
            io<__nv_bfloat16>::unpack(in ? __ldg(reinterpret_cast<const uint4 *>(q_row + 32 * x) + i) : make_uint4(0, 0, 0, 0), v + 8 * i);
          }
          rotate32<1, 32>(v, had);
          uint32_t u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]), top = fmaxf(top, fabsf(v[i]));
          store32(s_at + 32 * x, u);
        }
        stores_done();
        if (had > 32) {
          top = 0.f;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float v[32];
            load_across<DP>(s_at + 8 * i, v);
            rotate32<8, 4>(v, had / 4);
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, fabsf(v[k]));
#pragma unroll
            for (int x = 0; x < DP / 32; ++x) store8(s_at + 32 * x + 8 * i, v + 8 * x);
          }
          stores_done();
        }
        const float by_q = a.scale2 * (had > 1 ? a.unit_k : 1.f);
        const uint32_t top_bits = __float_as_uint(fabsf(top * by_q));
        int e = (int)(top_bits >> 23) - 127 + 1;
        e = top_bits == 0 || top_bits >= 0x7f800000u ? 0 : e < -100 ? -100 : e;
        const float up = __uint_as_float((uint32_t)(127 + 15 - e) << 23), f = __uint_as_float((uint32_t)(127 - 15 + e) << 23);
#pragma unroll 1
        for (int x = 0; x < DP / 32; ++x) {
          uint32_t u[32];
          load32(s_at + 32 * x, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = pair16(__uint_as_float(u[8 * i + k]) * by_q * up, __uint_as_float(u[8 * i + k + 4]) * by_q * up);
            *reinterpret_cast<uint4 *>(q_tile + (x >> 1) * (kRowsTile * 128) + r * 128 + (((4 * (x & 1) + i) ^ (r & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        fence_before();
        bulk::fence_proxy();
        arrive(bars + 8 * (kQReady + w));

        // ---- what the row sees
        const int j = g.rows.j0 + (real ? rr / g.rows.heads : 0);
        const int past = g.s.past, lim = a.tree ? past : past + j + 1, safe = a.tree ? past : past + g.rows.j0 + 1;
        const unsigned long long mask = a.tree && real ? (unsigned long long)a.tree[g.s.row0 + j] : 0;
        float m = -INFINITY, l = 0.f;  // m: the maximum less kTcShift, so that weights are 2^kTcShift at it
        uint32_t nan_groups = 0;
        float4 factors = make_float4(1.f, 1.f, 1.f, 1.f);  // the values' after the last tile
        int t0 = at.unit * kKeys;
        for (int u = 0; u < g.run; ++u, ++it, t0 += kKeys) {
          const uint32_t tile = slot + u;
          // A segment's first scores before its scales: rows that skip segments are ahead of the others, and the slot's
          // barrier might still be at an earlier phase of the same parity. Scores are not made before the weights of the
          // tile before are taken, so that from the first ones on the barrier is at this tile's phase or has just left it.
          if (u == 0) wait(kSFull + 2 * w, it & 1);
          wait(kScFull + tile % kScaleSlots, tile / kScaleSlots & 1);
          const TileScales &sc = *reinterpret_cast<const TileScales *>(smem + S::kScales + (tile % kScaleSlots) * sizeof(TileScales));
          const uint4 live = *reinterpret_cast<const uint4 *>(sc.live);
          const float fk = f * inverse2(sc.keys);
          const f32x2 ff = both(fk, fk);
          const bool masked = t0 + kKeys > safe || (live.x & live.y & live.z & live.w) != ~0u;
          uint32_t vis[4] = {live.x, live.y, live.z, live.w};
          if (masked) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int tb = t0 + 32 * x, left_of = lim - tb, d = tb - past;
              uint32_t s = left_of >= 32 ? ~0u : left_of > 0 ? (1u << left_of) - 1u : 0u;
              if (a.tree) s |= d >= 64 || d <= -32 ? 0u : d >= 0 ? (uint32_t)(mask >> d) : (uint32_t)(mask << -d);
              vis[x] &= s;
            }
          }
          // (taken while the weights are due: behind them the slot may be another tile's)
          if (u + 1 == g.run) factors = *reinterpret_cast<const float4 *>(sc.values);
          if (sc.bad) {
            for (int t = 0; t < 32; ++t)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (vis[x] >> t & 1) nan_groups |= sc.groups[32 * x + t];
          }
          // One copy of this loop's code for both halves and both tries: more of it does not stay in the instruction
          // cache (unrolled, 730 us for 4 chunks of 1021 behind 2048 where this took 440).
#pragma unroll 1
          for (int h = 0; h < 2; ++h, ++halves) {
            const uint32_t from = s_at + 64 * h, on0 = h ? vis[2] : vis[0], on1 = h ? vis[3] : vis[1];
            wait(kSFull + 2 * w + h, it & 1);
            fence_after();
            float turn = 1.f;  // of the sums so far
            auto raise = [&] {  // the maximum to the half's largest visible score
              float top = -INFINITY;
#pragma unroll 1
              for (int x = 0; x < 2; ++x) {
                const uint32_t on = x ? on1 : on0;
                uint32_t v[32];
                load32(from + 32 * x, v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (on >> i & 1) top = fmaxf(top, __uint_as_float(v[i]));
              }
              const float now = fmaxf(m, top * fk - kTcShift);
              turn = now == -INFINITY ? 1.f : exp2_fast(m - now);
              m = now;
            };
            // rows that have seen nothing have no maximum yet
            if (__any_sync(~0u, m == -INFINITY)) raise();
            uint32_t p[32];
            auto weights = [&](auto hidden) {  // and their sum, for the maximum as it stands
              const float base = m == -INFINITY ? 0.f : m;
              const f32x2 mm = both(-base, -base);
              f32x2 total[2] = {0, 0};
              float v[2][16];
              columns16(from, v[0]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                float *z = v[x & 1];
                columns_done(z);
                if (x < 3) columns16(from + 16 * (x + 1), v[(x + 1) & 1]);  // on its way meanwhile
                uint32_t on = ~0u;
                if constexpr (decltype(hidden)::value) on = (x >> 1 ? on1 : on0) >> (16 * (x & 1));
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  float e[2];
                  split(fma2(both(z[i], z[i + 1]), ff, mm), e[0], e[1]);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    e[k] = exp2_fast(e[k]);
                    if constexpr (decltype(hidden)::value) e[k] = on >> (i + k) & 1 ? e[k] : 0.f;
                  }
                  total[i >> 1 & 1] = add2(total[i >> 1 & 1], both(e[0], e[1]));
                  p[8 * x + i / 2] = pair16(e[0], e[1]);
                }
              }
              float s0, s1;
              split(add2(total[0], total[1]), s0, s1);
              return s0 + s1;
            };
            float part;
#pragma unroll 1
            for (bool again = u + h > 0;; again = false) {
              part = masked ? weights(std::true_type()) : weights(std::false_type());
              if (!again || !__any_sync(~0u, !(part <= kTcSum))) break;
              const float before = turn;
              raise();
              turn *= before;
            }
            store32(from, p);  // over scores that have been read
            // the sums so far in the new units, once the products before are done
            const bool grown = h == 0 && sc.grown;
            if (u + h > 0 && __any_sync(~0u, turn != 1.f || grown)) {
              wait(kPDone + w, (halves - 1) & 1);
              fence_after();
#pragma unroll 1
              for (int x = 0; x < DP / 32; ++x) {
                const float by = grown ? turn * sc.grow[x] : turn;
                uint32_t v[32];
                load32(o_at + 32 * x, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
                store32(o_at + 32 * x, v);
              }
            }
            l = (u + h > 0 ? l * turn : 0.f) + part;
            stores_done();
            fence_before();
            arrive(bars + 8 * (kPReady + 2 * w + h));
          }
        }
        // ---- the rows
        wait(kOFull + w, segment & 1);
        ++segment;
        fence_after();
        const bool done = g.starts && g.ends;
        const float share = done ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const int had_v = done ? a.v.had_block : 0;
        const int64_t row = real ? g.rows.q_row(rr) : 0, head = real ? g.rows.q_head(rr) : 0;
        const int DV = a.v.head_dim;
        auto put = [&](int c0, float *v) {  // eight channels from c0 on
          if (!real || c0 >= DV) return;
          if (done) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (row * a.q_heads + head) * DV + c0) = io<__nv_bfloat16>::pack(v);
          } else {
            float4 *dst = reinterpret_cast<float4 *>(piece_values(a, out_slot, rr) + c0);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]), dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        };
#pragma unroll 1
        for (int x = 0; x < DP / 32; ++x) {
          const float by = inverse2(x == 0 ? factors.x : x == 1 ? factors.y : x == 2 ? factors.z : factors.w) * share;
          uint32_t u[32];
          load32(o_at + 32 * x, u);
          float v[32];  // (place i of a chunk of eight is channel (i >> 1) + 4 (i & 1))
#pragma unroll
          for (int i = 0; i < 32; ++i) v[(i & ~7) + (i >> 1 & 3) + 4 * (i & 1)] = __uint_as_float(u[i]) * by;
          if (nan_groups && nan_groups >> (32 * x / a.v.group) & 1)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __int_as_float(0x7fc00000);
          rotate32<1, 32>(v, had_v);
          if (had_v > 1)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= a.unit_v;
          if (had_v > 32) {  // bits 5 and 6 of the channel: once all are back
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
            store32(o_at + 32 * x, u);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) put(32 * x + 8 * i, v + 8 * i);
          }
        }
        if (had_v > 32) {
          stores_done();
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float v[32];
            load_across<DP>(o_at + 8 * i, v);
            rotate32<8, 4>(v, had_v / 4);
#pragma unroll
            for (int x = 0; x < DP / 32; ++x) put(32 * x + 8 * i, v + 8 * x);
          }
        }
        if (real) {
          if (!done) piece_stats(a, out_slot, rr)[0] = m, piece_stats(a, out_slot, rr)[1] = l;
          else if (a.lse) a.lse[row * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        fence_before();
      }
      slot += g.run;
      if (threadIdx.x == kUnpackWarps * 32 && !(g.starts && g.ends))
        a.part_desc[out_slot] = make_int4(at.b, at.block, at.tile, g.ends ? kPieceThere | kPieceEnds : kPieceThere);
      g.next(a, &at, &left);
    }
    if (!ok) atomicOr(a.err, kErrTc);
  } else {
    // ------------------------------------------------------------ products
    bool ok = true;
    if (wide::elected()) {
      // D fp32, A and B f16; S: both K-major, N 128; O: A in TMEM, B MN-major, N DP
      constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kKeys / 2 >> 3) << 17) | (8u << 24);
      constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(DP >> 3) << 17) | (8u << 24);
      uint32_t it = 0, tiles[2] = {0, 0}, segment[2] = {0, 0};
      auto wait = [&](int bar, uint32_t parity) {
        ok = ok && wait_for(bars + 8 * bar, parity);
        fence_after();
      };
      // half h of the tile's tokens: 64 rows of 128 bytes on in a slab
      auto scores = [&](int w, int st, int h) {
        const uint64_t q = sw128(base + S::kQ + w * S::kTile), k = sw128(base + S::kK + st * S::kTile + h * (64 * 128));
#pragma unroll
        for (int x = 0; x < DP / 16; ++x) {
          const uint32_t off = (x >> 2) * (kKeys * 128 >> 4) + (x & 3) * 2;
          wide::product(tmem + 128 * w + 64 * h, q + off, k + off, kIdescS, x != 0);
        }
        commit(bars + 8 * (kSFull + 2 * w + h));
      };
      auto values = [&](int w, int st, int h, bool add) {
        const uint64_t v = sw128_mn(base + S::kV + st * S::kTile + h * (64 * 128));
#pragma unroll
        for (int x = 0; x < kKeys / 32; ++x)
          product_t(tmem + 256 + 128 * w, tmem + 128 * w + 64 * h + 8 * x, v + x * (16 * 128 >> 4), kIdescO, add || x != 0);
        commit(bars + 8 * (kPDone + w));
      };
      while (left > 0) {
        const Segment g(a, at, left);
        if (g.s.rows == 0) {
          ++at.b;
          continue;
        }
        const int count = g.rows.n > 128 ? 2 : 1;
        for (int w = 0; w < count; ++w) wait(kQReady + w, segment[w] & 1);
        for (int u = 0; u <= g.run; ++u) {  // scores of tile u behind values of tile u - 1, half by half
          const int st = it & 1, before = (it - 1) & 1;
          const bool more = u < g.run;
          if (more) wait(kKFull + st, it >> 1 & 1);
          if (u > 0) wait(kVFull + before, (it - 1) >> 1 & 1);
          for (int h = 0; h < 2; ++h)
            for (int w = 0; w < count; ++w) {
              if (u > 0) {
                wait(kPReady + 2 * w + h, (tiles[w] - 1) & 1);
                values(w, before, h, u + h > 1);
                if (!more && h) commit(bars + 8 * (kOFull + w));
              }
              if (more) scores(w, st, h);
            }
          for (int w = 0; w < count; ++w) tiles[w] += more, segment[w] += !more;
          if (more) commit(bars + 8 * (kKEmpty + st));
          if (u > 0) commit(bars + 8 * (kVEmpty + before));
          it += more;
        }
        g.next(a, &at, &left);
      }
      // the last rows' readers have met kOFull; nothing is in flight behind it
      if (!ok) atomicOr(a.err, kErrTc);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *coarse_s) a.part_desc[2 * blockIdx.x].w |= *coarse_s;
  if (warp == kIssue) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcCols) : "memory");
  }
}

template <int DP>
cudaError_t launch_tc(const AttnArgs &a, cudaStream_t s) {
  static std::atomic<size_t> allowed[64];
  auto kernel = attention_tc_kernel<DP>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), TcSmem<DP>::kTotal, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<a.ctas, kTcThreads, TcSmem<DP>::kTotal, s>>>(a, 0x64006400u);
  return cudaGetLastError();
}

}  // namespace

// Heads of whole runs of 32 channels up to 128, in groups of whole runs; bf16.
bool attention_tc_takes(const AttnArgs &a) {
  const int D = a.k.head_dim;
  return !a.f32 && D % 32 == 0 && D <= 128 && a.k.group % 32 == 0 && a.v.group % 32 == 0;
}
cudaError_t launch_attention_tc(const AttnArgs &a, cudaStream_t s) {
  return a.k.head_dim <= 64 ? launch_tc<64>(a, s) : launch_tc<128>(a, s);
}

}  // namespace qwha
