// Matrix-vector products with the packed base weight for a few tokens, and the
// adapted layer on them:
//   Y[t][i] = sum_k W_Q[i][k] X[t][k]  (+ alpha sum_{j in row i} c_j Z[t][k_j]),
//   W_Q[i][k] = scales[i][k/group] * (q[i][k] - zeros[i][k/group]),  Z = X H.
// The weight is read once, in its packed form, and never written out: for one
// token the codes are nearly all the bytes there are. A row's group factors out
// of the sum,
//   sum_k W_Q x = sum_g scales_g * sum_{k in g} (q_k - zeros_g) x_k,
// and q - zeros is a small integer, so no weight is ever rounded.

#include <algorithm>

#include "bulk.cuh"
#include "common.cuh"
#include "gemv_mma.cuh"
#include "gemv_wide.cuh"
#include "kernels.h"

namespace qwha {
namespace {

using gemv::load8;

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 8;  // tokens a row kernel's CTA takes (the rest are further grid rows)

// The BITS bytes holding codes k0 .. k0+7 of a row (k0 a multiple of 8).
template <int BITS>
__device__ __forceinline__ uint32_t run_word(const uint8_t *p) {
  if constexpr (BITS == 4) return *reinterpret_cast<const uint32_t *>(p);
  if constexpr (BITS == 2) return *reinterpret_cast<const uint16_t *>(p);
  return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// One warp per output row: lanes stride over the row's runs of eight codes (a
// run lies in one group, as groups are multiples of 8). Takes every group the
// format has, and calls without a base term.
template <int BITS, typename T>
__global__ void __launch_bounds__(kRowThreads) gemv_rows_kernel(const __grid_constant__ GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int t0 = blockIdx.y * kRowTokens;
  const int nt = a.T - t0 < kRowTokens ? a.T - t0 : kRowTokens;
  float base[kRowTokens];
#pragma unroll
  for (int u = 0; u < kRowTokens; ++u) base[u] = 0.f;
  if (row < a.d_out && a.qw) {
    const T *x = static_cast<const T *>(a.x) + (int64_t)t0 * a.d_in;
    const int runs = a.d_in / 8, ng = a.d_in / a.group;
    const uint8_t *qw = a.qw + row * runs * BITS;
    constexpr uint32_t mask = (1u << BITS) - 1u;
#pragma unroll 2  // rows of a narrow layer need two runs in flight (1024 rows, one token: 7.2 instead of 10.1 us)
    for (int r = lane; r < runs; r += 32) {
      const uint32_t w = run_word<BITS>(qw + (int64_t)r * BITS);
      const int64_t g = row * ng + r * 8 / a.group;
      const float s = a.scales[g], z = (float)a.zeros[g];
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)((w >> (BITS * i)) & mask) - z;
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u) {
        if (u >= nt) break;
        float v[8], sum = 0.f;
        load8(x + (int64_t)u * a.d_in + r * 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(q[i], v[i], sum);
        base[u] = fmaf(s, sum, base[u]);
      }
    }
  }
  unsigned again = 0;  // tokens whose sum left fp32's range
  auto put = [&](int u, float v) {
    if (a.y_ad) v += a.alpha * a.y_ad[row * a.tp + t0 + u];
    io<T>::store1(static_cast<T *>(a.y) + (int64_t)(t0 + u) * a.d_out + row, v);
  };
#pragma unroll
  for (int u = 0; u < kRowTokens; ++u) {
    if (u >= nt) break;
    const float v = warp_sum(base[u]);
    if (!gemv::finite(v)) again |= 1u << u;
    if (lane == 0 && row < a.d_out) put(u, v);
  }
  if (row >= a.d_out || !a.qw) return;
  for (; again; again &= again - 1) {  // in fp64, as gemv::plain_dot
    const int u = __ffs(again) - 1;
    const T *x = static_cast<const T *>(a.x) + (int64_t)(t0 + u) * a.d_in;
    double sum = 0.;
    for (int r = lane; r < a.d_in / 8; r += 32) {
      const int64_t g = row * (a.d_in / a.group) + r * 8 / a.group;
      const uint32_t w = run_word<BITS>(a.qw + (row * (a.d_in / 8) + r) * BITS);
      sum = fma((double)a.scales[g], gemv::run_dot<1>(w, BITS, a.zeros[g], x + r * 8), sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) put(u, (float)sum);
  }
}

constexpr int kPrepThreads = 256;
// Columns above which tcgen05 takes the product: one border, a compromise. Both sides grow with the columns, the
// unpacking into shared memory less than the other (bf16 tokens, groups of 128, us, mma.sync / tcgen05):
//   14336 x 4096, 4 bits     16: 23 / 24   20: 29 / 24   24: 31 / 24   32: 38 / 25   64: 64 / 28
//   4096 x 14336, 2 bits     16: 19 / 25   20: 25 / 27   24: 25 / 27   32: 31 / 29   64: 47 / 36
//   4096 x 14336, 3 bits     16: 21 / 29   20: 27 / 31   24: 26 / 32   32: 32 / 34   64: 48 / 42
//   1024 x 4096, 4 bits      16: 7.5 / 11  20: 9.7 / 12  24: 10 / 12   32: 11 / 14   64: 18 / 18
// At 20 columns it leaves 5 us of 29 in the first row; above it costs up to 6 of 26 where codes have three bits or
// rows are few: a border by width and rows would serve these better.
constexpr int kWideAbove = 20;

// Shared-memory place of element i of a span: four floats of padding every
// sixteen, so that sixteen consecutive elements a thread and elements sixteen
// apart are both free of bank conflicts (two ways at most).
__host__ __device__ constexpr int span_at(int i) { return i + (i >> 4) * 4; }

// NB butterfly stages from stage s on over d elements, sixteen or fewer to a
// thread and turn, in registers.
template <int NB>
__device__ __forceinline__ void span_pass(float *row, int d, int s) {
  constexpr int N = 1 << NB;
  for (int q = threadIdx.x; q < (d >> NB); q += kPrepThreads) {
    const int base = ((q >> s) << (s + NB)) | (q & ((1 << s) - 1));
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row[span_at(base + (i << s))];
#pragma unroll
    for (int h = 1; h < N; h *= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(i & h)) {
          const float x = v[i], y = v[i + h];
          v[i] = x + y, v[i + h] = x - y;
        }
#pragma unroll
    for (int i = 0; i < N; ++i) row[span_at(base + (i << s))] = v[i];
  }
  __syncthreads();
}

// Token slots of a pass of the product for many columns: they cover the padding too.
__host__ __device__ inline int wide_slots(const GemvArgs &a) { return (a.npad + a.pieces - 1) / a.pieces; }

// What a product needs of its tokens beforehand: the operands (CTAs from
// `spans` on), and Z = X H, one CTA per token and span of whole Hadamard
// blocks: zt in fp32 with the tg tokens of a group side by side, so that an
// entry of E finds its column of all of them in one place, and columns of zeros
// behind; z_out [T, d_in] in X's type for the backward, on request. Latency
// bounds it: four stages a pass, so 4096 columns take three turns through shared memory.
template <int BITS, typename T>
__global__ void __launch_bounds__(kPrepThreads) decode_prepare_kernel(const GemvArgs a, int logn, int span, int spans,
                                                                      float scale, T *z_out) {
  extern __shared__ __align__(16) float row[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product may start on the weight
  if (a.ready && blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0;
  if ((int)blockIdx.x >= spans && a.npad) {
    wide::wide_prepare<BITS, T>(a, blockIdx.x - spans, wide_slots(a));
    return;
  }
  if ((int)blockIdx.x >= spans) {
    const int parts = (a.d_in + 127) / 128 * 16, i = (blockIdx.x - spans) * kPrepThreads + threadIdx.x;
    gemv::prepare_piece<BITS, false, T>(a, i / parts, i % parts, i < a.T * parts, a.T * a.pieces, a.xpieces, a.xfac);
    return;
  }
  const int per = (a.d_in + span - 1) / span;
  const int t = blockIdx.x / per, k0 = blockIdx.x % per * span;
  const int d = a.d_in - k0 < span ? a.d_in - k0 : span;  // a multiple of 8
  const T *src = static_cast<const T *>(a.x) + (int64_t)t * a.d_in + k0;
  for (int k = threadIdx.x * 4; k < d; k += kPrepThreads * 4) {
    float v[4];
    gemv::load4(src + k, v);
    *reinterpret_cast<float4 *>(row + span_at(k)) = make_float4(v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
  for (int s = 0; s < logn; s += 4) {
    if (logn - s >= 4) span_pass<4>(row, d, s);
    else if (logn - s == 3) span_pass<3>(row, d, s);
    else if (logn - s == 2) span_pass<2>(row, d, s);
    else span_pass<1>(row, d, s);
  }
  for (int k = threadIdx.x; k < d; k += kPrepThreads) {
    const float v = row[span_at(k)] * scale;
    if (a.zt) a.zt[((int64_t)(t / a.tg) * z_cols(a.d_in) + k0 + k) * a.tg + t % a.tg] = v;
    if (z_out) io<T>::store1(z_out + (int64_t)t * a.d_in + k0 + k, v);
  }
  if (a.zt && k0 + d == a.d_in && threadIdx.x < z_cols(a.d_in) - a.d_in)
    a.zt[((int64_t)(t / a.tg) * z_cols(a.d_in) + a.d_in + threadIdx.x) * a.tg + t % a.tg] = 0.f;
}

constexpr int kEntThreads = 512, kEntWarps = kEntThreads / 32;
constexpr int kEntRows = 1024;  // rows of a CTA whose borders are kept in shared memory
constexpr int kLongRow = 256, kHugeRow = 1024;
constexpr size_t kEntSmem = 200 * 1024, kEntZ = 136 * 1024;

// 16 bytes into shared memory, zeros behind the first `bytes`.
__device__ __forceinline__ void copy16(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(bulk::saddr(dst)), "l"(src), "r"(bytes) : "memory");
}

// Sum over n entries by 1 << LANES_LOG2 lanes, four entries a lane in flight.
template <int TG, int LANES_LOG2>
__device__ __forceinline__ void row_sum(const int32_t *cols, const float *coefs, int n, const float *zs, int d_in, int lane,
                                        float *acc) {
  constexpr int L = 1 << LANES_LOG2;
#pragma unroll
  for (int i = 0; i < TG; ++i) acc[i] = 0.f;
  for (int j = lane; j < n; j += 4 * L) {
    int k[4];
    float c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool there = j + u * L < n;
      k[u] = there ? cols[j + u * L] : -1;
      c[u] = there ? coefs[j + u * L] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // behind the last entry and outside the layer: 0 times the column of zeros (0 * Z would be NaN for an infinite Z)
      if ((unsigned)k[u] >= (unsigned)d_in) k[u] = d_in, c[u] = 0.f;
      const float *z = zs + (int64_t)k[u] * TG;
      if constexpr (TG >= 4) {
#pragma unroll
        for (int i = 0; i < TG; i += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(z + i);
          acc[i] = fmaf(c[u], v.x, acc[i]), acc[i + 1] = fmaf(c[u], v.y, acc[i + 1]);
          acc[i + 2] = fmaf(c[u], v.z, acc[i + 2]), acc[i + 3] = fmaf(c[u], v.w, acc[i + 3]);
        }
      } else if constexpr (TG == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(z);
        acc[0] = fmaf(c[u], v.x, acc[0]), acc[1] = fmaf(c[u], v.y, acc[1]);
      } else {
        acc[0] = fmaf(c[u], *z, acc[0]);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < L; o *= 2)
#pragma unroll
    for (int i = 0; i < TG; ++i) acc[i] += __shfl_xor_sync(~0u, acc[i], o);
}

// The entries of E against the transformed tokens: y_ad[i][t] = sum_{j in row i}
// c_j Z[t][k_j], fp32. Gathering Z from L2 costs a sector an entry and waits
// for each, so a group of TG tokens is brought into shared memory and an entry
// a lane gathers there (down layer, five fp32 tokens, the whole call: three
// turns of two tokens 50 us, eight from L2 11 more); only layers whose single
// token does not fit gather from L2. The entries are copied to shared memory
// beside it, before the preparing launch is complete. 512 threads of 64
// registers leave a CTA of the product room on the SM (gate layer, sixteen
// tokens, the whole call: 48 us; with 1024 threads and the product behind 5
// more).
//
// Rows differ in length by orders of magnitude (the budget follows the row's
// quantization error): a CTA takes whole rows that hold its even share of the
// entries; 8 to 32 lanes, as the CTA's rows are many or few, take a row of up
// to kLongRow entries, a warp a longer one, the CTA one above kHugeRow. Every sum has one place and one order.
template <int TG>
__global__ void __launch_bounds__(kEntThreads, 2)
    decode_entries_kernel(const GemvArgs a, int buffers, int stage) {
  extern __shared__ __align__(16) float zs_all[];  // [buffers][z_cols][TG], columns [stage], coefficients [stage]
  __shared__ int rp_s[kEntRows + 1];
  __shared__ float part[kEntWarps][TG];
  __shared__ uint64_t s_bar[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 2) {
    bulk::init(bulk::saddr(s_bar + threadIdx.x), 1);
    bulk::fence_init();
  }
  auto border = [&](int r) {
    const int b = a.row_ptr[r];
    return b < 0 ? 0 : b > a.p ? (int)a.p : b;
  };
  // The CTA's rows: those whose entries start at or behind its share's first entry, before the next share's. The
  // first such row lies behind the last of every step-th row that starts before the share.
  const int64_t share = (a.p + gridDim.x - 1) / gridDim.x;
  const int step = (a.d_out + kEntThreads - 1) / kEntThreads;
  int r_of[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t at = (blockIdx.x + e) * share;
    const int r = (int)threadIdx.x * step;
    const int n = __syncthreads_count(r < a.d_out && border(r) < at);
    const int from = n ? (n - 1) * step + 1 : 0, to = n * step < a.d_out ? n * step : a.d_out;
    int more = 0;
    for (int q = from; q < to; q += kEntThreads) {
      const int i = q + (int)threadIdx.x;
      more += __syncthreads_count(i < to && border(i) < at);
    }
    r_of[e] = from + more;
  }
  const int r0 = blockIdx.x == 0 ? 0 : r_of[0], r1 = blockIdx.x == gridDim.x - 1 ? a.d_out : r_of[1] > r0 ? r_of[1] : r0;
  const bool near = r1 - r0 <= kEntRows;
  for (int i = threadIdx.x; near && i <= r1 - r0; i += kEntThreads) rp_s[i] = border(r0 + i);
  auto row_at = [&](int r) { return near ? rp_s[r - r0] : border(r); };
  // the entries of these rows, as many as there is room for, from a multiple of four on
  const int e0 = border(r0) & ~3;
  int staged = border(r1) - e0;
  staged = staged < 0 ? 0 : staged < stage ? staged : stage;
  int32_t *cols_s = reinterpret_cast<int32_t *>(zs_all + (size_t)buffers * z_cols(a.d_in) * TG);
  float *coefs_s = reinterpret_cast<float *>(cols_s + stage);
  for (int i = threadIdx.x * 4; i < staged; i += kEntThreads * 4) {
    const int64_t left = a.p - e0 - i;
    const uint32_t bytes = left < 4 ? (uint32_t)left * 4 : 16;
    copy16(cols_s + i, a.col_idx + e0 + i, bytes);
    copy16(coefs_s + i, a.coef + e0 + i, bytes);
  }

  // Z is the preparing launch's output. The product behind this launch may start once that is complete, and runs
  // beside it: it waits for `ready` before it reads the operands and for this launch before it adds the sums.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0)
    asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(a.ready) : "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("cp.async.wait_all;" ::: "memory");
  // turn n: the tokens of group n; with two buffers the next turn's Z is on its way
  const int turns = a.tp / TG, group = z_cols(a.d_in) * TG;
  const uint32_t bytes = group * 4;
  auto copy_z = [&](int n) {
    const uint32_t bar = bulk::saddr(s_bar + n % 2);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
    bulk::fence_proxy();
    bulk::copy(bulk::saddr(zs_all) + (buffers == 2 ? n % 2 * bytes : 0), a.zt + (int64_t)n * group, bytes, bar);
  };
  if (buffers && threadIdx.x == 0) copy_z(0);
  for (int n = 0; n < turns; ++n) {
    const int t0 = n * TG;
    const float *zs = !buffers ? a.zt + (int64_t)n * group : zs_all + (buffers == 2 ? n % 2 * group : 0);
    __syncthreads();  // the last turn's gathers are done (and the rows' borders are there)
    if (buffers) {
      if (threadIdx.x == 0 && (buffers == 2 ? n + 1 < turns : n > 0)) copy_z(buffers == 2 ? n + 1 : n);
      // incomplete if it gives up, reported through the error word
      if (!bulk::wait(bulk::saddr(s_bar + n % 2), (uint32_t)(n / 2 & 1))) atomicOr(a.err, kErrEntries);
      __syncwarp();
    }
    auto put = [&](int r, const float *acc) {
      float *out = a.y_ad + (int64_t)r * a.tp + t0;
      if constexpr (TG >= 4) {
#pragma unroll
        for (int i = 0; i < TG; i += 4)
          *reinterpret_cast<float4 *>(out + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < TG; ++i) out[i] = acc[i];
      }
    };
    float acc[TG];
    // the short rows, `1 << LL` lanes each
    auto short_rows = [&](auto LL) {
      constexpr int ll = decltype(LL)::value, rows = 32 >> ll;
      for (int q = r0 + warp * rows; q < r1; q += kEntWarps * rows) {
        const int r = q + (lane >> ll);
        int b = 0, len = -1;
        if (r < r1) {
          b = row_at(r);
          len = row_at(r + 1) - b;
          if (len < 0) len = 0;
        }
        const int at = b - e0;
        const bool near_by = at >= 0 && at + len <= staged;
        row_sum<TG, ll>(near_by ? cols_s + at : a.col_idx + b, near_by ? coefs_s + at : a.coef + b,
                        len > kLongRow ? 0 : len, zs, a.d_in, lane & ((1 << ll) - 1), acc);
        if ((lane & ((1 << ll) - 1)) == 0 && len >= 0 && len <= kLongRow) put(r, acc);
      }
    };
    if (r1 - r0 <= kEntWarps) short_rows(std::integral_constant<int, 5>());
    else if (r1 - r0 <= 2 * kEntWarps) short_rows(std::integral_constant<int, 4>());
    else short_rows(std::integral_constant<int, 3>());
    // a warp a long row, the CTA a huge one (the longest row would otherwise be the kernel's time)
    for (int q = r0; q < r1; q += 32) {
      const int r = q + lane;
      const int mine = r < r1 ? row_at(r + 1) - row_at(r) : 0;
      unsigned some = __ballot_sync(~0u, mine > kLongRow && mine <= kHugeRow), huge = __ballot_sync(~0u, mine > kHugeRow);
      while (some) {
        const int at = __ffs(some) - 1, b = row_at(q + at), len = row_at(q + at + 1) - b;
        some &= some - 1;
        if (((q - r0) + at) % kEntWarps != warp) continue;
        const bool near_by = b >= e0 && b - e0 + len <= staged;
        row_sum<TG, 5>(near_by ? cols_s + (b - e0) : a.col_idx + b, near_by ? coefs_s + (b - e0) : a.coef + b, len, zs,
                       a.d_in, lane, acc);
        if (lane == 0) put(q + at, acc);
      }
      while (huge) {
        const int at = __ffs(huge) - 1, b = row_at(q + at), len = row_at(q + at + 1) - b;
        huge &= huge - 1;
        const int per = (len + kEntWarps - 1) / kEntWarps, lo = warp * per < len ? warp * per : len;
        const int n_here = len - lo < per ? len - lo : per;
        row_sum<TG, 5>(a.col_idx + b + lo, a.coef + b + lo, n_here, zs, a.d_in, lane, acc);
        if (lane == 0)
#pragma unroll
          for (int i = 0; i < TG; ++i) part[warp][i] = acc[i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int i = 0; i < TG; ++i) acc[i] = warp_sum(lane < kEntWarps ? part[lane][i] : 0.f);
          if (lane == 0) put(q + at, acc);
        }
        __syncthreads();
      }
    }
  }
}

template <int TG>
cudaError_t entries(const GemvArgs &a, cudaStream_t s) {
  const size_t group_bytes = (size_t)z_cols(a.d_in) * TG * sizeof(float);
  const int buffers = 2 * group_bytes <= kEntSmem * 2 / 3 && a.tp > TG ? 2 : group_bytes <= kEntSmem ? 1 : 0;
  // a CTA an SM, with 256 entries at least
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(sm_count(), a.p / 256));
  // room for a share of the entries, and half of one more: whole rows make shares uneven
  const int64_t room = (int64_t)(kEntSmem - buffers * group_bytes) / 8, share = cdiv(a.p, grid);
  const int stage = (int)std::min<int64_t>(room, share + share / 2 + 256) & ~3;
  const size_t smem = buffers * group_bytes + (size_t)stage * 8;
  auto kernel = decode_entries_kernel<TG>;
  static std::atomic<size_t> allowed[64];
  const cudaError_t e = allow_smem((const void *)kernel, smem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kEntThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;  // overlaps the preparing launch, which is the one before
  return cudaLaunchKernelEx(&cfg, kernel, a, buffers, stage);
}

template <int BITS, typename T>
cudaError_t prepare(const GemvArgs &a, int logn, void *z_out, cudaStream_t s) {
  const int n = 1 << logn;
  // spans of whole blocks, about 2048 columns where the blocks are shorter
  const int span = n >= 2048 ? n : 2048;
  const int spans = a.zt || z_out ? a.T * (int)cdiv(a.d_in, span) : 0;
  const int passes = a.npad ? (int)cdiv(a.T, a.tpp) : 0;
  const int parts = !a.xpieces ? 0 : a.npad ? passes * wide_slots(a) * kPrepThreads : a.T * (int)cdiv(a.d_in, 128) * 16;
  const size_t smem = spans ? (size_t)span_at(span) * sizeof(float) : 0;
  auto kernel = decode_prepare_kernel<BITS, T>;
  static std::atomic<size_t> allowed[64];
  const cudaError_t e = allow_smem((const void *)kernel, smem, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(spans + cdiv(parts, kPrepThreads)), kPrepThreads, smem, s>>>(
      a, logn, span, spans, (float)(1.0 / sqrt((double)n)), static_cast<T *>(z_out));
  return cudaGetLastError();
}

}  // namespace

bool gemv_on_tensor_cores(const uint8_t *qw, int group) { return qw && group % 32 == 0; }

namespace {
int pieces_of(bool f32) { return f32 ? 3 : 1; }
// The last n-tile of a chunk is whole, whatever the group: up to seven columns more than there are.
size_t xpieces_bytes(int32_t d_in, int64_t T, bool f32) {
  return align_up((size_t)cdiv(d_in, 128) * 256 * (T * pieces_of(f32) + 7), 256);
}
}  // namespace

// A bf16 token or two by themselves: the product's CTAs make the operands, which saves the call a launch and a workspace.
// That is 4 of 17 us of an eager call of 1024 x 4096. On the GPU one token takes 5.0 us instead of 5.3 (14336 x 4096: 15.5
// instead of 15.7), two take 6.3 instead of 5.1 (17.7 instead of 15.7): every CTA repeats the work. The size bounds that
// work. One n-tile has to hold the columns; with two at most it does for every group, which workspace sizes do not know.
bool gemv_own_x(int32_t d_in, int64_t T, bool f32) {
  return T * pieces_of(f32) <= 2 && T * pieces_of(f32) * d_in <= 16384;
}

namespace {
// Tokens of a pass and its padded columns for the product of many columns; npad 0 where the other takes the call.
void wide_shape(int64_t T, bool f32, int *tpp, int *npad) {
  const int P = pieces_of(f32);
  *tpp = *npad = 0;
  if (T * P <= kWideAbove) return;
  const int64_t passes = cdiv(T * P, 128);
  *tpp = (int)cdiv(T, passes);
  *npad = (*tpp * P + 15) / 16 * 16;
}
}  // namespace

size_t gemv_x_bytes(int32_t d_in, int64_t T, bool f32) {
  if (T <= 0) return 0;
  int tpp, npad;
  wide_shape(T, f32, &tpp, &npad);
  if (npad) return (size_t)cdiv(T, tpp) * cdiv(d_in, 128) * npad * 256 + align_up(T * 4, 256);
  return xpieces_bytes(d_in, T, f32) + align_up((size_t)cdiv(d_in, 128) * 32 * x_tiles((int)T * pieces_of(f32), 4), 256);
}

void gemv_place_x(GemvArgs *a, void *ws) {
  a->pieces = pieces_of(a->f32);
  a->xpieces = static_cast<uint4 *>(ws);
  wide_shape(a->T, a->f32, &a->tpp, &a->npad);
  if (a->npad) {
    const size_t bytes = (size_t)cdiv(a->T, a->tpp) * cdiv(a->d_in, 128) * a->npad * 256;
    a->fac = reinterpret_cast<float *>(static_cast<char *>(ws) + bytes);
    return;
  }
  a->xfac = reinterpret_cast<float *>(static_cast<char *>(ws) + xpieces_bytes(a->d_in, a->T, a->f32));
}

namespace {
// Tokens of a group: as many as there are up to two, then four (a 16-byte gather) or eight, and so few that a group's
// Z fits into shared memory beside the entries where any does.
int group_tokens(int64_t T, int32_t d_in) {
  int n = T <= 2 ? (int)T : T <= 4 ? 4 : 8;
  while (n > 1 && (int64_t)n * d_in * 4 > kEntZ) n /= 2;
  return n;
}
}  // namespace

size_t gemv_z_bytes(int32_t d_out, int32_t d_in, int64_t T) {
  if (T <= 0) return 0;
  const size_t tp = cdiv(T, group_tokens(T, d_in)) * group_tokens(T, d_in);
  return align_up(tp * z_cols(d_in) * 4, 256) + align_up(tp * d_out * 4, 256) + 256;
}

void gemv_place_z(GemvArgs *a, void *ws) {
  a->tg = group_tokens(a->T, a->d_in);
  a->tp = (a->T + a->tg - 1) / a->tg * a->tg;
  a->ready = static_cast<unsigned int *>(ws);
  a->zt = reinterpret_cast<float *>(static_cast<char *>(ws) + 256);
  a->y_ad = a->zt + align_up((size_t)a->tp * z_cols(a->d_in) * 4, 256) / 4;
}

cudaError_t launch_decode_entries(const GemvArgs &a, cudaStream_t s) {
  return a.tg == 1 ? entries<1>(a, s) : a.tg == 2 ? entries<2>(a, s) : a.tg == 4 ? entries<4>(a, s) : entries<8>(a, s);
}

cudaError_t launch_decode_prepare(const GemvArgs &a, int logn, void *z_out, cudaStream_t s) {
  if (a.bits == 2)
    return a.f32 ? prepare<2, float>(a, logn, z_out, s) : prepare<2, __nv_bfloat16>(a, logn, z_out, s);
  if (a.bits == 3)
    return a.f32 ? prepare<3, float>(a, logn, z_out, s) : prepare<3, __nv_bfloat16>(a, logn, z_out, s);
  return a.f32 ? prepare<4, float>(a, logn, z_out, s) : prepare<4, __nv_bfloat16>(a, logn, z_out, s);
}

namespace {
template <int BITS>
cudaError_t gemv_rows(const GemvArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)cdiv(a.d_out, kRowThreads / 32), (unsigned)cdiv(a.T, kRowTokens));
  if (a.f32) gemv_rows_kernel<BITS, float><<<grid, kRowThreads, 0, s>>>(a);
  else gemv_rows_kernel<BITS, __nv_bfloat16><<<grid, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t s) {
  if (gemv_on_tensor_cores(a.qw, a.group))
    return a.bits == 4 ? launch_gemv_b4(a, s) : a.bits == 3 ? launch_gemv_b3(a, s) : launch_gemv_b2(a, s);
  return a.bits == 3 ? gemv_rows<3>(a, s) : a.bits == 2 ? gemv_rows<2>(a, s) : gemv_rows<4>(a, s);
}

}  // namespace qwha
