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

#include "common.cuh"
#include "gemv_mma.cuh"
#include "kernels.h"

namespace qwha {
namespace {

using gemv::load8;

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 8;  // tokens a row kernel's CTA takes (the rest are further grid rows)

// The b bytes holding codes k0 .. k0+7 of a row (k0 a multiple of 8).
__device__ __forceinline__ uint32_t run_word(const uint8_t *p, int bits) {
  if (bits == 4) return *reinterpret_cast<const uint32_t *>(p);
  if (bits == 2) return *reinterpret_cast<const uint16_t *>(p);
  return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// One warp per output row: lanes stride over the row's runs of eight codes (a
// run lies in one group, as groups are multiples of 8), then over the row's
// entries of E. Takes every group the format has.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) gemv_rows_kernel(const GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int t0 = blockIdx.y * kRowTokens;
  const int nt = a.T - t0 < kRowTokens ? a.T - t0 : kRowTokens;
  float base[kRowTokens], ad[kRowTokens];
#pragma unroll
  for (int u = 0; u < kRowTokens; ++u) base[u] = ad[u] = 0.f;
  if (row < a.d_out && a.qw) {
    const T *x = static_cast<const T *>(a.x) + (int64_t)t0 * a.d_in;
    const int runs = a.d_in / 8, ng = a.d_in / a.group;
    const uint8_t *qw = a.qw + row * runs * a.bits;
    const uint32_t mask = (1u << a.bits) - 1u;
    for (int r = lane; r < runs; r += 32) {
      const uint32_t w = run_word(qw + (int64_t)r * a.bits, a.bits);
      const int64_t g = row * ng + r * 8 / a.group;
      const float s = a.scales[g], z = (float)a.zeros[g];
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)((w >> (a.bits * i)) & mask) - z;
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
  if (row < a.d_out && a.row_ptr) {
    int64_t b = a.row_ptr[row], e = a.row_ptr[row + 1];
    if (b < 0) b = 0;
    if (e > a.p) e = a.p;
    for (int64_t j = b + lane; j < e; j += 32) {
      const int k = a.col_idx[j];
      if ((unsigned)k >= (unsigned)a.d_in) continue;
      const float c = a.coef[j];
      const float *z = a.zt + (int64_t)k * a.tp + t0;
#pragma unroll
      for (int u = 0; u < kRowTokens; ++u)
        if (u < nt) ad[u] = fmaf(c, z[u], ad[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kRowTokens; ++u) {
    if (u >= nt) break;
    const float v = warp_sum(base[u]) + a.alpha * warp_sum(ad[u]);
    if (lane == 0 && row < a.d_out)
      io<T>::store1(static_cast<T *>(a.y) + (int64_t)(t0 + u) * a.d_out + row, v);
  }
}

constexpr int kPrepThreads = 256;

// What a product needs of its tokens beforehand: the operands above (CTAs from
// `spans` on), and Z = X H, one CTA per token and span of whole Hadamard
// blocks: zt in fp32 with the tokens of one column side by side (zt[k * tp +
// t]), so that an entry of E finds its column of every token in one place, and
// z_out [T, d_in] in X's type for the backward, on request.
template <int BITS, typename T>
__global__ void __launch_bounds__(kPrepThreads) decode_prepare_kernel(const GemvArgs a, int logn, int span, int spans,
                                                                      float scale, T *z_out) {
  extern __shared__ __align__(16) float row[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product may start on the weight
  if ((int)blockIdx.x >= spans) {
    const int parts = (a.d_in + 127) / 128 * 16, i = (blockIdx.x - spans) * kPrepThreads + threadIdx.x;
    gemv::prepare_piece<BITS, T>(a, i / parts, i % parts, i < a.T * parts, a.T * a.pieces, a.xpieces, a.xsums);
    return;
  }
  const int per = (a.d_in + span - 1) / span;
  const int t = blockIdx.x / per, k0 = blockIdx.x % per * span;
  const int d = a.d_in - k0 < span ? a.d_in - k0 : span;
  const T *src = static_cast<const T *>(a.x) + (int64_t)t * a.d_in + k0;
  for (int k = threadIdx.x; k < d; k += blockDim.x) row[k] = io<T>::load1(src + k);
  __syncthreads();
  butterflies_smem_f32(row, d, logn);
  for (int k = threadIdx.x; k < d; k += blockDim.x) {
    const float v = row[k] * scale;
    if (a.zt) a.zt[(int64_t)(k0 + k) * a.tp + t] = v;
    if (z_out) io<T>::store1(z_out + (int64_t)t * a.d_in + k0 + k, v);
  }
}

template <int BITS, typename T>
cudaError_t prepare(const GemvArgs &a, int logn, void *z_out, cudaStream_t s) {
  const int n = 1 << logn;
  // spans of whole blocks, about 2048 columns where the blocks are shorter
  const int span = n >= 2048 ? n : 2048;
  const int spans = a.zt || z_out ? a.T * (int)cdiv(a.d_in, span) : 0;
  const int parts = gemv_prepares_x(a) ? a.T * (int)cdiv(a.d_in, 128) * 16 : 0;
  const size_t smem = spans ? (size_t)span * sizeof(float) : 0;
  auto kernel = decode_prepare_kernel<BITS, T>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * 4);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(spans + cdiv(parts, kPrepThreads)), kPrepThreads, smem, s>>>(
      a, logn, span, spans, (float)(1.0 / sqrt((double)n)), static_cast<T *>(z_out));
  return cudaGetLastError();
}

}  // namespace

int decode_tokens_padded(int64_t T) {
  int tp = 1;
  while (tp < T) tp *= 2;
  return tp;
}

bool gemv_on_tensor_cores(const uint8_t *qw, int group) { return qw && group % 32 == 0; }

bool gemv_prepares_x(const GemvArgs &a) { return a.xpieces; }

namespace {
int pieces_of(bool f32) { return f32 ? 3 : 1; }
// The last n-tile of a chunk is whole, whatever the group: up to seven columns more than there are.
size_t xpieces_bytes(int32_t d_in, int64_t T, bool f32) {
  return align_up((size_t)cdiv(d_in, 128) * 256 * (T * pieces_of(f32) + 7), 256);
}
}  // namespace

size_t gemv_x_bytes(int32_t d_in, int64_t T, bool f32) {
  if (T <= 0) return 0;
  return xpieces_bytes(d_in, T, f32) + align_up((size_t)cdiv(d_in, 128) * 64 * x_tiles((int)T * pieces_of(f32), 4), 256);
}

void gemv_place_x(GemvArgs *a, void *ws) {
  a->pieces = pieces_of(a->f32);
  a->xpieces = static_cast<uint4 *>(ws);
  a->xsums = reinterpret_cast<float2 *>(static_cast<char *>(ws) + xpieces_bytes(a->d_in, a->T, a->f32));
}

cudaError_t launch_decode_prepare(const GemvArgs &a, int logn, void *z_out, cudaStream_t s) {
  if (a.bits == 2)
    return a.f32 ? prepare<2, float>(a, logn, z_out, s) : prepare<2, __nv_bfloat16>(a, logn, z_out, s);
  if (a.bits == 3)
    return a.f32 ? prepare<3, float>(a, logn, z_out, s) : prepare<3, __nv_bfloat16>(a, logn, z_out, s);
  return a.f32 ? prepare<4, float>(a, logn, z_out, s) : prepare<4, __nv_bfloat16>(a, logn, z_out, s);
}

cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t s) {
  if (gemv_on_tensor_cores(a.qw, a.group))
    return a.bits == 4 ? launch_gemv_b4(a, s) : a.bits == 3 ? launch_gemv_b3(a, s) : launch_gemv_b2(a, s);
  const dim3 grid((unsigned)cdiv(a.d_out, kRowThreads / 32), (unsigned)cdiv(a.T, kRowTokens));
  if (a.f32) gemv_rows_kernel<float><<<grid, kRowThreads, 0, s>>>(a);
  else gemv_rows_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qwha
