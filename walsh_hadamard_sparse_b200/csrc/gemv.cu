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
#include "kernels.h"

namespace qwha {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 8;  // tokens a row kernel's CTA takes (the rest are further grid rows)

// The b bytes holding codes k0 .. k0+7 of a row (k0 a multiple of 8).
__device__ __forceinline__ uint32_t run_word(const uint8_t *p, int bits) {
  if (bits == 4) return *reinterpret_cast<const uint32_t *>(p);
  if (bits == 2) return *reinterpret_cast<const uint16_t *>(p);
  return (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16;
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *v) {
#pragma unroll
  for (int u = 0; u < 8; u += io<T>::kVec) io<T>::unpack(*reinterpret_cast<const uint4 *>(p + u), v + u);
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

// Z = X H for the few tokens of a decode call, in fp32 with the tokens of one
// column side by side (zt[k * tp + t]), so that an entry of E finds its column
// of every token in one place; and, on request, z_out [T, d_in] in X's type
// for the backward. One CTA per token and span of whole Hadamard blocks.
template <typename T>
__global__ void __launch_bounds__(512) decode_fwht_kernel(const T *__restrict__ x, int d_in, int logn, int span,
                                                          float scale, float *zt, int tp, T *z_out) {
  extern __shared__ __align__(16) float row[];
  const int t = blockIdx.y, k0 = blockIdx.x * span;
  const int d = d_in - k0 < span ? d_in - k0 : span;
  const T *src = x + (int64_t)t * d_in + k0;
  for (int k = threadIdx.x; k < d; k += blockDim.x) row[k] = io<T>::load1(src + k);
  __syncthreads();
  butterflies_smem_f32(row, d, logn);
  for (int k = threadIdx.x; k < d; k += blockDim.x) {
    const float v = row[k] * scale;
    if (zt) zt[(int64_t)(k0 + k) * tp + t] = v;
    if (z_out) io<T>::store1(z_out + (int64_t)t * d_in + k0 + k, v);
  }
}

template <typename T>
cudaError_t transform(const void *x, int T_, int d_in, int logn, float *zt, int tp, void *z_out, cudaStream_t s) {
  const int n = 1 << logn;
  // spans of whole blocks, about 2048 columns where the blocks are shorter
  const int span = n >= 2048 ? n : 2048;
  const size_t smem = (size_t)span * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(decode_fwht_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)cdiv(d_in, span), (unsigned)T_);
  decode_fwht_kernel<T><<<grid, 512, smem, s>>>(static_cast<const T *>(x), d_in, logn, span,
                                                (float)(1.0 / sqrt((double)n)), zt, tp, static_cast<T *>(z_out));
  return cudaGetLastError();
}

}  // namespace

int decode_tokens_padded(int64_t T) {
  int tp = 1;
  while (tp < T) tp *= 2;
  return tp;
}

cudaError_t launch_decode_fwht(qwha_dtype dt, const void *x, int T, int d_in, int logn, float *zt, int tp,
                               void *z_out, cudaStream_t s) {
  return dt == QWHA_F32 ? transform<float>(x, T, d_in, logn, zt, tp, z_out, s)
                        : transform<__nv_bfloat16>(x, T, d_in, logn, zt, tp, z_out, s);
}

cudaError_t launch_gemv(qwha_dtype dt, const GemvArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)cdiv(a.d_out, kRowThreads / 32), (unsigned)cdiv(a.T, kRowTokens));
  if (dt == QWHA_F32) gemv_rows_kernel<float><<<grid, kRowThreads, 0, s>>>(a);
  else gemv_rows_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qwha
