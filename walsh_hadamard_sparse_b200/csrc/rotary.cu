// Rotary positions: pairs of channels of every head turn by the angle
// positions[i] * freq[c], and are scaled by a factor.
//
// Memory bounds it (each value read and written once). The sines and cosines of
// a token are shared by all its heads: a CTA takes one token, or some heads of
// it, computes them into shared memory while its first values are on their way,
// and then streams 16-byte vectors.
//
// The angle is formed in fp64, pos * (freq / 2 pi) turns, because in fp32 a
// position of 10^6 would leave 0.06 of a radian; the whole turns and the nearest
// quarter are taken off there, and what is left (at most an eighth of a turn)
// goes to sine and cosine in fp32.

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace qwha {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kInFlight = 4;  // items whose loads a thread has under way

// Channels (c, c + rot/2) in whole vectors; (2c, 2c + 1); (c, c + rot/2) one by one.
enum { kHalfVectors, kPairs, kHalfSingle };

template <typename T, int MODE>
struct Item {
  static constexpr int V = io<T>::kVec;
  uint4 a, b;
  const T *src;
  T *dst;
  int c;  // first channel; pairs with c + half
  bool live;
};

__device__ __forceinline__ float2 turn_of(int64_t pos, double freq, float factor, bool inverse) {
  double t = (double)pos * (freq * 0.15915494309189533577);
  const double q = rint(4.0 * t);
  const float r = (float)(2.0 * (t - 0.25 * q));  // in half turns, at most a quarter
  float s, c;
  sincospif(r, &s, &c);
  const int k = (int)((long long)q & 3);
  const float sk = k & 1 ? c : s, ck = k & 1 ? s : c;
  const float sin_a = k & 2 ? -sk : sk, cos_a = (k + 1) & 2 ? -ck : ck;
  return make_float2(cos_a * factor, (inverse ? -sin_a : sin_a) * factor);
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs r) {
  constexpr int V = io<T>::kVec;
  __shared__ float2 turn_s[128];
  const int half = r.rot / 2, D = r.head_dim;
  // items of a head: vectors, of which kHalfVectors takes two that turn together at once
  const int turned = MODE == kHalfVectors ? half / V : 0;
  const int per_head = MODE == kHalfVectors ? turned + (D - r.rot) / V : MODE == kPairs ? D / V : D - half;
  const int heads = r.heads[0] + r.heads[1];
  for (int64_t i = blockIdx.y; i < r.n; i += gridDim.y) {
    const int h0 = (int)((int64_t)heads * blockIdx.x / gridDim.x), h1 = (int)((int64_t)heads * (blockIdx.x + 1) / gridDim.x);
    const int total = (h1 - h0) * per_head;
    bool first = true;
    for (int base = threadIdx.x; first || base < total; base += kRotaryThreads * kInFlight) {
      const T *src[kInFlight];
      T *dst[kInFlight];
      int at[kInFlight];
      uint4 a[kInFlight], b[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int item = base + u * kRotaryThreads;
        at[u] = -1;
        if (item >= total) continue;
        const int hh = item / per_head, j = item - hh * per_head, h = h0 + hh, w = h >= r.heads[0];
        const int64_t head = (int64_t)(w ? h - r.heads[0] : h) * D;
        src[u] = static_cast<const T *>(r.x[w]) + i * r.x_stride[w] + head;
        dst[u] = static_cast<T *>(r.y[w]) + i * r.y_stride[w] + head;
        if constexpr (MODE == kHalfVectors) {
          at[u] = j < turned ? j * V : r.rot + (j - turned) * V;
          a[u] = *reinterpret_cast<const uint4 *>(src[u] + at[u]);
          if (j < turned) b[u] = *reinterpret_cast<const uint4 *>(src[u] + at[u] + half);
        } else if constexpr (MODE == kPairs) {
          at[u] = j * V;
          a[u] = *reinterpret_cast<const uint4 *>(src[u] + at[u]);
        } else {
          at[u] = j < half ? j : j + half;
          a[u].x = __float_as_uint(io<T>::load1(src[u] + at[u]));
          if (j < half) a[u].y = __float_as_uint(io<T>::load1(src[u] + at[u] + half));
        }
      }
      if (first) {
        __syncthreads();  // the last token's turns are used
        const int64_t pos = r.positions[i];
        for (int c = threadIdx.x; c < half; c += kRotaryThreads)
          turn_s[c] = turn_of(pos, r.freq[c], r.factor, r.inverse);
        __syncthreads();
        first = false;
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (at[u] < 0) continue;
        const int c = at[u];
        if constexpr (MODE == kHalfVectors) {
          if (c < half) {
            float p[V], q[V];
            io<T>::unpack(a[u], p), io<T>::unpack(b[u], q);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float2 t = turn_s[c + e];
              const float y = p[e] * t.x - q[e] * t.y;
              q[e] = q[e] * t.x + p[e] * t.y;
              p[e] = y;
            }
            *reinterpret_cast<uint4 *>(dst[u] + c) = io<T>::pack(p);
            *reinterpret_cast<uint4 *>(dst[u] + c + half) = io<T>::pack(q);
          } else {
            *reinterpret_cast<uint4 *>(dst[u] + c) = a[u];
          }
        } else if constexpr (MODE == kPairs) {
          float p[V];
          io<T>::unpack(a[u], p);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            if (c + e < r.rot) {
              const float2 t = turn_s[(c + e) / 2];
              const float y = p[e] * t.x - p[e + 1] * t.y;
              p[e + 1] = p[e + 1] * t.x + p[e] * t.y;
              p[e] = y;
            }
          }
          *reinterpret_cast<uint4 *>(dst[u] + c) = io<T>::pack(p);
        } else {
          const float p = __uint_as_float(a[u].x), q = __uint_as_float(a[u].y);
          if (c < half) {
            const float2 t = turn_s[c];
            io<T>::store1(dst[u] + c, p * t.x - q * t.y);
            io<T>::store1(dst[u] + c + half, q * t.x + p * t.y);
          } else {
            io<T>::store1(dst[u] + c, p);
          }
        }
      }
    }
  }
}

template <typename T>
void launch_mode(const RotaryArgs &r, dim3 grid, cudaStream_t s) {
  if (r.pairs) rotary_kernel<T, kPairs><<<grid, kRotaryThreads, 0, s>>>(r);
  else if (r.rot / 2 % io<T>::kVec == 0) rotary_kernel<T, kHalfVectors><<<grid, kRotaryThreads, 0, s>>>(r);
  else rotary_kernel<T, kHalfSingle><<<grid, kRotaryThreads, 0, s>>>(r);
}

}  // namespace

cudaError_t launch_rotary(qwha_dtype dt, const RotaryArgs &r, cudaStream_t s) {
  // a token's heads over several CTAs while the tokens alone do not fill the GPU
  const int heads = r.heads[0] + r.heads[1];
  const int64_t want = cdiv((int64_t)sm_count() * 4, r.n);
  const dim3 grid((unsigned)std::clamp<int64_t>(want, 1, std::max(1, heads / 8)), (unsigned)std::min<int64_t>(r.n, 65535));
  if (dt == QWHA_F32) launch_mode<float>(r, grid, s);
  else launch_mode<__nv_bfloat16>(r, grid, s);
  return cudaGetLastError();
}

}  // namespace qwha
