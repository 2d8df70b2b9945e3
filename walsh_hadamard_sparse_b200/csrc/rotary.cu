// Rotary positions: pairs of channels of every head turn by the angle
// positions[i] * freq[c], and are scaled by a factor.
//
// Memory bounds it (each value read and written once; 16381 tokens of 40 heads of
// 80 in fp32, 419 MB both ways: 92 us, 4.6 TB/s, where a copy takes 64; 64 tokens of 40
// heads of 128 in bf16: 5 us, a launch and two latencies). The sines and cosines of
// a token are shared by all its heads: a CTA takes a tile of tokens (or some heads
// of one, while the tokens alone do not fill the GPU), computes them into shared
// memory while its first values are on their way, and then streams 16-byte
// vectors.
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
constexpr int kInFlight = 4;     // items whose loads a thread has under way
constexpr int kTurnPairs = 1024;  // pairs of channels whose turns a CTA keeps

// Channels (c, c + rot/2) in whole vectors; (2c, 2c + 1); (c, c + rot/2) one by one.
enum { kHalfVectors, kPairs, kHalfSingle };

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

// x / d for x below 2^21, inv = 1 / d: half a step away from the border, where three roundings of 2^-24 do not matter.
__device__ __forceinline__ int quotient(int x, float inv) { return (int)(((float)x + 0.5f) * inv); }

template <typename T, int MODE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs r, int tile) {
  constexpr int V = io<T>::kVec;
  __shared__ float2 turn_s[kTurnPairs];
  const int half = r.rot / 2, D = r.head_dim;
  // items of a head: vectors, of which kHalfVectors takes two that turn together at once
  const int turned = MODE == kHalfVectors ? half / V : 0;
  const int per_head = MODE == kHalfVectors ? turned + (D - r.rot) / V : MODE == kPairs ? D / V : D - half;
  const int heads = r.heads[0] + r.heads[1];
  const int h0 = (int)((int64_t)heads * blockIdx.x / gridDim.x), h1 = (int)((int64_t)heads * (blockIdx.x + 1) / gridDim.x);
  const int per_token = (h1 - h0) * per_head;
  const float inv_head = 1.f / per_head, inv_token = 1.f / per_token, inv_half = half ? 1.f / half : 0.f;
  for (int64_t i0 = (int64_t)blockIdx.y * tile; i0 < r.n; i0 += (int64_t)gridDim.y * tile) {
    const int tokens = r.n - i0 < tile ? (int)(r.n - i0) : tile, total = tokens * per_token;
    bool first = true;
    for (int base = threadIdx.x; first || base < total; base += kRotaryThreads * kInFlight) {
      const T *src[kInFlight];
      T *dst[kInFlight];
      int at[kInFlight], turn[kInFlight];
      uint4 a[kInFlight], b[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int item = base + u * kRotaryThreads;
        at[u] = -1;
        if (item >= total) continue;
        const int tok = quotient(item, inv_token), in = item - tok * per_token, hh = quotient(in, inv_head);
        const int j = in - hh * per_head, h = h0 + hh, w = h >= r.heads[0];
        const int64_t head = (int64_t)(w ? h - r.heads[0] : h) * D, i = i0 + tok;
        turn[u] = tok * half;
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
        __syncthreads();  // the last tile's turns are used
        for (int c = threadIdx.x; c < tokens * half; c += kRotaryThreads) {
          const int tok = quotient(c, inv_half);
          turn_s[c] = turn_of(r.positions[i0 + tok], r.freq[c - tok * half], r.factor, r.inverse);
        }
        __syncthreads();
        first = false;
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (at[u] < 0) continue;
        const int c = at[u];
        const float2 *turns = turn_s + turn[u];
        if constexpr (MODE == kHalfVectors) {
          if (c < half) {
            float p[V], q[V];
            io<T>::unpack(a[u], p), io<T>::unpack(b[u], q);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float2 t = turns[c + e];
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
              const float2 t = turns[(c + e) / 2];
              const float y = p[e] * t.x - p[e + 1] * t.y;
              p[e + 1] = p[e + 1] * t.x + p[e] * t.y;
              p[e] = y;
            }
          }
          *reinterpret_cast<uint4 *>(dst[u] + c) = io<T>::pack(p);
        } else {
          const float p = __uint_as_float(a[u].x), q = __uint_as_float(a[u].y);
          if (c < half) {
            const float2 t = turns[c];
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
void launch_mode(const RotaryArgs &r, dim3 grid, int tile, cudaStream_t s) {
  if (r.pairs) rotary_kernel<T, kPairs><<<grid, kRotaryThreads, 0, s>>>(r, tile);
  else if (r.rot / 2 % io<T>::kVec == 0) rotary_kernel<T, kHalfVectors><<<grid, kRotaryThreads, 0, s>>>(r, tile);
  else rotary_kernel<T, kHalfSingle><<<grid, kRotaryThreads, 0, s>>>(r, tile);
}

}  // namespace

cudaError_t launch_rotary(qwha_dtype dt, const RotaryArgs &r, cudaStream_t s) {
  // A token's heads over several CTAs while the tokens alone do not fill the GPU; else tiles of tokens of four rounds of
  // the CTA's loads, as far as eight CTAs to an SM remain.
  const int heads = r.heads[0] + r.heads[1];
  const int64_t want = cdiv((int64_t)sm_count() * 4, r.n), values = (int64_t)heads * r.head_dim;
  int64_t tile = (int64_t)kRotaryThreads * kInFlight * 4 * (dt == QWHA_F32 ? 4 : 8) / values;
  tile = std::min({tile, r.n / ((int64_t)sm_count() * 8), r.rot ? (int64_t)kTurnPairs / (r.rot / 2) : (int64_t)64, (int64_t)64});
  tile = std::max<int64_t>(tile, 1);
  // (the items of a tile stay below 2^21: one token has at most 65535 x 2 heads of which a CTA takes some)
  const int64_t split = std::max({std::clamp<int64_t>(want, 1, std::max(1, heads / 8)), cdiv(values, 1 << 20), (int64_t)1});
  const dim3 grid((unsigned)split, (unsigned)std::min<int64_t>(cdiv(r.n, tile), 65535));
  if (dt == QWHA_F32) launch_mode<float>(r, grid, (int)tile, s);
  else launch_mode<__nv_bfloat16>(r, grid, (int)tile, s);
  return cudaGetLastError();
}

}  // namespace qwha
