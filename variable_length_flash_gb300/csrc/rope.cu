// Rotary positions with several axes: y = R(t) x for the rows of packed queries and keys.
//
// A head's first `rot` columns form rot / 2 pairs (x_a, x_b); pair c belongs to one position axis
// (time, height, width, ...; the sections give each axis a run of consecutive pairs) and turns by
//     t = position[axis(c)][token] * inv_freq[c],
//     y_a = x_a cos t - x_b sin t,   y_b = x_b cos t + x_a sin t,
// the other columns pass through.  The gradient of x is R(-t) applied to the gradient of y, the
// same kernel with the sign of sin turned.
//
// The angle.  t grows to position * frequency, a million radians and more, where an fp32 product
// is off by whole percents of a turn.  Positions are integers, so the turn fraction is formed in
// 64-bit fixed point instead: F = frac(inv_freq / 2 pi) 2^64 (one double product per pair), and
// position * F mod 2^64 IS the fraction of a turn, with an error of |position| inv_freq 2^-55
// turns; its top 32 bits, a number in [-1/2, 1/2), go to sincospi.
//
// Bound: HBM, every element read once and written once.  A thread owns one chunk of pairs (two
// 16-byte loads: V pairs) of one token, computes its V sines and cosines once and applies them to
// `hpt` consecutive heads of q and k, so that the trigonometry and the 64-bit products are a small
// share of the instructions.
#include "common.cuh"
#include "kernels.h"

namespace vlf {
namespace {

template <typename T> struct alignas(16) Vec16 { T e[16 / sizeof(T)]; };

// V elements at p as fp32 (V = 16 / sizeof(T): one 16-byte access; V = 1: one element).
template <typename T, int V>
__device__ __forceinline__ void load_v(const T *p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f32<T>(*p);
  } else {
    const Vec16<T> v = *reinterpret_cast<const Vec16<T> *>(p);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = to_f32<T>(v.e[e]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(x[0]);
  } else {
    Vec16<T> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = from_f32<T>(x[e]);
    *reinterpret_cast<Vec16<T> *>(p) = v;
  }
}

// cos and sin of position * f radians (see the head of this file).
__device__ __forceinline__ void turn(int pos, float f, float &c, float &s) {
  double t = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  const unsigned long long F = (unsigned long long)(t * 18446744073709551616.0);
  const long long ph = (long long)((unsigned long long)(long long)pos * F);
  // rounded to 32 bits (a half turn wraps to minus a half turn: the same angle)
  const int p32 = (int)((unsigned long long)(ph + 0x80000000ll) >> 32);
  sincospif((float)p32 * 4.6566128730773926e-10f, &s, &c);  // 2^-31: in half turns
}

// One thread: chunk u of token `tok`, heads [h0, h0 + hpt).  Chunks u < half / V hold V pairs;
// the ones behind them 2 V columns that pass through.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  const int half = p.rot / 2, nrot = half / V;
  const int units = nrot + (p.copy_tail ? (p.d - p.rot + 2 * V - 1) / (2 * V) : 0);
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(id % units);
  const long long rest = id / units;
  const int tok = (int)(rest / p.phases), h0 = (int)(rest % p.phases) * p.hpt;
  if (tok >= p.total) return;
  const int h1 = min(h0 + p.hpt, p.h_q + p.h_k);
  auto in_at = [&](int h) {
    return h < p.h_q ? static_cast<const T *>(p.q) + (long long)tok * p.q_stride + (long long)h * p.d
                     : static_cast<const T *>(p.k) + (long long)tok * p.k_stride + (long long)(h - p.h_q) * p.d;
  };
  auto out_at = [&](int h) {
    return h < p.h_q ? static_cast<T *>(p.q_out) + (long long)tok * p.q_out_stride + (long long)h * p.d
                     : static_cast<T *>(p.k_out) + (long long)tok * p.k_out_stride + (long long)(h - p.h_q) * p.d;
  };
  if (u >= nrot) {  // columns that pass through (copied as they are)
    const int c0 = p.rot + (u - nrot) * 2 * V;
    for (int h = h0; h < h1; ++h) {
      const T *src = in_at(h);
      T *dst = out_at(h);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int c = c0 + w * V;
        if (c >= p.d) continue;
        if constexpr (V == 1) dst[c] = src[c];
        else *reinterpret_cast<Vec16<T> *>(dst + c) = *reinterpret_cast<const Vec16<T> *>(src + c);
      }
    }
    return;
  }
  float cs[V], sn[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = u * V + e;
    int a = 0;
#pragma unroll
    for (int x = 1; x < 4; ++x) a += c >= p.first[x] ? 1 : 0;  // (first[x] = half for unused axes)
    turn(__ldg(p.positions + (long long)a * p.total + tok), __ldg(p.inv_freq + c), cs[e], sn[e]);
    if (p.inverse) sn[e] = -sn[e];
  }
  const int ca = INTER ? 2 * V * u : V * u, cb = INTER ? ca + V : half + V * u;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const T *src = in_at(h);
    T *dst = out_at(h);
    float a[V], b[V], ya[V], yb[V];
    load_v<T, V>(src + ca, a);
    load_v<T, V>(src + cb, b);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (INTER && V > 1) {
        // neighbours: pair e is (2e, 2e + 1) of the chunk's 2 V columns, in a then b
        float *y = e < V / 2 ? &ya[2 * e] : &yb[2 * e - V];
        const float x0 = e < V / 2 ? a[(2 * e) % V] : b[(2 * e) % V];
        const float x1 = e < V / 2 ? a[(2 * e + 1) % V] : b[(2 * e + 1) % V];
        y[0] = fmaf(x0, cs[e], -(x1 * sn[e]));
        y[1] = fmaf(x1, cs[e], x0 * sn[e]);
      } else {
        ya[e] = fmaf(a[e], cs[e], -(b[e] * sn[e]));
        yb[e] = fmaf(b[e], cs[e], a[e] * sn[e]);
      }
    }
    store_v<T, V>(dst + ca, ya);
    store_v<T, V>(dst + cb, yb);
  }
}

template <typename T>
cudaError_t launch(RopeParams p, cudaStream_t st) {
  constexpr int VW = 16 / sizeof(T);
  // 16-byte accesses where every row, half and tail starts and ends on 16 bytes
  auto whole = [&](long long n) { return n % VW == 0; };
  const bool vec = whole(p.rot / 2) && whole(p.d) && whole(p.q_stride) && whole(p.q_out_stride) &&
                   (p.h_k == 0 || (whole(p.k_stride) && whole(p.k_out_stride)));
  const int v = vec ? VW : 1;
  const long long units = p.rot / 2 / v + (p.copy_tail ? (p.d - p.rot + 2 * v - 1) / (2 * v) : 0);
  if (units == 0) return cudaSuccess;  // nothing turns, and the rest is already in place
  // Heads per thread: 8 once that leaves enough threads to fill the GPU (152 SMs x 1024), fewer
  // for a decode step's few tokens, where the heads are the parallelism.
  const int heads = p.h_q + p.h_k;
  p.hpt = 8;
  while (p.hpt > 1 && units * p.total * ((heads + p.hpt - 1) / p.hpt) < 152ll * 1024) p.hpt /= 2;
  p.phases = (heads + p.hpt - 1) / p.hpt;
  const long long blocks = (units * p.total * p.phases + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (vec) {
    if (p.interleaved) rope_kernel<T, VW, true><<<grid, 256, 0, st>>>(p);
    else rope_kernel<T, VW, false><<<grid, 256, 0, st>>>(p);
  } else {
    // (one pair a thread: neighbours sit at 2u and 2u + 1)
    if (p.interleaved) rope_kernel<T, 1, true><<<grid, 256, 0, st>>>(p);
    else rope_kernel<T, 1, false><<<grid, 256, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t rope(const RopeParams &p, cudaStream_t st) {
  if (p.dtype == VLF_F32) return launch<float>(p, st);
  if (p.dtype == VLF_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}

}  // namespace vlf
