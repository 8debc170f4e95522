// What the kernels that turn pairs of columns share (rope.cu, norm_rope.cu): 16-byte chunks of a row, the
// fraction of a turn in fixed point, and which columns and pairs a thread has.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace vlf {
namespace turning {

// V elements in one access (16 bytes; V = 1: one element).
template <typename T, int V> struct Chunk {
  uint4 r;
  __device__ __forceinline__ void get(float (&x)[V]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(x[i]);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T> struct Chunk<T, 1> {
  T r;
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f32<T>(r); }
  __device__ __forceinline__ void set(const float (&x)[1]) { r = from_f32<T>(x[0]); }
};

// f / 2 pi less the nearest whole number, in units of 2^-64 (as an unsigned number: mod 2^64).  Counted
// from the nearest whole number, not from the one below, a small negative turn keeps its bits.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  double t = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  return (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
}
// cos and sin of pos * F turns.
__device__ __forceinline__ void turn(int pos, unsigned long long F, float &c, float &s) {
  const long long ph = (long long)((unsigned long long)(long long)pos * F);
  // rounded to 32 bits (a half turn wraps to minus a half turn: the same angle)
  const int p32 = (int)((unsigned long long)(ph + 0x80000000ll) >> 32);
  sincospif((float)p32 * 4.6566128730773926e-10f, &s, &c);  // 2^-31: in half turns
}

// Unit u of a row: chunks u < nrot hold V pairs -- columns V u and rot / 2 + V u, whose partners they
// are, or (INTER, V > 1) the V / 2 pairs of neighbours in each --, the ones behind them two chunks of
// columns that pass through.
template <int V, bool INTER> struct Unit {
  int ca, cb;  // first columns of its two chunks
  bool rot, two;  // whether it turns; whether the second chunk is there (an odd number pass through)
  int pair[V], axis[V];
  // first[x]: the first pair of axis x (half for the axes that are not there)
  __device__ __forceinline__ Unit(int u, int nrot, int ntail, int half, int d, const int (&first)[4]) {
    rot = u < nrot;
    if (rot) {
      ca = INTER && V == 1 ? 2 * u : V * u;
      cb = INTER && V == 1 ? ca + 1 : half + V * u;
    } else {
      ca = 2 * half + V * (u - nrot);
      cb = ca + V * ntail;
    }
    two = cb < d;
    if (!two) cb = ca;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      int c = V * u + e;
      if (INTER && V > 1) c = e < V / 2 ? V / 2 * u + e : half / 2 + V / 2 * (u - 1) + e;
      pair[e] = rot ? c : 0;
      int a = 0;
#pragma unroll
      for (int x = 1; x < 4; ++x) a += pair[e] >= first[x] && first[x] < half ? 1 : 0;
      axis[e] = a;
    }
  }
  // The two columns of pair e of the unit.
  __device__ __forceinline__ void columns(int e, int &l, int &h) const {
    if constexpr (INTER && V > 1) {
      l = (e < V / 2 ? ca : cb) + 2 * (e % (V / 2));
      h = l + 1;
    } else {
      l = ca + e;
      h = cb + e;
    }
  }
};
// The two chunks' values turned, each pair by factors of its own: y_l = x_l A - x_h B, y_h = x_h C + x_l D.
template <int V, bool INTER>
__device__ __forceinline__ void rotate(const float (&a)[V], const float (&b)[V], const float (&A)[V], const float (&B)[V],
                                       const float (&C)[V], const float (&D)[V], float (&ya)[V], float (&yb)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if constexpr (INTER && V > 1) {
      float *o = e < V / 2 ? ya : yb;
      const float *i = e < V / 2 ? a : b;
      const int c = 2 * (e % (V / 2));
      o[c] = fmaf(i[c], A[e], -(i[c + 1] * B[e]));
      o[c + 1] = fmaf(i[c + 1], C[e], i[c] * D[e]);
    } else {
      ya[e] = fmaf(a[e], A[e], -(b[e] * B[e]));
      yb[e] = fmaf(b[e], C[e], a[e] * D[e]);
    }
  }
}
// The two chunks' values turned.
template <int V, bool INTER>
__device__ __forceinline__ void rotate(const float (&a)[V], const float (&b)[V], const float (&cs)[V],
                                       const float (&sn)[V], float (&ya)[V], float (&yb)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if constexpr (INTER && V > 1) {
      // pair e < V / 2: columns 2 e, 2 e + 1 of chunk a; the others of chunk b
      float *o = e < V / 2 ? ya : yb;
      const float *i = e < V / 2 ? a : b;
      const int c = 2 * (e % (V / 2));
      o[c] = fmaf(i[c], cs[e], -(i[c + 1] * sn[e]));
      o[c + 1] = fmaf(i[c + 1], cs[e], i[c] * sn[e]);
    } else {
      ya[e] = fmaf(a[e], cs[e], -(b[e] * sn[e]));
      yb[e] = fmaf(b[e], cs[e], a[e] * sn[e]);
    }
  }
}

}  // namespace turning
}  // namespace vlf
