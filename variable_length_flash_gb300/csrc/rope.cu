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
// 64-bit fixed point instead: F = inv_freq / 2 pi mod 1 in units of 2^-64 (one double product per
// pair), and position * F mod 2^64 IS the fraction of a turn, with an error of at most
// |position| (|inv_freq| 2^-55 + 2^-64) turns: the product's rounding and F's own.  Its top 32 bits, a
// number in [-1/2, 1/2), go to sincospi.
//
// Bound: HBM, every element read once and written once.  A thread owns V pairs of one token (two
// 16-byte chunks, neighbouring threads on neighbouring chunks), computes their sines and cosines
// once and applies them to `hpt` consecutive heads.  The fp64 products, which this chip is slow at,
// run once per pair and block (a table in shared memory; done by each thread they took 94 us where
// this takes 65), and a block walks several runs of tokens.  Measured: 20011 tokens of 40 heads of
// 128 in bf16, sliced from a fused projection, 65 us = 94% of the copy rate; 16384 tokens of 32 heads
// of 96 in fp16, 64 columns of which turn, 35 us = 85% (segments of 64 bytes, and 782 blocks where 304 are
// resident: the third wave is half full); 64 tokens 3 us, which is a launch.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace vlf {
namespace {

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

// Grid y: a run of hpt heads of q or k; x: runs of 256 / units tokens, walked with the grid's stride.
// Thread: chunk u of a token.  Chunks u < nrot hold V pairs -- columns V u and rot / 2 + V u, whose
// partners they are, or (INTER, V > 1) the V / 2 pairs of neighbours in each --, the ones behind
// them two chunks of columns that pass through.  HEADS: heads whose loads are in flight.
template <typename T, int V, bool INTER, int HEADS>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  __shared__ unsigned long long F[128];
  const int half = p.rot / 2, nrot = half / V;
  for (int c = threadIdx.x; c < half; c += 256) F[c] = turns_of(__ldg(p.inv_freq + c));
  __syncthreads();
  const int tail = p.copy_tail ? (p.d - p.rot + V - 1) / V : 0, ntail = (tail + 1) / 2;
  const int units = nrot + ntail, run = 256 / units;
  const int u = threadIdx.x % units, g = threadIdx.x / units;
  if (g >= run) return;
  const int phases_q = (p.h_q + p.hpt - 1) / p.hpt, ph = blockIdx.y;
  const bool is_k = ph >= phases_q;
  const int h0 = (is_k ? ph - phases_q : ph) * p.hpt, h1 = min(h0 + p.hpt, is_k ? p.h_k : p.h_q);
  const bool rot = u < nrot;
  int ca, cb;  // first columns of the thread's two chunks
  if (rot) {
    ca = INTER && V == 1 ? 2 * u : V * u;
    cb = INTER && V == 1 ? ca + 1 : half + V * u;
  } else {
    ca = p.rot + V * (u - nrot);
    cb = ca + V * ntail;
  }
  const bool two = cb < p.d;  // (a tail of an odd number of chunks: its last unit has one)
  if (!two) cb = ca;
  int pair[V], axis[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    int c = V * u + e;
    if (INTER && V > 1) c = e < V / 2 ? V / 2 * u + e : half / 2 + V / 2 * (u - 1) + e;
    pair[e] = rot ? c : 0;
    int a = 0;
#pragma unroll
    for (int x = 1; x < 4; ++x) a += pair[e] >= p.first[x] && p.first[x] < half ? 1 : 0;
    axis[e] = a;
  }
  const long long si = is_k ? p.k_stride : p.q_stride, so = is_k ? p.k_out_stride : p.q_out_stride;
  const T *in = static_cast<const T *>(is_k ? p.k : p.q);
  T *out = static_cast<T *>(is_k ? p.k_out : p.q_out);
  using C = Chunk<T, V>;
  for (long long tok = (long long)blockIdx.x * run + g; tok < p.total; tok += (long long)gridDim.x * run) {
    float cs[V], sn[V];
    if (rot) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        turn(__ldg(p.positions + (long long)axis[e] * p.total + tok), F[pair[e]], cs[e], sn[e]);
        if (p.inverse) sn[e] = -sn[e];
      }
    }
    const T *src = in + tok * si + (long long)h0 * p.d;
    T *dst = out + tok * so + (long long)h0 * p.d;
    auto apply = [&](C &x, C &y) {
      float a[V], b[V], ya[V], yb[V];
      x.get(a);
      y.get(b);
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
      x.set(ya);
      y.set(yb);
    };
    // HEADS heads' loads are in flight before the first store (in place the compiler could not
    // move a load over a store by itself)
    for (int h = h0; h < h1; h += HEADS, src += HEADS * p.d, dst += HEADS * p.d) {
      C x[HEADS], y[HEADS];
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (h + i >= h1) continue;
        x[i] = *reinterpret_cast<const C *>(src + i * p.d + ca);
        y[i] = *reinterpret_cast<const C *>(src + i * p.d + cb);
      }
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (h + i >= h1) continue;
        if (rot) apply(x[i], y[i]);
        *reinterpret_cast<C *>(dst + i * p.d + ca) = x[i];
        if (two) *reinterpret_cast<C *>(dst + i * p.d + cb) = y[i];
      }
    }
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
  const int units = p.rot / 2 / v + (p.copy_tail ? ((p.d - p.rot + v - 1) / v + 1) / 2 : 0);
  if (units == 0) return cudaSuccess;  // nothing turns, and the rest is already in place
  // Heads per thread: 16 (the trigonometry is then a small share) where that still gives every one of
  // the 152 SMs a block, fewer for a decode step's few tokens, where the heads are the parallelism (908
  // tokens of 40 heads: 6.4 us with four heads each, 8.3 and 12.4 us when two or four blocks per SM were
  // asked for).
  const long long runs = ((long long)p.total + 256 / units - 1) / (256 / units);
  auto phases = [&](int hpt) { return (p.h_q + hpt - 1) / hpt + (p.h_k + hpt - 1) / hpt; };
  p.hpt = 16;
  while (p.hpt > 1 && runs * phases(p.hpt) < 152) p.hpt /= 2;
  while (phases(p.hpt) > 65535) p.hpt *= 2;
  // a grid of up to eight blocks per SM, each with the same number of runs (resident are two of the
  // kernel with eight heads in flight, 128 registers, and three with two, 74-80)
  const long long y = phases(p.hpt), turns = (runs * y + 152 * 8 - 1) / (152 * 8);
  const dim3 grid((unsigned)((runs + turns - 1) / turns), (unsigned)y);
  // (eight heads in flight take 64 registers of data: where a thread has fewer, more blocks fit instead)
  const bool many = p.hpt >= 8;
  auto pick = [&](auto v_, auto inter_) {
    constexpr int V = decltype(v_)::value;
    constexpr bool INTER = decltype(inter_)::value;
    return many ? (const void *)rope_kernel<T, V, INTER, 8> : (const void *)rope_kernel<T, V, INTER, 2>;
  };
  using W = std::integral_constant<int, VW>;
  using One = std::integral_constant<int, 1>;
  const void *kern = vec ? (p.interleaved ? pick(W{}, std::true_type{}) : pick(W{}, std::false_type{}))
                         : (p.interleaved ? pick(One{}, std::true_type{}) : pick(One{}, std::false_type{}));
  void *args[1] = {&p};
  return launch_plain(kern, grid, 256, 0, st, args);
}

}  // namespace

cudaError_t rope(const RopeParams &p, cudaStream_t st) {
  if (p.dtype == VLF_F32) return launch<float>(p, st);
  if (p.dtype == VLF_BF16) return launch<__nv_bfloat16>(p, st);
  return launch<__half>(p, st);
}

}  // namespace vlf
