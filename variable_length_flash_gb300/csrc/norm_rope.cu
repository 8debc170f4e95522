// Root-mean-square norm of each head of packed queries and keys with the rotary positions in the same
// pass, and its gradients:
//     r = 1 / sqrt(mean_c x_c^2 + eps),   y = R(t) (r w o x),
//     g = R(-t) dy,   dw = sum over tokens and heads of r g o x,
//     dx = r (g o w) - x r^3 mean_c(g_c w_c x_c),
// with R(t) as in rope.cu.  r is formed again in the backward: the rows it needs are read there anyway.
//
// Bound: HBM; forward every element read once and written once, backward x and dy read once and dx written
// once.  G lanes (a power of two, at least a row's units) have a token and walk `hpt` heads, so sines,
// cosines and weights are made once for them; a head's sums go over its G lanes by shuffles.  A lane's
// columns are the same for every row, so dw is summed in registers over all its rows, then over
// the block's tokens, and a second launch adds the blocks' parts: every sum in a fixed order.
//
// Measured: 20011 tokens of 40 heads of 128 in bf16, sliced from a fused projection, 77 us (79% of the copy
// rate; the weights times sine and cosine are made once for a token, which took it from 92), in fp32 123 (98%); the
// gradients of 16384 tokens of 32 heads of 96 in fp16, 64 columns of which turn in pairs of neighbours, 70.4 us (63%),
// in fp32 104 (86%), of heads of 128 in bf16 69 (86%), in fp32 135 (88%).  At 96 a
// quarter of what it issues is for lanes that have no columns (12 chunks of a row over 8 lanes), and the sums,
// weights and turns that a lane keeps leave one block an SM its registers, eight warps.  So what the next heads need
// is on its way to shared memory meanwhile, each thread's to places of its own (85 us with the loads in
// registers, four heads at a time), and two numbers go through an instruction where there is one for two (74
// without).  Two heads at a time 73, two such blocks an SM 116.  64 tokens 4.1 us, which is a launch.
#include "kernels.h"
#include "rope.cuh"
#include "tc_common.cuh"

namespace vlf {
namespace {

using namespace turning;

constexpr int kMostBlocks = 152 * 2;  // of the backward: the parts of dw that the workspace has room for

__device__ __forceinline__ float weight_at(const void *w, int dtype, int c) {
  if (!w) return 1.f;
  if (dtype == VLF_F32) return ld(static_cast<const float *>(w) + c);
  if (dtype == VLF_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]);
  return __half2float(static_cast<const __half *>(w)[c]);
}

constexpr int kSlots = 3;  // of the backward: heads' values on their way or in use

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Grid y: a run of hpt heads of q or k; x: runs of 256 / G tokens, walked with the grid's stride.  Lane
// u of a token's G has its units u, u + G, ... (NU of them; one where they hold 16 bytes).  HEADS:
// heads whose loads are in flight.
template <typename T, int V, bool INTER, int NU, int HEADS, bool BWD, bool ODD>
__global__ void __launch_bounds__(256, BWD || V == 1 ? 1 : 2) norm_rope_kernel(const NormRopeParams p) {
  constexpr bool AHEAD = BWD && V > 1;
  extern __shared__ __align__(16) uint4 slots[];  // [kSlots][HEADS][4][256]
  __shared__ unsigned long long F[128];
  __shared__ float red[BWD ? 512 * V : 1][BWD && NU > 1 ? NU : 1];
  const int half = p.rot / 2, nrot = half / V;
  __shared__ float w[256 + 8];  // (a unit's columns may pass the end, as its weights may)
  const int phases_q = (p.h_q + p.hpt - 1) / p.hpt, ph = blockIdx.y;
  const bool is_k = ph >= phases_q;
  const Rows &rows = is_k ? p.k : p.q;
  tc::pdl_trigger();
  tc::pdl_wait();
  {
    // (both loads before a store, which would hold the second one up; half <= 128, d <= 256)
    const int c = threadIdx.x;
    const float f = c < half ? ld(p.inv_freq + c) : 0.f, x = c < p.d ? weight_at(rows.w, p.w_dtype, c) : 0.f;
    if (c < half) F[c] = turns_of(f);
    w[c] = x;
    if (c < 8) w[256 + c] = 0.f;
  }
  __syncthreads();
  const int ntail = ((p.d - p.rot + V - 1) / V + 1) / 2, units = nrot + ntail;
  const int G = p.lanes, run = 256 / G, u = threadIdx.x % G, g = threadIdx.x / G;
  const uint32_t mask = (G == 32 ? 0xffffffffu : (1u << G) - 1) << (threadIdx.x % 32 & ~(G - 1));
  const int h0 = (is_k ? ph - phases_q : ph) * p.hpt, h1 = min(h0 + p.hpt, is_k ? p.h_k : p.h_q);
  const float over_d = 1.f / (float)p.d;
  using C = Chunk<T, V>;

  // what this lane has of a row: per unit its columns, its weights
  bool have[NU], two[NU], rot[NU];
  int ca[NU], cb[NU];
  float wa[BWD ? NU : 1][V], wb[BWD ? NU : 1][V], sa[BWD ? NU : 1][V], sb[BWD ? NU : 1][V];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int un = u + n * G;
    have[n] = un < units;
    const Unit<V, INTER> at(have[n] ? un : 0, nrot, ntail, half, p.d, p.first);
    two[n] = have[n] && at.two;
    rot[n] = have[n] && at.rot;
    ca[n] = at.ca;
    cb[n] = at.cb;
    if constexpr (BWD) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        wa[n][e] = have[n] ? w[ca[n] + e] : 0.f;
        wb[n][e] = two[n] ? w[cb[n] + e] : 0.f;
        sa[n][e] = sb[n][e] = 0.f;
      }
    }
  }
  // AHEAD: the l's and h's of a unit's pairs (Unit::columns), two pairs in a register pair for the fp32 instructions that
  // have two of each operand: they are most of what the kernel issues
  constexpr int P = V / 2 > 0 ? V / 2 : 1;
  uint64_t wl[P], wh[P], sl[P], sh[P];
  auto low = [&](const float (&a)[V], const float (&b)[V], int e) { return INTER && V > 1 ? (e < V / 2 ? a : b)[2 * e % V] : a[e]; };
  auto high = [&](const float (&a)[V], const float (&b)[V], int e) { return INTER && V > 1 ? (e < V / 2 ? a : b)[2 * e % V + 1] : b[e]; };
  auto pairs = [&](const float (&a)[V], const float (&b)[V], uint64_t (&l)[P], uint64_t (&h)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      l[k] = tc::f2pack(low(a, b, 2 * k), low(a, b, 2 * k + 1));
      h[k] = tc::f2pack(high(a, b, 2 * k), high(a, b, 2 * k + 1));
    }
  };
  if constexpr (AHEAD) {
    pairs(wa[0], wb[0], wl, wh);
#pragma unroll
    for (int k = 0; k < P; ++k) sl[k] = sh[k] = 0;
  }
  // HEADS heads of a token at a time
  C x[HEADS][NU], y[HEADS][NU], dx[BWD ? HEADS : 1][NU], dy[BWD ? HEADS : 1][NU];
  const long long step = (long long)gridDim.x * run;
  // AHEAD: what a thread reads of the heads after the next ones goes to its own places in shared memory meanwhile
  int slot = 0, to_slot = 0, next_h = h0;
  long long next_tok = (long long)blockIdx.x * run + g;
  auto fetch = [&]() {
    if (next_tok < p.total && have[0]) {
      const T *x0 = static_cast<const T *>(rows.x) + next_tok * rows.x_stride + (long long)next_h * p.d;
      const T *dy0 = static_cast<const T *>(rows.dy) + next_tok * rows.dy_stride + (long long)next_h * p.d;
      const uint32_t to = tc::smem_u32(slots) + ((uint32_t)to_slot * HEADS * 4 * 256 + threadIdx.x) * 16;
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (next_h + i >= h1) continue;
        copy16(to + (4 * i) * 4096, x0 + i * p.d + ca[0]);
        copy16(to + (4 * i + 1) * 4096, x0 + i * p.d + cb[0]);
        copy16(to + (4 * i + 2) * 4096, dy0 + i * p.d + ca[0]);
        copy16(to + (4 * i + 3) * 4096, dy0 + i * p.d + cb[0]);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    to_slot = to_slot == kSlots - 1 ? 0 : to_slot + 1;
    if ((next_h += HEADS) >= h1) {
      next_h = h0;
      next_tok += step;
    }
  };
  if constexpr (AHEAD)
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) fetch();
  for (long long tok = (long long)blockIdx.x * run + g; tok < p.total; tok += step) {
    // The weights and the rotation of a pair (l, h) in one: forward y_l = x_l A - x_h B, y_h = x_h C + x_l D with
    // A = w_l cos, B = w_h sin, C = w_h cos, D = w_l sin; backward with g = R(-t) dy alone: A = C = cos, B = D = -sin.
    float A[NU][V], B[NU][V], Cc[NU][V], Dd[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const Unit<V, INTER> at(have[n] ? u + n * G : 0, nrot, ntail, half, p.d, p.first);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float cs = 1.f, sn = 0.f;
        if (rot[n]) turn(ld(p.positions + (long long)at.axis[e] * p.total + tok), F[at.pair[e]], cs, sn);
        if (BWD) sn = -sn;
        A[n][e] = cs;
        B[n][e] = sn;
        if constexpr (!BWD) {
          int l, hi;
          at.columns(e, l, hi);
          const float wl = w[l], wh = w[hi];
          A[n][e] = wl * cs;
          B[n][e] = wh * sn;
          Cc[n][e] = wh * cs;
          Dd[n][e] = wl * sn;
        }
      }
    }
    uint64_t A2[P], B2[P], N2[P];
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        A2[k] = tc::f2pack(A[0][2 * k], A[0][2 * k + 1]);
        B2[k] = tc::f2pack(B[0][2 * k], B[0][2 * k + 1]);
        N2[k] = tc::f2pack(-B[0][2 * k], -B[0][2 * k + 1]);
      }
    }
    T *out0 = static_cast<T *>(rows.out) + tok * rows.out_stride + (long long)h0 * p.d;
    const T *x0 = static_cast<const T *>(rows.x) + tok * rows.x_stride + (long long)h0 * p.d;
    const T *dy0 = BWD ? static_cast<const T *>(rows.dy) + tok * rows.dy_stride + (long long)h0 * p.d : nullptr;
    for (int h = h0; h < h1; h += HEADS, x0 += HEADS * p.d, dy0 += BWD ? HEADS * p.d : 0, out0 += HEADS * p.d) {
      if constexpr (AHEAD) {
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
        const uint4 *at = slots + (slot * HEADS * 4 * 256 + threadIdx.x);
        slot = slot == kSlots - 1 ? 0 : slot + 1;
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
          x[i][0] = *reinterpret_cast<const C *>(at + 4 * i * 256);
          y[i][0] = *reinterpret_cast<const C *>(at + (4 * i + 1) * 256);
          dx[i][0] = *reinterpret_cast<const C *>(at + (4 * i + 2) * 256);
          dy[i][0] = *reinterpret_cast<const C *>(at + (4 * i + 3) * 256);
        }
      } else
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (h + i >= h1) continue;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!have[n]) continue;
          x[i][n] = *reinterpret_cast<const C *>(x0 + i * p.d + ca[n]);
          y[i][n] = *reinterpret_cast<const C *>(x0 + i * p.d + cb[n]);
          if constexpr (BWD) {
            dx[i][n] = *reinterpret_cast<const C *>(dy0 + i * p.d + ca[n]);
            dy[i][n] = *reinterpret_cast<const C *>(dy0 + i * p.d + cb[n]);
          }
        }
      }
      if constexpr (AHEAD) {
        uint64_t gl[HEADS][P], gh[HEADS][P];
        float ss[HEADS], xs[HEADS];
        auto values2 = [&](const C &c0, const C &c1, uint64_t (&l)[P], uint64_t (&h)[P]) {
          float a[V], b[V];
          c0.get(a);
          c1.get(b);
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (ODD && !two[0]) b[e] = 0.f;
          pairs(a, b, l, h);
        };
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
          ss[i] = xs[i] = 0.f;
          if (h + i >= h1 || !have[0]) continue;
          uint64_t xl[P], xh[P], dl[P], dh[P], s2 = 0, t2 = 0;
          values2(x[i][0], y[i][0], xl, xh);
          values2(dx[i][0], dy[i][0], dl, dh);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            gl[i][k] = tc::fma2(dh[k], N2[k], tc::mul2(dl[k], A2[k]));
            gh[i][k] = tc::fma2(dl[k], B2[k], tc::mul2(dh[k], A2[k]));
            s2 = tc::fma2(xl[k], xl[k], tc::fma2(xh[k], xh[k], s2));
            t2 = tc::fma2(tc::mul2(gl[i][k], wl[k]), xl[k], t2);
            t2 = tc::fma2(tc::mul2(gh[i][k], wh[k]), xh[k], t2);
          }
          const float2 s = tc::f2unpack(s2), t = tc::f2unpack(t2);
          ss[i] = s.x + s.y;
          xs[i] = t.x + t.y;
        }
        for (int o = G / 2; o > 0; o /= 2) {
#pragma unroll
          for (int i = 0; i < HEADS; ++i) {
            ss[i] += __shfl_xor_sync(mask, ss[i], o);
            xs[i] += __shfl_xor_sync(mask, xs[i], o);
          }
        }
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
          if (h + i >= h1 || !have[0]) continue;
          const float r = rsqrtf(fmaf(ss[i], over_d, p.eps)), pull = -xs[i] * over_d * r * r * r;
          const uint64_t r2 = tc::f2pack(r, r), p2 = tc::f2pack(pull, pull);
          uint64_t xl[P], xh[P];
          values2(x[i][0], y[i][0], xl, xh);
          float oa[V], ob[V];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const uint64_t vl = tc::mul2(gl[i][k], r2), vh = tc::mul2(gh[i][k], r2);
            sl[k] = tc::fma2(vl, xl[k], sl[k]);
            sh[k] = tc::fma2(vh, xh[k], sh[k]);
            const float2 ol = tc::f2unpack(tc::fma2(xl[k], p2, tc::mul2(vl, wl[k])));
            const float2 oh = tc::f2unpack(tc::fma2(xh[k], p2, tc::mul2(vh, wh[k])));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int e = 2 * k + q;
              const float l1 = q ? ol.y : ol.x, h1_ = q ? oh.y : oh.x;
              if constexpr (INTER) {
                float *o = e < V / 2 ? oa : ob;
                o[2 * e % V] = l1;
                o[2 * e % V + 1] = h1_;
              } else {
                oa[e] = l1;
                ob[e] = h1_;
              }
            }
          }
          C ra, rb;
          ra.set(oa);
          rb.set(ob);
          *reinterpret_cast<C *>(out0 + i * p.d + ca[0]) = ra;
          if (two[0]) *reinterpret_cast<C *>(out0 + i * p.d + cb[0]) = rb;
        }
        continue;
      }
      // a head's values in fp32 (what a lane does not have is zero), and its gradients turned back
      auto values = [&](int i, int n, float (&a)[V], float (&b)[V]) {
        x[i][n].get(a);
        y[i][n].get(b);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (ODD && !two[n]) b[e] = 0.f;
      };
      auto turned = [&](int i, int n, float (&ga)[V], float (&gb)[V]) {
        float da[V], db[V];
        dx[i][n].get(da);
        dy[i][n].get(db);
        rotate<V, INTER>(da, db, A[n], B[n], ga, gb);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (ODD && !two[n]) gb[e] = 0.f;
      };
      // the sums of all heads in flight go over the lanes together: one after the other they wait for
      // a shuffle at each step (20011 tokens of 40 heads: 109 us where this took 92)
      float ss[HEADS], xs[HEADS], ga[BWD ? HEADS : 1][NU][V], gb[BWD ? HEADS : 1][NU][V];
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        ss[i] = xs[i] = 0.f;
        if (h + i >= h1) continue;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!have[n]) continue;
          float a[V], b[V];
          values(i, n, a, b);
#pragma unroll
          for (int e = 0; e < V; ++e) ss[i] = fmaf(a[e], a[e], fmaf(b[e], b[e], ss[i]));
          if constexpr (BWD) {
            turned(i, n, ga[i][n], gb[i][n]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              xs[i] = fmaf(ga[i][n][e] * wa[n][e], a[e], xs[i]);
              xs[i] = fmaf(gb[i][n][e] * wb[n][e], b[e], xs[i]);
            }
          }
        }
      }
      for (int o = G / 2; o > 0; o /= 2) {
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
          ss[i] += __shfl_xor_sync(mask, ss[i], o);
          if (BWD) xs[i] += __shfl_xor_sync(mask, xs[i], o);
        }
      }
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (h + i >= h1) continue;
        const float r = rsqrtf(fmaf(ss[i], over_d, p.eps));
        const float pull = BWD ? xs[i] * over_d * r * r * r : 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!have[n]) continue;
          float a[V], b[V], oa[V], ob[V];
          values(i, n, a, b);
          if constexpr (BWD) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float va = ga[i][n][e] * r, vb = gb[i][n][e] * r;
              sa[n][e] = fmaf(va, a[e], sa[n][e]);
              sb[n][e] = fmaf(vb, b[e], sb[n][e]);
              oa[e] = fmaf(-a[e], pull, va * wa[n][e]);
              ob[e] = fmaf(-b[e], pull, vb * wb[n][e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              a[e] *= r;
              b[e] *= r;
            }
            rotate<V, INTER>(a, b, A[n], B[n], Cc[n], Dd[n], oa, ob);
          }
          C ra, rb;
          ra.set(oa);
          rb.set(ob);
          *reinterpret_cast<C *>(out0 + i * p.d + ca[n]) = ra;
          if (two[n]) *reinterpret_cast<C *>(out0 + i * p.d + cb[n]) = rb;
        }
      }
    }
  }
  if constexpr (BWD) {
    if (!p.part) return;
    float *sums = &red[0][0];  // [run][d]
    if constexpr (AHEAD) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 l = tc::f2unpack(sl[e / 2]), h = tc::f2unpack(sh[e / 2]);
        const float l1 = e % 2 ? l.y : l.x, h1_ = e % 2 ? h.y : h.x;
        if constexpr (INTER) {
          (e < V / 2 ? sa : sb)[0][2 * e % V] = l1;
          (e < V / 2 ? sa : sb)[0][2 * e % V + 1] = h1_;
        } else {
          sa[0][e] = l1;
          sb[0][e] = h1_;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (have[n]) sums[g * p.d + ca[n] + e] = sa[n][e];
        if (two[n]) sums[g * p.d + cb[n] + e] = sb[n][e];
      }
    __syncthreads();
    float *part = p.part + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * p.d;
    for (int c = threadIdx.x; c < p.d; c += 256) {
      float s = 0.f;
      for (int i = 0; i < run; ++i) s += sums[i * p.d + c];
      part[c] = s;
    }
  }
}

// dw: grid y is q or k, x 32 columns; the blocks' parts [begin, end) in order, eight at a time.
__global__ void __launch_bounds__(256) norm_rope_weights_kernel(const float *part, int d, int q_parts, int parts,
                                                               void *dwq, void *dwk, int w_dtype) {
  __shared__ float red[8][32];
  tc::pdl_trigger();
  tc::pdl_wait();
  void *dw = blockIdx.y ? dwk : dwq;
  if (!dw) return;
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
  const int end = blockIdx.y ? parts : q_parts;
  float s = 0.f;
  if (c < d)
    for (int i = (blockIdx.y ? q_parts : 0) + r; i < end; i += 8) s += part[(long long)i * d + c];
  red[r][threadIdx.x % 32] = s;
  __syncthreads();
  if (r == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    if (w_dtype == VLF_F32) static_cast<float *>(dw)[c] = s;
    else if (w_dtype == VLF_BF16) static_cast<__nv_bfloat16 *>(dw)[c] = __float2bfloat16_rn(s);
    else static_cast<__half *>(dw)[c] = __float2half_rn(s);
  }
}

template <typename T, bool BWD>
cudaError_t launch(NormRopeParams p, cudaStream_t st) {
  constexpr int VW = 16 / sizeof(T);
  // 16-byte accesses where every row, half and tail starts and ends on 16 bytes
  auto whole = [&](long long n) { return n % VW == 0; };
  auto rows = [&](const Rows &r) { return whole(r.x_stride) && whole(r.out_stride) && (!BWD || whole(r.dy_stride)); };
  const bool vec = whole(p.rot / 2) && whole(p.d) && rows(p.q) && (p.h_k == 0 || rows(p.k));
  const int v = vec ? VW : 1;
  const int units = p.rot / 2 / v + ((p.d - p.rot + v - 1) / v + 1) / 2;
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < units) p.lanes *= 2;
  const int run = 256 / p.lanes;
  const long long runs = ((long long)p.total + run - 1) / run;
  auto phases = [&](int hpt) { return (long long)(p.h_q + hpt - 1) / hpt + (p.h_k + hpt - 1) / hpt; };
  // heads per lane: as in rope.cu, 16 where that gives every SM a block, fewer for few tokens
  p.hpt = 16;
  // (q's runs and k's the same size where that is to be had: blocks then end together)
  if (p.h_q % 8 == 0 && p.h_k % 8 == 0 && (p.h_q % 16 || p.h_k % 16)) p.hpt = 8;
  while (p.hpt > 1 && runs * phases(p.hpt) < 152) p.hpt /= 2;
  while (phases(p.hpt) > 256) p.hpt *= 2;
  const long long y = phases(p.hpt), most = BWD ? 152 : 152 * 2;  // (as many as are resident: they end together)
  long long turns = (runs * y + most - 1) / most;
  long long x = turns ? (runs + turns - 1) / turns : 0;
  if (BWD && x * y > kMostBlocks) x = kMostBlocks / y;
  if (x > 0) {
    const bool many = p.hpt >= 8, odd = (p.d - p.rot) / v % 2 != 0;
    int heads = 1;
    auto pick = [&](auto v_, auto inter_) {
      constexpr int V = decltype(v_)::value;
      constexpr bool INTER = decltype(inter_)::value;
      constexpr int NU = V == 1 ? 4 : 1;
      constexpr int MANY = V == 1 ? 1 : BWD ? 4 : 8, FEW = V == 1 ? 1 : 2;
      heads = odd || !many ? FEW : MANY;
      if (odd || V == 1) return (const void *)norm_rope_kernel<T, V, INTER, NU, V == 1 ? 1 : 2, BWD, true>;
      return many ? (const void *)norm_rope_kernel<T, V, INTER, NU, MANY, BWD, V == 1>
                  : (const void *)norm_rope_kernel<T, V, INTER, NU, FEW, BWD, V == 1>;
    };
    using W = std::integral_constant<int, VW>;
    using One = std::integral_constant<int, 1>;
    const void *kern = vec ? (p.interleaved ? pick(W{}, std::true_type{}) : pick(W{}, std::false_type{}))
                           : (p.interleaved ? pick(One{}, std::true_type{}) : pick(One{}, std::false_type{}));
    void *args[1] = {&p};
    const int smem = BWD && vec ? kSlots * heads * 4 * 256 * 16 : 0;
    cudaError_t e = smem ? set_smem_once(kern, smem) : cudaSuccess;
    if (e == cudaSuccess) e = launch_dependent(kern, dim3((unsigned)x, (unsigned)y), 256, smem, st, args);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  if (!BWD || !p.part) return cudaSuccess;
  int d = p.d, q_parts = (int)(x * ((p.h_q + p.hpt - 1) / p.hpt)), parts = (int)(x * y), wd = p.w_dtype;
  const float *part = p.part;
  void *dwq = p.q.dw, *dwk = p.k.dw;
  void *args[7] = {&part, &d, &q_parts, &parts, &dwq, &dwk, &wd};
  const cudaError_t e = launch_dependent((const void *)norm_rope_weights_kernel, dim3((unsigned)((d + 31) / 32), 2), 256, 0, st, args);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

size_t norm_rope_workspace(int d) { return (size_t)kMostBlocks * (size_t)d * sizeof(float); }

cudaError_t norm_rope(const NormRopeParams &p, bool backward, cudaStream_t st) {
  auto go = [&](auto t) {
    using T = decltype(t);
    return backward ? launch<T, true>(p, st) : launch<T, false>(p, st);
  };
  if (p.dtype == VLF_F32) return go(float{});
  if (p.dtype == VLF_BF16) return go(__nv_bfloat16{});
  return go(__half{});
}

}  // namespace vlf
