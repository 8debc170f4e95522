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
#include "kernels.h"
#include "rope.cuh"

namespace vlf {
namespace {

using namespace turning;

constexpr int kMostBlocks = 152 * 8;  // of the backward: the parts of dw that the workspace has room for

__device__ __forceinline__ float weight_at(const void *w, int dtype, int c) {
  if (!w) return 1.f;
  if (dtype == VLF_F32) return __ldg(static_cast<const float *>(w) + c);
  if (dtype == VLF_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]);
  return __half2float(static_cast<const __half *>(w)[c]);
}

// Grid y: a run of hpt heads of q or k; x: runs of 256 / G tokens, walked with the grid's stride.  Lane
// u of a token's G has its units u, u + G, ... (NU of them; one where they hold 16 bytes).  HEADS:
// heads whose loads are in flight.
template <typename T, int V, bool INTER, int NU, int HEADS, bool BWD>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeParams p) {
  __shared__ unsigned long long F[128];
  __shared__ float red[BWD ? 512 * V : 1][BWD && NU > 1 ? NU : 1];
  const int half = p.rot / 2, nrot = half / V;
  for (int c = threadIdx.x; c < half; c += 256) F[c] = turns_of(__ldg(p.inv_freq + c));
  __syncthreads();
  const int ntail = ((p.d - p.rot + V - 1) / V + 1) / 2, units = nrot + ntail;
  const int G = p.lanes, run = 256 / G, u = threadIdx.x % G, g = threadIdx.x / G;
  const uint32_t mask = (G == 32 ? 0xffffffffu : (1u << G) - 1) << (threadIdx.x % 32 & ~(G - 1));
  const int phases_q = (p.h_q + p.hpt - 1) / p.hpt, ph = blockIdx.y;
  const bool is_k = ph >= phases_q;
  const int h0 = (is_k ? ph - phases_q : ph) * p.hpt, h1 = min(h0 + p.hpt, is_k ? p.h_k : p.h_q);
  const Rows &rows = is_k ? p.k : p.q;
  const float over_d = 1.f / (float)p.d;
  using C = Chunk<T, V>;

  // what this lane has of a row: per unit its columns, its weights
  bool have[NU], two[NU], rot[NU];
  int ca[NU], cb[NU], pair[NU][V], axis[NU][V];
  float wa[NU][V], wb[NU][V], sa[NU][V], sb[NU][V];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int un = u + n * G;
    have[n] = un < units;
    const Unit<V, INTER> at(have[n] ? un : 0, nrot, ntail, half, p.d, p.first);
    two[n] = have[n] && at.two;
    rot[n] = have[n] && at.rot;
    ca[n] = at.ca;
    cb[n] = at.cb;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      pair[n][e] = at.pair[e];
      axis[n][e] = at.axis[e];
      wa[n][e] = have[n] ? weight_at(rows.w, p.w_dtype, ca[n] + e) : 0.f;
      wb[n][e] = two[n] ? weight_at(rows.w, p.w_dtype, cb[n] + e) : 0.f;
      sa[n][e] = sb[n][e] = 0.f;
    }
  }
  auto sum = [&](float x) {
    for (int o = G / 2; o > 0; o /= 2) x += __shfl_xor_sync(mask, x, o);
    return x;
  };
  for (long long tok = (long long)blockIdx.x * run + g; tok < p.total; tok += (long long)gridDim.x * run) {
    float cs[NU][V], sn[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        cs[n][e] = 1.f;
        sn[n][e] = 0.f;
        if (!rot[n]) continue;
        turn(__ldg(p.positions + (long long)axis[n][e] * p.total + tok), F[pair[n][e]], cs[n][e], sn[n][e]);
        if (BWD) sn[n][e] = -sn[n][e];
      }
    const T *x0 = static_cast<const T *>(rows.x) + tok * rows.x_stride + (long long)h0 * p.d;
    const T *dy0 = BWD ? static_cast<const T *>(rows.dy) + tok * rows.dy_stride + (long long)h0 * p.d : nullptr;
    T *out0 = static_cast<T *>(rows.out) + tok * rows.out_stride + (long long)h0 * p.d;
    for (int h = h0; h < h1; h += HEADS, x0 += HEADS * p.d, dy0 += BWD ? HEADS * p.d : 0, out0 += HEADS * p.d) {
      C x[HEADS][NU], y[HEADS][NU], dx[BWD ? HEADS : 1][NU], dy[BWD ? HEADS : 1][NU];
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
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        if (h + i >= h1) continue;
        float a[NU][V], b[NU][V], ga[NU][V], gb[NU][V], ss = 0.f, xs = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!have[n]) continue;
          x[i][n].get(a[n]);
          y[i][n].get(b[n]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if (!two[n]) b[n][e] = 0.f;
            ss = fmaf(a[n][e], a[n][e], ss);
            ss = fmaf(b[n][e], b[n][e], ss);
          }
          if constexpr (BWD) {
            float da[V], db[V];
            dx[i][n].get(da);
            dy[i][n].get(db);
            rotate<V, INTER>(da, db, cs[n], sn[n], ga[n], gb[n]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              if (!two[n]) gb[n][e] = 0.f;
              xs = fmaf(ga[n][e] * wa[n][e], a[n][e], xs);
              xs = fmaf(gb[n][e] * wb[n][e], b[n][e], xs);
            }
          }
        }
        const float r = rsqrtf(fmaf(sum(ss), over_d, p.eps));
        const float pull = BWD ? sum(xs) * over_d * r * r : 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!have[n]) continue;
          float oa[V], ob[V];
          if constexpr (BWD) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float ua = a[n][e] * r, ub = b[n][e] * r;
              sa[n][e] = fmaf(ga[n][e], ua, sa[n][e]);
              sb[n][e] = fmaf(gb[n][e], ub, sb[n][e]);
              oa[e] = r * fmaf(-a[n][e], pull, ga[n][e] * wa[n][e]);
              ob[e] = r * fmaf(-b[n][e], pull, gb[n][e] * wb[n][e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              a[n][e] *= r * wa[n][e];
              b[n][e] *= r * wb[n][e];
            }
            rotate<V, INTER>(a[n], b[n], cs[n], sn[n], oa, ob);
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
  while (p.hpt > 1 && runs * phases(p.hpt) < 152) p.hpt /= 2;
  while (phases(p.hpt) > 256) p.hpt *= 2;
  const long long y = phases(p.hpt), most = BWD ? 152 * 3 : kMostBlocks;
  long long turns = (runs * y + most - 1) / most;
  long long x = turns ? (runs + turns - 1) / turns : 0;
  if (BWD && x * y > kMostBlocks) x = kMostBlocks / y;
  if (x > 0) {
    const bool many = p.hpt >= 8;
    auto pick = [&](auto v_, auto inter_) {
      constexpr int V = decltype(v_)::value;
      constexpr bool INTER = decltype(inter_)::value;
      constexpr int NU = V == 1 ? 4 : 1;
      constexpr int MANY = V == 1 ? 1 : BWD ? 4 : 8, FEW = V == 1 ? 1 : 2;
      return many ? (const void *)norm_rope_kernel<T, V, INTER, NU, MANY, BWD>
                  : (const void *)norm_rope_kernel<T, V, INTER, NU, FEW, BWD>;
    };
    using W = std::integral_constant<int, VW>;
    using One = std::integral_constant<int, 1>;
    const void *kern = vec ? (p.interleaved ? pick(W{}, std::true_type{}) : pick(W{}, std::false_type{}))
                           : (p.interleaved ? pick(One{}, std::true_type{}) : pick(One{}, std::false_type{}));
    void *args[1] = {&p};
    const cudaError_t e = launch_plain(kern, dim3((unsigned)x, (unsigned)y), 256, 0, st, args);
    if (e != cudaSuccess) return e;
  }
  if (!BWD || !p.part) return cudaSuccess;
  int d = p.d, q_parts = (int)(x * ((p.h_q + p.hpt - 1) / p.hpt)), parts = (int)(x * y), wd = p.w_dtype;
  const float *part = p.part;
  void *dwq = p.q.dw, *dwk = p.k.dw;
  void *args[7] = {&part, &d, &q_parts, &parts, &dwq, &dwk, &wd};
  return launch_plain((const void *)norm_rope_weights_kernel, dim3((unsigned)((d + 31) / 32), 2), 256, 0, st, args);
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
