// Attention of a batch whose sequences all start with the same keys: the keys of sequence s are the
// shared prefix [0, P) followed by its own kv_len keys,
//   logit(i, j) = scale * q_i . k_j,   j < P: prefix key j;  j >= P: own key j - P,
// with the end-aligned causal and window rules over the P + kv_len keys (row i stands at key
// i + P + kv_len - q_len).  out and lse are those of the forward on the concatenated keys.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ fp32 FMA kernel
// Every type and head width up to 256.  A block of 128 threads owns 16 query rows of one (sequence,
// head); thread t works on row t / 8 and every 8th column, over tiles of 32 keys -- the prefix's,
// then the sequence's own (a tile never crosses the two).  Shared rows stay apart from their
// neighbours: a key or value behind the segment's end is staged as zero, never read.
constexpr int kRows = 16, kTile = 32, kThreads = 128;

__device__ __forceinline__ float lanes8_max(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float lanes8_sum(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
__device__ __forceinline__ void stage(float *dst, int ld, const T *src, long long row0, int n, int cap,
                                      int heads, int head, int d) {
  for (int idx = threadIdx.x; idx < cap * d; idx += kThreads) {
    const int r = idx / d, c = idx - r * d;
    dst[r * ld + c] = r < n ? to_f32<T>(src[((size_t)(row0 + r) * heads + head) * d + c]) : 0.f;
  }
}

template <typename T, int DVPT>
__global__ void __launch_bounds__(kThreads) simt_prefix_kernel(const PrefixParams pp) {
  extern __shared__ float smem[];
  const Params &p = pp.p;
  const int s = blockIdx.z, h = blockIdx.y, hk = h / p.group;
  Seq sq;
  if (!load_seq(p, s, sq)) return;
  if (s == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_kv) != 0)) set_error(p.err, VLF_ERR_BAD_SEQLENS);
  if (s == p.num_seqs - 1 && (sq.q0 + sq.q_len != p.total_q || sq.k0 + sq.kv_len != p.total_kv))
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
  const int r0 = blockIdx.x * kRows;
  if (r0 >= sq.q_len) return;
  const int r1 = min(r0 + kRows, sq.q_len);
  const int P = pp.prefix_len, keys = P + sq.kv_len;
  const int dq = p.d_qk, dv = p.d_v, ldq = dq + 1;
  float *Qs = smem;                // [kRows][ldq]
  float *Ks = Qs + kRows * ldq;    // [kTile][ldq]
  float *Vs = Ks + kTile * ldq;    // [kTile][dv]
  float *Ps = Vs + kTile * dv;     // [kRows][kTile + 1]
  const int t = threadIdx.x, r = t >> 3, sub = t & 7, i = r0 + r;
  const bool row_ok = i < r1;
  const int off = keys - sq.q_len;
  int vlo, vhi;  // this row's visible keys
  visible_range(i, off, keys, p.causal, p.window, vlo, vhi);
  if (!row_ok) vhi = vlo;
  int lo, hi;    // the block's
  kv_band(r0, r1, sq.q_len, keys, p.causal, p.window, lo, hi);
  stage<T>(Qs, ldq, static_cast<const T *>(p.q), sq.q0 + r0, r1 - r0, kRows, p.h_q, h, dq);

  float m = -INFINITY, l = 0.f, o[DVPT];
#pragma unroll
  for (int u = 0; u < DVPT; ++u) o[u] = 0.f;
#pragma unroll 1
  for (int seg = 0; seg < 2; ++seg) {
    const int a = seg == 0 ? 0 : P, b = seg == 0 ? P : keys;  // the segment's keys
    const T *k = static_cast<const T *>(seg == 0 ? pp.k_pre : p.k);
    const T *v = static_cast<const T *>(seg == 0 ? pp.v_pre : p.v);
    const long long base = seg == 0 ? 0 : (long long)sq.k0 - P;  // packed row of key j: base + j
    const int e = min(b, hi);
#pragma unroll 1
    for (int kt = a + max(0, lo - a) / kTile * kTile; kt < e; kt += kTile) {
      const int nk = min(kTile, b - kt);
      __syncthreads();  // the tile before is consumed
      stage<T>(Ks, ldq, k, base + kt, nk, kTile, p.h_kv, hk, dq);
      stage<T>(Vs, dv, v, base + kt, nk, kTile, p.h_kv, hk, dv);
      __syncthreads();
      float sc[4], tmax = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int jj = sub + 8 * x, j = kt + jj;
        float y = -INFINITY;
        if (jj < nk && j >= vlo && j < vhi) {
          float acc = 0.f;
          for (int c = 0; c < dq; ++c) acc = fmaf(Qs[r * ldq + c], Ks[jj * ldq + c], acc);
          y = p.scale * acc;
        }
        sc[x] = y;
        tmax = fmaxf(tmax, y);
      }
      const float m_new = fmaxf(m, lanes8_max(tmax));
      float alpha = 1.f, psum = 0.f;
      if (m_new != -INFINITY) {
        alpha = expf(m - m_new);  // m = -inf: 0
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sc[x] = expf(sc[x] - m_new);  // masked: 0
          psum += sc[x];
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[x] = 0.f;
      }
      l = l * alpha + lanes8_sum(psum);
      m = m_new;
#pragma unroll
      for (int x = 0; x < 4; ++x) Ps[r * (kTile + 1) + sub + 8 * x] = sc[x];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < DVPT; ++u) o[u] *= alpha;
#pragma unroll 2
      for (int jj = 0; jj < nk; ++jj) {
        const float pj = Ps[r * (kTile + 1) + jj];
        const float *vrow = Vs + jj * dv;
#pragma unroll
        for (int u = 0; u < DVPT; ++u)
          if (sub + 8 * u < dv) o[u] = fmaf(pj, vrow[sub + 8 * u], o[u]);
      }
    }
  }
  if (!row_ok) return;
  const size_t grow = (size_t)sq.q0 + i;
  T *out = static_cast<T *>(p.out) + (grow * p.h_q + h) * dv;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int u = 0; u < DVPT; ++u)
    if (sub + 8 * u < dv) out[sub + 8 * u] = from_f32<T>(o[u] * inv);
  if (p.lse && sub == 0) p.lse[(size_t)h * p.total_q + grow] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T, int DVPT>
cudaError_t launch_simt(const PrefixParams &pp, cudaStream_t st) {
  const Params &p = pp.p;
  const int smem = (int)sizeof(float) * ((kRows + kTile) * (p.d_qk + 1) + kTile * p.d_v + kRows * (kTile + 1));
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(simt_prefix_kernel<T, DVPT>), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.max_q + kRows - 1) / kRows), p.h_q, p.num_seqs);
  simt_prefix_kernel<T, DVPT><<<grid, kThreads, smem, st>>>(pp);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t simt_by_width(const PrefixParams &pp, cudaStream_t st) {
  if (pp.p.d_v <= 64) return launch_simt<T, 8>(pp, st);
  if (pp.p.d_v <= 128) return launch_simt<T, 16>(pp, st);
  return launch_simt<T, 32>(pp, st);
}

}  // namespace

cudaError_t simt_prefix(const PrefixParams &pp, cudaStream_t st) {
  if (pp.p.dtype == VLF_F32) return simt_by_width<float>(pp, st);
  if (pp.p.dtype == VLF_BF16) return simt_by_width<__nv_bfloat16>(pp, st);
  return simt_by_width<__half>(pp, st);
}

}  // namespace vlf
