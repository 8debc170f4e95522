// Attention weight received by each key:
//   weights[g, j] = prev[g, j] + sum over the query rows i that see key j and the heads h of kv
//                   head g of exp(scale * q_i,h . k_j,g - lse[h, i]),
// the column sums of the attention matrix, recomputed from the forward's log-sum-exp.  A row whose
// lse is -inf (it sees no key) gives nothing.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ fp32 FMA kernel
// Every type and head width up to 256.  A block of 128 threads owns 32 keys of one (sequence, kv
// head) and walks the rows that may see them, all heads of the group, 16 (row, head) pairs at a
// time: thread t takes key t mod 32 against four of the pairs, so that a key's value read from
// shared memory serves four products.  Sums stay in one thread, in a fixed order.
constexpr int kKeys = 32, kPairs = 16, kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) simt_key_weights_kernel(const KeyWeightParams kp) {
  extern __shared__ float smem[];
  const Params &p = kp.p;
  const int s = blockIdx.z, hk = blockIdx.y, j0 = blockIdx.x * kKeys;
  Seq sq;
  if (!load_seq(p, s, sq)) return;
  if (s == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_kv) != 0)) set_error(p.err, VLF_ERR_BAD_SEQLENS);
  if (s == p.num_seqs - 1 && (sq.q0 + sq.q_len != p.total_q || sq.k0 + sq.kv_len != p.total_kv))
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
  if (j0 >= sq.kv_len) return;
  const int d = p.d_qk, ld = d + 1, nk = min(kKeys, sq.kv_len - j0);
  float *Ks = smem;               // [kKeys][ld]
  float *Qs = Ks + kKeys * ld;    // [kPairs][d]
  float *Ls = Qs + kPairs * d;    // [kPairs]
  float *Ws = Ls + kPairs;        // [kThreads]
  const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k);
  const int t = threadIdx.x, key = t & 31, sub = t >> 5, j = j0 + key;
  for (int idx = t; idx < kKeys * d; idx += kThreads) {
    const int r = idx / d, c = idx - r * d;
    Ks[r * ld + c] = r < nk ? to_f32<T>(k[((size_t)(sq.k0 + j0 + r) * p.h_kv + hk) * d + c]) : 0.f;
  }
  const int off = sq.kv_len - sq.q_len;
  int rlo, rhi, lo, hi;  // the rows that see this key, and the block's
  visible_rows(min(j, sq.kv_len - 1), off, sq.q_len, p.causal, p.window, rlo, rhi);
  q_band(j0, j0 + nk, sq.q_len, sq.kv_len, p.causal, p.window, lo, hi);
  float sum = 0.f;
  const long long end = (long long)hi * p.group;
  for (long long c0 = (long long)lo * p.group; c0 < end; c0 += kPairs) {
    __syncthreads();  // the pairs before are consumed
    for (int idx = t; idx < kPairs * d; idx += kThreads) {
      const int r = idx / d, c = idx - r * d;
      const long long pr = c0 + r;
      float x = 0.f;
      if (pr < end)
        x = to_f32<T>(q[((size_t)(sq.q0 + pr / p.group) * p.h_q + hk * p.group + pr % p.group) * d + c]);
      Qs[r * d + c] = x;
    }
    if (t < kPairs) {
      const long long pr = c0 + t;
      Ls[t] = pr < end ? kp.lse[(size_t)(hk * p.group + pr % p.group) * p.total_q + sq.q0 + pr / p.group] : -INFINITY;
    }
    __syncthreads();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < d; ++c) {
      const float x = Ks[key * ld + c];
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[u] = fmaf(x, Qs[(4 * sub + u) * d + c], acc[u]);
    }
    float part = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = (c0 + 4 * sub + u) / p.group;
      const float lse = Ls[4 * sub + u];
      if (i >= rlo && i < rhi && lse != -INFINITY) part += expf(p.scale * acc[u] - lse);
    }
    sum += part;
  }
  Ws[t] = sum;
  __syncthreads();
  if (t < nk) {
    const size_t at = (size_t)hk * p.total_kv + sq.k0 + j0 + t;
    const float w = (Ws[t] + Ws[t + 32]) + (Ws[t + 64] + Ws[t + 96]);
    kp.weights[at] = kp.prev ? kp.prev[at] + w : w;
  }
}

template <typename T>
cudaError_t launch_simt(const KeyWeightParams &kp, cudaStream_t st) {
  const Params &p = kp.p;
  const int smem = (int)sizeof(float) * (kKeys * (p.d_qk + 1) + kPairs * (p.d_qk + 1) + kThreads);
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(simt_key_weights_kernel<T>), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.max_kv + kKeys - 1) / kKeys), p.h_kv, p.num_seqs);
  simt_key_weights_kernel<T><<<grid, kThreads, smem, st>>>(kp);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t simt_key_weights(const KeyWeightParams &kp, cudaStream_t st) {
  if (kp.p.dtype == VLF_F32) return launch_simt<float>(kp, st);
  if (kp.p.dtype == VLF_BF16) return launch_simt<__nv_bfloat16>(kp, st);
  return launch_simt<__half>(kp, st);
}

}  // namespace vlf
