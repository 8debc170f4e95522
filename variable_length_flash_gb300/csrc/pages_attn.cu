// Attention of packed queries over a cache of pages held in e4m3 (pages.cu): sequence s has kv_lens[s]
// keys, key j is slot j mod page of page table[s][j / page], its value byte times that page's scale.  Rows
// stand end-aligned, as in the forward.
#include "e4m3.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ fp32 FMA
// Any type and width up to 256: a block has one query row of one head, its warps take 32 keys in turn.  A
// lane has a key's whole dot product, then its columns of the output.  Each warp keeps a running
// maximum and sum; they are joined at the end.
constexpr int kFmaWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kFmaWarps) pages_fma_kernel(const PagesAttnParams a) {
  __shared__ float q[256];
  __shared__ float o_part[kFmaWarps][256], m_part[kFmaWarps], l_part[kFmaWarps];
  const Params &p = a.p;
  const int head = blockIdx.y, kv_head = head / p.group;
  int s = 0;  // the sequence of row blockIdx.x: the last that begins at it or before
  for (int end = p.num_seqs; end - s > 1;) {
    const int mid = (s + end) / 2;
    if (__ldg(p.cu_q + mid) <= (int)blockIdx.x) s = mid;
    else end = mid;
  }
  const int q0 = __ldg(p.cu_q + s), q1 = __ldg(p.cu_q + s + 1), len = __ldg(a.kv_lens + s);
  if (q0 < 0 || q0 > q1 || q1 > p.total_q || q1 - q0 > p.max_q || len < 0 ||
      (len > 0 && (len - 1) >> a.log2_page >= a.max_pages)) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_BAD_SEQLENS);
    return;
  }
  const int i = (int)blockIdx.x - q0;
  if (i < 0 || i >= q1 - q0) return;
  const long long row = (long long)(q0 + i) * p.h_q + head;
  for (int c = threadIdx.x; c < p.d_qk; c += 32 * kFmaWarps) q[c] = to_f32<T>(static_cast<const T *>(p.q)[row * p.d_qk + c]);
  __syncthreads();
  int lo, hi;
  visible_range(i, len - (q1 - q0), len, p.causal, p.window, lo, hi);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) o[c] = 0.f;
  for (int j0 = (lo & ~31) + 32 * warp; j0 < hi; j0 += 32 * kFmaWarps) {
    // (32 keys lie in one or two pages)
    const int j = j0 + lane;
    bool see = j >= lo && j < hi;
    int page = see ? __ldg(a.table + (long long)s * a.max_pages + (j >> a.log2_page)) : 0;
    if (page < 0 || page >= a.num_pages) {
      set_error(p.err, VLF_ERR_BAD_PAGES);
      see = false;
      page = 0;
    }
    const long long slot = (long long)page * p.h_kv + kv_head;
    const long long at = slot * a.page + (j & (a.page - 1));
    float x = -INFINITY;
    if (see) {
      const uint8_t *k = a.k_pages + at * p.d_qk;
      float dot = 0.f;
      int c = 0;
      if (p.d_qk % 16 == 0) {
        for (; c < p.d_qk; c += 16) {
          const uint4 r = *reinterpret_cast<const uint4 *>(k + c);
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = e4m3_pair(w[e / 2] >> 16 * (e % 2));
            dot = fmaf(q[c + 2 * e], f.x, dot);
            dot = fmaf(q[c + 2 * e + 1], f.y, dot);
          }
        }
      }
      for (; c < p.d_qk; ++c) dot = fmaf(q[c], e4m3_pair(k[c]).x, dot);
      x = dot * __ldg(a.k_scale + slot) * p.scale_log2;
    }
    float top = m;
    float y = x;
#pragma unroll
    for (int k = 16; k > 0; k /= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, k));
    top = fmaxf(top, y);
    if (top == -INFINITY) top = 0.f;  // (nothing seen yet, or NaN: exp2 of it reaches the sum)
    const float fix = exp2f(m - top), w = see ? exp2f(x - top) : 0.f;
    m = fmaxf(m, y);
    l = l * fix + w;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] *= fix;
    uint32_t seen = __ballot_sync(0xffffffffu, see);
    const float wv = see ? w * __ldg(a.v_scale + slot) : 0.f;
    while (seen) {
      const int k = __ffs(seen) - 1;
      seen &= seen - 1;
      const float f = __shfl_sync(0xffffffffu, wv, k);
      const uint8_t *v = a.v_pages + __shfl_sync(0xffffffffu, at, k) * p.d_v;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (lane + 32 * c < p.d_v) o[c] = fmaf(f, e4m3_pair(v[lane + 32 * c]).x, o[c]);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k /= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) {
    m_part[warp] = m;
    l_part[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) o_part[warp][lane + 32 * c] = o[c];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kFmaWarps; ++w) top = fmaxf(top, m_part[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kFmaWarps; ++w) sum += l_part[w] * exp2f(m_part[w] - ref);
  for (int c = threadIdx.x; c < p.d_v; c += 32 * kFmaWarps) {
    float x = 0.f;
    for (int w = 0; w < kFmaWarps; ++w) x += o_part[w][c] * exp2f(m_part[w] - ref);
    static_cast<T *>(p.out)[row * p.d_v + c] = from_f32<T>(sum == 0.f ? 0.f : x / sum);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[(long long)head * p.total_q + q0 + i] =
        sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

// Whether a sequence's rows of a kv head's group are enough for the kernel that has them as rows of its products.
bool many_rows(int max_q, int group) { return (long long)max_q * group > 32; }

}  // namespace

size_t pages_attn_workspace(int num_seqs, int max_q, int h_q, int h_kv, int d_qk, int d_v, int dtype, unsigned flags,
                            int num_sms) {
  if (num_seqs < 1 || !pages_tc_supported(d_qk, d_v, dtype, flags)) return 0;
  if (num_sms < 1) return 0;
  return many_rows(max_q, h_q / h_kv) ? pages_rows_workspace(d_qk, num_sms) : pages_tc_workspace(max_q, h_q / h_kv, d_qk, num_sms);
}

cudaError_t pages_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st) {
  const Params &p = a.p;
  // (a tensor map needs a page, and its coordinates are ints)
  const long long heads = (long long)a.num_pages * p.h_kv;
  if (pages_tc_supported(p.d_qk, p.d_v, p.dtype, p.flags) && heads > 0 && heads < 0x7fffffff)
    return many_rows(p.max_q, p.group) ? pages_rows_forward(a, workspace, num_sms, st) : pages_tc_forward(a, workspace, num_sms, st);
  const dim3 grid((unsigned)p.total_q, (unsigned)p.h_q);
  PagesAttnParams copy = a;
  void *args[1] = {&copy};
  const void *kern = p.dtype == VLF_F32    ? (const void *)pages_fma_kernel<float>
                     : p.dtype == VLF_BF16 ? (const void *)pages_fma_kernel<__nv_bfloat16>
                                           : (const void *)pages_fma_kernel<__half>;
  return launch_plain(kern, grid, 32 * kFmaWarps, 0, st, args);
}

}  // namespace vlf
