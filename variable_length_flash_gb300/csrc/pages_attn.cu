// Attention of packed queries over a cache of pages held in e4m3 (pages.cu): sequence s has kv_lens[s]
// keys, key j is slot j mod page of page table[s][j / page], its value byte times that page's scale.  Rows
// stand end-aligned, as in the forward.
#include <cooperative_groups.h>

#include "e4m3.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ fp32 FMA
// Any type and width up to 256: a block has one query row of H heads of a kv head's group, its warps take 32
// keys in turn, so a byte is read and made a number once for the H heads.  A lane has a key's whole dot products, then
// four columns of the output in 128.  Each warp keeps a running maximum and sum; they are joined at
// the end, over the cluster's blocks as well where the launch has few rows and gives a row's keys to several.
//
// Bound: latency of a warp's dependent steps (loads, sums, exponentials), then issue.  A decode step of 64 caches of
// 1000 to 16384 keys, 32 heads over 8 of 128 in fp32: 814 us, 21% of the copy rate (3451 with a block for each head
// and bytes of values read singly; 907 with four keys in flight); width 96 in bf16 703 us; one cache of 131071 keys
// 497 us.  Four blocks an SM, by bounding the registers, were 10% faster on the 64 caches and 65% slower
// on the one.  Rows of one sequence share nothing here: 16 chats with 64 to 436 new rows take 21 ms, 17 at width 96.
constexpr int kFmaWarps = 8, kFmaSplit = 8;  // warps of a block; blocks of a row, if it is shared out

template <typename T, int H>
__global__ void __launch_bounds__(32 * kFmaWarps) pages_fma_kernel(const PagesAttnParams a, const int splits) {
  constexpr int NT = 32 * kFmaWarps, KV = 8;  // keys whose values are in flight
  __shared__ __align__(16) float q[256][H];   // then the block's sums
  __shared__ float o_part[kFmaWarps][H][256], m_part[kFmaWarps][H], l_part[kFmaWarps][H], m_all[H], l_all[H];
  __shared__ __align__(16) float weight[kFmaWarps][32][H];
  __shared__ long long place[kFmaWarps][32];
  const Params &p = a.p;
  const int per = (p.group + H - 1) / H, kv_head = blockIdx.y / per, h0 = blockIdx.y % per * H;
  const int heads = min(H, p.group - h0), row_at = blockIdx.x / splits, split = blockIdx.x % splits;
  int s = 0;  // the sequence of the row: the last that begins at it or before
  for (int end = p.num_seqs; end - s > 1;) {
    const int mid = (s + end) / 2;
    if (__ldg(p.cu_q + mid) <= row_at) s = mid;
    else end = mid;
  }
  const int q0 = __ldg(p.cu_q + s), q1 = __ldg(p.cu_q + s + 1), len = __ldg(a.kv_lens + s);
  if (q0 < 0 || q0 > q1 || q1 > p.total_q || q1 - q0 > p.max_q || len < 0 ||
      (len > 0 && (len - 1) >> a.log2_page >= a.max_pages)) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_BAD_SEQLENS);
    return;
  }
  const int i = row_at - q0;
  if (i < 0 || i >= q1 - q0) return;
  const long long first = (long long)(q0 + i) * p.h_q + (long long)kv_head * p.group + h0;  // row of the first head
  for (int x = threadIdx.x; x < p.d_qk * H; x += NT) {
    const int c = x % p.d_qk, h = x / p.d_qk;
    const float y = h < heads ? to_f32<T>(static_cast<const T *>(p.q)[(first + h) * p.d_qk + c]) : 0.f;
    q[c][h] = fmaf(y, 0.f, y);  // (an infinity becomes a NaN, and the row with it, as on the tensor cores)
  }
  __syncthreads();
  int lo, hi;
  visible_range(i, len - (q1 - q0), len, p.causal, p.window, lo, hi);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float m[H], l[H], o[H][8];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[h][c] = 0.f;
  }
  for (int j0 = (lo & ~31) + 32 * (split * kFmaWarps + warp); j0 < hi; j0 += 32 * kFmaWarps * splits) {
    // (32 keys lie in one or two pages)
    const int j = j0 + lane;  // (lengths stay 2^16 below the largest int)
    bool see = j >= lo && j < hi;
    int page = see ? __ldg(a.table + (long long)s * a.max_pages + (j >> a.log2_page)) : 0;
    if (page < 0 || page >= a.num_pages) {
      if (see) set_error(p.err, VLF_ERR_BAD_PAGES);
      see = false;
      page = 0;
    }
    const long long slot = (long long)page * p.h_kv + kv_head;
    const long long at = slot * a.page + (j & (a.page - 1));
    float dot[H];
#pragma unroll
    for (int h = 0; h < H; ++h) dot[h] = 0.f;
    float sk = 0.f, sv = 0.f;
    if (see) {
      sk = __ldg(a.k_scale + slot) * p.scale_log2;
      sv = __ldg(a.v_scale + slot);
      const uint8_t *k = a.k_pages + at * p.d_qk;
      int c = 0;
      if (p.d_qk % 16 == 0) {
#pragma unroll 4
        for (; c < p.d_qk; c += 16) {
          const uint4 r = *reinterpret_cast<const uint4 *>(k + c);
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = e4m3_pair(w[e / 2] >> 16 * (e % 2));
#pragma unroll
            for (int h = 0; h < H; ++h) {
              dot[h] = fmaf(q[c + 2 * e][h], f.x, dot[h]);
              dot[h] = fmaf(q[c + 2 * e + 1][h], f.y, dot[h]);
            }
          }
        }
      }
      for (; c < p.d_qk; ++c) {
        const float f = e4m3_pair(k[c]).x;
#pragma unroll
        for (int h = 0; h < H; ++h) dot[h] = fmaf(q[c][h], f, dot[h]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float x = see ? dot[h] * sk : -INFINITY;
      float y = x;
#pragma unroll
      for (int k = 16; k > 0; k /= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, k));
      float top = fmaxf(m[h], y);
      if (top == -INFINITY) top = 0.f;  // (nothing seen yet, or NaN: exp2 of it reaches the sum)
      const float fix = exp2f(m[h] - top), w = see ? exp2f(x - top) : 0.f;
      m[h] = fmaxf(m[h], y);
      l[h] = l[h] * fix + w;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[h][c] *= fix;
      weight[warp][lane][h] = see ? w * sv : 0.f;
    }
    place[warp][lane] = at;
    const uint32_t seen = __ballot_sync(0xffffffffu, see);
    __syncwarp();
    // KV keys' values at a time (a key that is not seen is not read: its slot may hold anything)
#pragma unroll 1
    for (int k0 = 0; k0 < 32; k0 += KV) {
      if (!(seen >> k0 & ((1u << KV) - 1))) continue;
      uint32_t v[KV][2];
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int c = 4 * lane + 128 * b;
          v[k][b] = 0;
          if ((seen >> (k0 + k) & 1u) && c < p.d_v) {
            const uint8_t *x = a.v_pages + place[warp][k0 + k] * p.d_v + c;
            if (p.d_v % 4 == 0) {
              v[k][b] = *reinterpret_cast<const uint32_t *>(x);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (c + e < p.d_v) v[k][b] |= (uint32_t)x[e] << 8 * e;
            }
          }
        }
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        float w[H];
#pragma unroll
        for (int h = 0; h < H; ++h) w[h] = weight[warp][k0 + k][h];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (128 * b >= p.d_v) continue;
          const float2 x = e4m3_pair(v[k][b]), y = e4m3_pair(v[k][b] >> 16);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            o[h][4 * b] = fmaf(w[h], x.x, o[h][4 * b]);
            o[h][4 * b + 1] = fmaf(w[h], x.y, o[h][4 * b + 1]);
            o[h][4 * b + 2] = fmaf(w[h], y.x, o[h][4 * b + 2]);
            o[h][4 * b + 3] = fmaf(w[h], y.y, o[h][4 * b + 3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2) l[h] += __shfl_xor_sync(0xffffffffu, l[h], k);
    if (lane == 0) {
      m_part[warp][h] = m[h];
      l_part[warp][h] = l[h];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) o_part[warp][h][4 * lane + 128 * (c / 4) + c % 4] = o[h][c];
  }
  __syncthreads();
  // the block's maximum, sum and output of each head (q is not needed again)
  float (*const sums)[256] = reinterpret_cast<float (*)[256]>(&q[0][0]);
#pragma unroll 1
  for (int h = 0; h < H; ++h) {
    float top = -INFINITY, sum = 0.f, x = 0.f;
    for (int w = 0; w < kFmaWarps; ++w) top = fmaxf(top, m_part[w][h]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kFmaWarps; ++w) {
      const float f = exp2f(m_part[w][h] - ref);
      sum += l_part[w][h] * f;
      x += o_part[w][h][threadIdx.x] * f;
    }
    sums[h][threadIdx.x] = x;
    if (threadIdx.x == 0) {
      m_all[h] = top;
      l_all[h] = sum;
    }
  }
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  if (splits > 1) cluster.sync();
  else __syncthreads();
  if (split == 0)
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      float top = -INFINITY, sum = 0.f, x = 0.f;
      for (int r = 0; r < splits; ++r) top = fmaxf(top, splits > 1 ? *cluster.map_shared_rank(m_all + h, r) : m_all[h]);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int r = 0; r < splits; ++r) {
        const float f = exp2f((splits > 1 ? *cluster.map_shared_rank(m_all + h, r) : m_all[h]) - ref);
        sum += (splits > 1 ? *cluster.map_shared_rank(l_all + h, r) : l_all[h]) * f;
        x += (splits > 1 ? *cluster.map_shared_rank(&sums[h][threadIdx.x], r) : sums[h][threadIdx.x]) * f;
      }
      const int c = threadIdx.x;
      if (c < p.d_v) static_cast<T *>(p.out)[(first + h) * p.d_v + c] = from_f32<T>(sum == 0.f ? 0.f : x / sum);
      if (c == 0 && p.lse)
        p.lse[((long long)kv_head * p.group + h0 + h) * p.total_q + q0 + i] =
            sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
    }
  if (splits > 1) cluster.sync();  // (the others' shared memory is read above)
}

template <typename T> cudaError_t fma_forward(const PagesAttnParams &a, int num_sms, cudaStream_t st) {
  const Params &p = a.p;
  const int H = p.group == 1 ? 1 : 4;
  const int ys = p.h_kv * ((p.group + H - 1) / H);
  // a row's keys go to eight blocks where the rows alone leave SMs without one
  int splits = (long long)p.total_q * ys < 4ll * num_sms ? kFmaSplit : 1;
  const void *kern = H == 1 ? (const void *)pages_fma_kernel<T, 1> : (const void *)pages_fma_kernel<T, 4>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.total_q * splits, (unsigned)ys);
  cfg.blockDim = dim3(32 * kFmaWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 1 : 0;
  PagesAttnParams copy = a;
  void *args[2] = {&copy, &splits};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
  if (e != cudaSuccess) cudaGetLastError();
  else count_launch();
  return e;
}

// Whether a sequence's rows of a kv head's group are enough for the kernel that has them as rows of its products.  64
// caches of 1000 to 16384 keys, groups of 4 heads of 128: 4 rows (16 with the heads) take 227 us as columns, 446 as
// rows; 8 rows 353 and 458; 9 rows 614 and 460 (two tiles of columns then, each reading the cache); 16 rows 659 and 467.
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
  if (p.dtype == VLF_F32) return fma_forward<float>(a, num_sms, st);
  if (p.dtype == VLF_BF16) return fma_forward<__nv_bfloat16>(a, num_sms, st);
  return fma_forward<__half>(a, num_sms, st);
}

}  // namespace vlf
