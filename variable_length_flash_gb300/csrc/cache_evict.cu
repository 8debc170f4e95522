// Cache eviction by accumulated attention weight: per sequence and kv head, the keys that stay,
// and the cache compacted to them.
//
// Of a sequence of L keys n = min(L, budget) stay.  With L > budget these are the first `sink`,
// the last `recent`, and of the keys between them the budget - sink - recent with the largest
// weight; of equal weights the lower index stays, a NaN counts as the lowest weight.  Kept keys
// keep their order.  Each kv head has a choice of its own, all heads of a sequence the same n.
//
// Two kernels.  The selection (a CTA per sequence and kv head) finds the m-th largest weight by
// radix: weights as order-preserving 32-bit keys, a histogram of the leading digit of those that
// still match, the digit in which the m-th falls, and on to the next digit; then one ordered pass
// writes the indices that stay.  The gather copies the kept rows of K and V and is the bulk of the
// work: bound by HBM, every kept row read once and written once.
#include "common.cuh"
#include "kernels.h"

namespace vlf {
namespace {

template <int B> struct Piece;
template <> struct Piece<16> { using type = uint4; };
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<2> { using type = uint16_t; };

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;  // 11-bit digits: 11 + 11 + 10 bits

// fp32 -> unsigned with the same order; -0 and +0 are equal, NaN is below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sum of x over the block, to every thread (red: 33 ints of shared memory).
__device__ __forceinline__ long long block_sum(long long x, long long *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  long long s = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) s += red[w];
  return s;
}

// Exclusive prefix sum of x over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane], winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    warp_sums[lane] = winc - w;
    if (lane == 31) *total = winc;
  }
  __syncthreads();
  return warp_sums[warp] + inc - x;
}

// The sequence's first key and length; false where cu_seqlens are bad.
__device__ __forceinline__ bool evict_seq(const EvictParams &p, int s, int &k0, int &len) {
  const int a = __ldg(p.cu_kv + s), b = __ldg(p.cu_kv + s + 1);
  k0 = a;
  len = b - a;
  return a >= 0 && b >= a && b <= p.total_kv && len <= p.max_kv && (s > 0 || a == 0) &&
         (s < p.num_seqs - 1 || b == p.total_kv);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[kBins];
  __shared__ long long red[kSelThreads / 32];
  __shared__ int warp_sums[32], bcast[3];
  const int s = blockIdx.x, h = blockIdx.y, t = threadIdx.x;
  int k0, len;
  // a sequence that cannot be kept leaves -1, and the gather skips it and the one behind it
  auto refuse = [&]() {
    if (t != 0) return;
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
    if (h == 0) p.cu_out[s + 1] = -1;
  };
  if (s == 0 && h == 0 && t == 0) p.cu_out[0] = 0;
  if (!evict_seq(p, s, k0, len)) {
    refuse();
    return;
  }
  const int n = min(len, p.budget);
  // first output row: what the sequences before this one keep
  long long before = 0;
  for (int i = t; i < s; i += kSelThreads)
    before += min(max(__ldg(p.cu_kv + i + 1) - __ldg(p.cu_kv + i), 0), p.budget);
  before = block_sum(before, red);
  if (before + n > p.total_out) {
    refuse();
    return;
  }
  const int out0 = (int)before;
  if (h == 0 && t == 0) p.cu_out[s + 1] = out0 + n;
  const float *w = p.weights + (size_t)h * p.total_kv + k0;
  int *index = p.index + (size_t)h * p.total_out + out0;
  float *w_out = p.weights_out + (size_t)h * p.total_out + out0;
  if (len <= p.budget) {
    for (int j = t; j < len; j += kSelThreads) {
      index[j] = j;
      w_out[j] = w[j];
    }
    return;
  }
  // the keys between the protected ones: [lo, hi), of which m stay
  const int lo = p.sink, hi = len - p.recent, m = p.budget - p.sink - p.recent;
  uint32_t thr = 0xffffffffu;  // the m-th largest order key
  int ties = 0;                // how many equal to it stay (the first ones)
  if (m > 0) {
    uint32_t prefix = 0, mask = 0;
    int left = m;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = t; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + t; j < hi; j += kSelThreads) {
        const uint32_t key = order_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // from the top: thread t takes bins - 1 - 2t and the one below it
      const int b0 = bins - 1 - 2 * t;
      const int c0 = b0 >= 0 ? hist[b0] : 0, c1 = b0 >= 1 ? hist[b0 - 1] : 0;
      const int above = block_scan(c0 + c1, warp_sums, &bcast[2]);
      if (above < left && above + c0 + c1 >= left) {
        const bool first = above + c0 >= left;
        bcast[0] = first ? b0 : b0 - 1;
        bcast[1] = left - above - (first ? 0 : c0);
      }
      __syncthreads();
      prefix |= (uint32_t)bcast[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      left = bcast[1];
      __syncthreads();
    }
    thr = prefix;
    ties = left;
  }
  // ordered pass: 1024 keys at a time; equal ones stay while ties are left
  int done = 0, tied = 0;
  for (int j0 = 0; j0 < len; j0 += kSelThreads) {
    const int j = j0 + t;
    bool keep = false, eq = false;
    float x = 0.f;
    if (j < len) {
      x = w[j];
      if (j < lo || j >= hi) keep = true;
      else if (m > 0) {
        const uint32_t key = order_key(x);
        keep = key > thr;
        eq = key == thr;
      }
    }
    const int te = block_scan(eq ? 1 : 0, warp_sums, &bcast[2]);
    const int all_eq = bcast[2];
    if (eq && tied + te < ties) keep = true;
    __syncthreads();
    const int at = done + block_scan(keep ? 1 : 0, warp_sums, &bcast[2]);
    if (keep) {
      index[at] = j;
      w_out[at] = x;
    }
    done += bcast[2];
    tied += all_eq;
    __syncthreads();
  }
}

// Kept rows of K and V: grid y = sequence, x = runs of 16-byte pieces (or single elements where
// rows are not whole 16-byte pieces).  Row r of the output, head h: source row index[h][r].
template <int B>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p, int es) {
  using P = typename Piece<B>::type;
  const int s = blockIdx.y;
  int k0, len;
  if (!evict_seq(p, s, k0, len)) return;
  const int out0 = p.cu_out[s];
  const int n = min(len, p.budget);
  if (out0 < 0 || (long long)out0 + n > p.total_out) return;
  const int rk = p.d_qk * es / B, rv = p.d_v * es / B;  // pieces per row
  const long long per = (long long)p.h_kv * (rk + rv);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < per * n; i += (long long)gridDim.x * 256) {
    const int r = (int)(i / per);
    int c = (int)(i % per);
    const bool is_v = c >= p.h_kv * rk;
    if (is_v) c -= p.h_kv * rk;
    const int w = is_v ? rv : rk, h = c / w;
    const int src = p.index[(size_t)h * p.total_out + out0 + r];
    if (src < 0 || src >= len) continue;
    const size_t row = (size_t)p.h_kv * w;
    const P *from = static_cast<const P *>(is_v ? p.v : p.k) + (size_t)(k0 + src) * row + c;
    P *to = static_cast<P *>(is_v ? p.v_out : p.k_out) + (size_t)(out0 + r) * row + c;
    *to = *from;
  }
}

}  // namespace

cudaError_t cache_evict(const EvictParams &p, cudaStream_t st) {
  evict_select_kernel<<<dim3(p.num_seqs, p.h_kv), kSelThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  const int es = p.dtype == VLF_F32 ? 4 : 2;
  const long long most = p.max_kv < p.budget ? p.max_kv : p.budget;
  if (most == 0) return cudaSuccess;
  const bool whole = p.d_qk * es % 16 == 0 && p.d_v * es % 16 == 0;
  const int b = whole ? 16 : es;
  const long long pieces = most * p.h_kv * (p.d_qk + p.d_v) * es / b;
  const long long x = (pieces + 1023) / 1024;  // four pieces a thread
  const dim3 grid((unsigned)(x < 0x7fffffffll ? x : 0x7fffffffll), p.num_seqs);
  if (b == 16) evict_gather_kernel<16><<<grid, 256, 0, st>>>(p, es);
  else if (b == 4) evict_gather_kernel<4><<<grid, 256, 0, st>>>(p, es);
  else evict_gather_kernel<2><<<grid, 256, 0, st>>>(p, es);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace vlf
