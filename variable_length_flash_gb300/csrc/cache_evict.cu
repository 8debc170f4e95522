// Cache eviction by accumulated attention weight: per sequence and kv head, the keys that stay,
// and the cache compacted to them.
//
// Of a sequence of L keys n = min(L, budget) stay.  With L > budget these are the first `sink`,
// the last `recent`, and of the keys between them the budget - sink - recent with the largest
// weight; of equal weights the lower index stays, a NaN counts as the lowest weight.  Kept keys
// keep their order.  Each kv head has a choice of its own, all heads of a sequence the same n.
//
// Two kernels.  The selection finds the budget-th largest weight of a (sequence, kv head) by radix:
// weights as order-preserving 32-bit keys (the protected ones above all), a histogram of the leading
// digit of those that still match, the digit in which the n-th falls, on to the next digit; then one
// ordered pass writes the indices that stay.  A cluster of up to eight CTAs shares a long sequence:
// each keeps its share of the keys in shared memory (one read of the weights from HBM) and the
// histograms are summed through distributed shared memory.  The gather copies the kept rows of K
// and V and is the bulk of the work: bound by HBM, every kept row read once and written once.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace {

template <int B> struct Piece;
template <> struct Piece<16> { using type = uint4; };
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<2> { using type = uint16_t; };

constexpr int kBins = 2048;          // 11-bit digits: 11 + 11 + 10 bits
constexpr int kMaxCluster = 8;
constexpr int kKeysHeld = 49152;     // keys a CTA keeps in shared memory (192 KB); more are read again
constexpr uint32_t kAlways = 0xffffffffu;  // the key of a protected one (+inf's is 0xff800000)

// fp32 -> unsigned with the same order; -0 and +0 are equal, NaN is below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The sequence's first key and length; false where cu_seqlens are bad.
__device__ __forceinline__ bool evict_seq(const EvictParams &p, int s, int &k0, int &len) {
  const int a = __ldg(p.cu_kv + s), b = __ldg(p.cu_kv + s + 1);
  k0 = a;
  len = b - a;
  return a >= 0 && b >= a && b <= p.total_kv && len <= p.max_kv && (s > 0 || a == 0) &&
         (s < p.num_seqs - 1 || b == p.total_kv);
}

// Exclusive prefix sum of x over the block's threads, and its total (sums: 33 ints).
__device__ __forceinline__ int block_scan(int x, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // (sums may still be read from the call before)
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int mine = lane < warps ? sums[lane] : 0, winc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += y;
  }
  total = __shfl_sync(0xffffffffu, winc, 31);
  return __shfl_sync(0xffffffffu, winc - mine, warp) + inc - x;
}

// Grid x: sequence * cluster + rank, y: kv head.  Blocks of 256 or 512 threads.
__global__ void __launch_bounds__(512) evict_select_kernel(const EvictParams p, int cluster, int held) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t key_s[];  // [held]
  __shared__ int hist[kBins];
  __shared__ int sums[33], found[2], counts[2];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster, h = blockIdx.y, t = threadIdx.x, nt = blockDim.x;
  const int lane = t & 31, warp = t >> 5, warps = nt >> 5;
  const bool first = rank == 0 && h == 0 && t == 0;
  // a sequence that cannot be kept leaves -1, and the gather skips it and the one behind it
  auto refuse = [&]() {
    if (rank != 0 || t != 0) return;
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
    if (h == 0) p.cu_out[s + 1] = -1;
  };
  if (s == 0 && first) p.cu_out[0] = 0;
  int k0, len;
  if (!evict_seq(p, s, k0, len)) {  // (the same for the whole cluster)
    refuse();
    return;
  }
  const int n = min(len, p.budget);
  // first output row: what the sequences before this one keep (at most total_kv, an int)
  int before = 0, out0;
  for (int i = t; i < s; i += nt) before += min(max(__ldg(p.cu_kv + i + 1) - __ldg(p.cu_kv + i), 0), p.budget);
  block_scan(before, sums, out0);
  if ((long long)out0 + n > p.total_out || out0 < 0) {
    refuse();
    return;
  }
  if (first) p.cu_out[s + 1] = out0 + n;
  if (n == 0) return;
  // this CTA's keys: [c0, c0 + cn)
  const int per = (len + cluster - 1) / cluster, c0 = min(len, rank * per), cn = min(per, len - c0);
  const float *w = p.weights + (size_t)h * p.total_kv + k0 + c0;
  int *index = p.index + (size_t)h * p.total_out + out0;
  float *w_out = p.weights_out + (size_t)h * p.total_out + out0;
  if (len <= p.budget) {
    for (int j = t; j < cn; j += nt) {
      index[c0 + j] = c0 + j;
      w_out[c0 + j] = w[j];
    }
    return;
  }
  const int last = len - p.recent;
  auto make_key = [&](int j) {
    const int i = c0 + j;
    return i < p.sink || i >= last ? kAlways : order_key(__ldg(w + j));
  };
  auto key_at = [&](int j) { return j < held ? key_s[j] : make_key(j); };
  // Counts the digits of the keys that match the prefix found so far.  Where many lanes of a warp
  // meet in one bin (weights of exactly nothing, protected keys) the first lane's bin is added once.
  auto count = [&](uint32_t key, bool in, int shift, int bins) {
    const unsigned act = __ballot_sync(0xffffffffu, in);
    if (!act) return;
    const int bin = (key >> shift) & (bins - 1);
    const int lead = __ffs(act) - 1, lead_bin = __shfl_sync(0xffffffffu, bin, lead);
    const unsigned same = __ballot_sync(0xffffffffu, in && bin == lead_bin);
    if (lane == lead) atomicAdd(&hist[bin], __popc(same));
    else if (in && bin != lead_bin) atomicAdd(&hist[bin], 1);
  };
  uint32_t prefix = 0, mask = 0;
  int left = n;  // how many of the matching keys stay
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int i = t; i < kBins; i += nt) hist[i] = 0;
    __syncthreads();
    const int rounds = (cn + nt - 1) / nt;
#pragma unroll 4
    for (int x = 0; x < rounds; ++x) {
      const int j = x * nt + t;
      uint32_t key = 0;
      if (j < cn) {
        if (pass == 0) {
          key = make_key(j);
          if (j < held) key_s[j] = key;
        } else {
          key = key_at(j);
        }
      }
      count(key, j < cn && (key & mask) == prefix, shift, bins);
    }
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    // bins from the top, kBins / nt to a thread, summed over the cluster
    const int own = bins / nt, top = bins - 1 - t * own;  // (own: 2, 4 or 8)
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 0;
      if (i >= own) continue;
      if (cluster > 1) {
        for (int r = 0; r < cluster; ++r) c[i] += cg::this_cluster().map_shared_rank(hist, r)[top - i];
      } else {
        c[i] = hist[top - i];
      }
      sum += c[i];
    }
    int total;
    int above = block_scan(sum, sums, total);
    if (above < left && above + sum >= left) {  // (one thread)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < own && above < left && above + c[i] >= left) {
          found[0] = top - i;
          found[1] = left - above;
        }
        above += c[i];
      }
    }
    // every CTA has read the histograms before any of them starts the next one
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    left = found[1];
  }
  // Keys above `prefix` stay, and the first `left` of those equal to it.  A warp owns a run of the
  // CTA's keys in order: it counts, the counts are summed up (over the cluster too), it writes.
  const int wper = (cn + warps * 32 - 1) / (warps * 32) * 32;
  const int a = min(cn, warp * wper), b = min(cn, a + wper);
  int gt = 0, eq = 0;
  for (int j0 = a; j0 < b; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < b ? key_at(j) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, j < b && key > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, j < b && key == prefix));
  }
  int all_eq, all_gt;
  int eq_at = block_scan(lane == 0 ? eq : 0, sums, all_eq);  // (lane 0's is its warp's)
  eq_at = __shfl_sync(0xffffffffu, eq_at, 0);
  int gt_at = block_scan(lane == 0 ? gt : 0, sums, all_gt);
  gt_at = __shfl_sync(0xffffffffu, gt_at, 0);
  if (cluster > 1) {
    if (t == 0) { counts[0] = all_eq; counts[1] = all_gt; }
    cg::this_cluster().sync();
    for (int r = 0; r < rank; ++r) {
      const int *c = cg::this_cluster().map_shared_rank(counts, r);
      eq_at += c[0];
      gt_at += c[1];
    }
  }
  int at = gt_at + min(eq_at, left);  // this warp's first output
  for (int j0 = a; j0 < b; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < b ? key_at(j) : 0u;
    const unsigned below = (1u << lane) - 1u;
    const unsigned eqs = __ballot_sync(0xffffffffu, j < b && key == prefix);
    const bool keep = j < b && (key > prefix || (key == prefix && eq_at + __popc(eqs & below) < left));
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      index[at + __popc(kept & below)] = c0 + j;
      w_out[at + __popc(kept & below)] = __ldg(w + j);
    }
    at += __popc(kept);
    eq_at += __popc(eqs);
  }
  // no CTA leaves while another may still read its counts
  if (cluster > 1) cg::this_cluster().sync();
}

// Kept rows of K and V.  Grid y = sequence, x = runs of (output row, head) items, heads fastest, so
// that a run's writes are one stretch.  A group of threads copies an item, a thread one B-byte piece
// of its K or V row (or every 256th, where a row has more); kUnroll items' loads are in flight.
constexpr int kUnroll = 8;
template <int B>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p, int rk, int rv) {
  using P = typename Piece<B>::type;
  tc::pdl_trigger();
  tc::pdl_wait();
  const int s = blockIdx.y;
  int k0, len;
  if (!evict_seq(p, s, k0, len)) return;
  const int out0 = p.cu_out[s], n = min(len, p.budget);
  if (out0 < 0 || (long long)out0 + n > p.total_out) return;
  const int pieces = rk + rv, groups = max(1, 256 / pieces), g = threadIdx.x / pieces;
  if (g >= groups) return;
  const long long items = (long long)n * p.h_kv;
  const long long i0 = (long long)blockIdx.x * groups * kUnroll + g;
  if (i0 >= items) return;
  const int r0 = (int)(i0 / p.h_kv), h0 = (int)(i0 % p.h_kv);  // output row and head of the first item
  const int dr = groups / p.h_kv, dh = groups % p.h_kv;        // and from one to the next
  for (int c0 = pieces > 256 ? (int)threadIdx.x : (int)threadIdx.x % pieces; c0 < pieces; c0 += 256) {
    const bool is_v = c0 >= rk;
    const int width = is_v ? rv : rk, c = is_v ? c0 - rk : c0;
    const P *from = static_cast<const P *>(is_v ? p.v : p.k);
    P *to = static_cast<P *>(is_v ? p.v_out : p.k_out) + ((size_t)out0 * p.h_kv + i0) * width + c;
    P x[kUnroll];
    int src[kUnroll];
    int r = r0, h = h0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      // (a plain load: the selection wrote the indices while this kernel may already have been here)
      src[u] = r < n ? p.index[(size_t)h * p.total_out + out0 + r] : -1;
      r += dr;
      h += dh;
      if (h >= p.h_kv) { h -= p.h_kv; ++r; }
    }
    h = h0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (src[u] >= 0 && src[u] < len) x[u] = __ldg(from + ((size_t)(k0 + src[u]) * p.h_kv + h) * width + c);
      h += dh;
      if (h >= p.h_kv) h -= p.h_kv;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (src[u] >= 0 && src[u] < len) to[(size_t)u * groups * width] = x[u];
  }
}

}  // namespace

cudaError_t cache_evict(const EvictParams &p, cudaStream_t st) {
  // CTAs per (sequence, kv head): one per 8192 keys of the longest sequence, eight at most; 512
  // threads each, 256 where their share is small
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)cluster * 8192 < p.max_kv) cluster *= 2;
  const int share = (p.max_kv + cluster - 1) / cluster;
  int threads = share > 1024 ? 512 : 256, held = std::min(share, kKeysHeld);
  const void *sel = reinterpret_cast<const void *>(evict_select_kernel);
  cudaError_t e = set_smem_once(sel, held * 4);
  if (e != cudaSuccess) return e;
  EvictParams a = p;
  void *args[3] = {&a, &cluster, &held};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_seqs * cluster, p.h_kv);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)held * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  e = cudaLaunchKernelExC(&cfg, sel, args);
  if (e != cudaSuccess) return e;
  count_launch();
  const int es = p.dtype == VLF_F32 ? 4 : 2;
  const long long most = std::min(p.max_kv, p.budget);
  if (most == 0 || p.total_out == 0) return cudaSuccess;
  const bool whole = p.d_qk * es % 16 == 0 && p.d_v * es % 16 == 0;
  const int b = whole ? 16 : es;
  int rk = p.d_qk * es / b, rv = p.d_v * es / b;
  const long long run = std::max(1, 256 / (rk + rv)) * kUnroll, x = (most * p.h_kv + run - 1) / run;
  if (x > 0x7fffffffll) return cudaErrorInvalidValue;
  const void *gather = b == 16 ? reinterpret_cast<const void *>(evict_gather_kernel<16>)
                     : b == 4 ? reinterpret_cast<const void *>(evict_gather_kernel<4>)
                              : reinterpret_cast<const void *>(evict_gather_kernel<2>);
  void *gargs[3] = {&a, &rk, &rv};
  e = launch_dependent(gather, dim3((unsigned)x, p.num_seqs), 256, 0, st, gargs);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace vlf
