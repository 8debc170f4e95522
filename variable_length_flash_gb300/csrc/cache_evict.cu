// Cache eviction by accumulated attention weight: per sequence and kv head, the keys that stay,
// and the cache compacted to them.
//
// Of a sequence of L keys n = min(L, budget) stay.  With L > budget these are the first `sink`,
// the last `recent`, and of the keys between them the budget - sink - recent with the largest
// weight; of equal weights the lower index stays, a NaN counts as the lowest weight.  Kept keys
// keep their order.  Each kv head has a choice of its own, all heads of a sequence the same n.
//
// Two kernels.  The selection finds the budget-th largest weight of a (sequence, kv head) by radix:
// weights as order-preserving 32-bit keys (the protected ones above all), the counts of the leading
// digit among those that still match, the digit in which the n-th falls, on to the next digit; then
// one ordered pass writes the indices that stay.  A cluster of up to eight CTAs shares a long sequence:
// each keeps its share of the keys in shared memory (one read of the weights from HBM) and the
// counts are summed through distributed shared memory.  The gather copies the kept rows of K
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

constexpr int kBins = 1024;
constexpr int kMaxCluster = 8;
constexpr int kKeysHeld = 49152;     // keys a CTA keeps in shared memory (192 KB) at most
constexpr int kBatch = 8;            // keys of a thread in flight
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

// Grid x: sequence * cluster + rank, y: kv head.  Blocks of 256 or 512 threads.  HELD: the CTA's keys
// fit its shared memory (rounded up to whole batches, the rest filled with the lowest key, which no
// count below sees); otherwise each pass reads the weights again.
template <bool HELD>
__global__ void __launch_bounds__(512) evict_select_kernel(const EvictParams p, int cluster) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t key_s[];
  __shared__ __align__(16) int hist[kBins];
  __shared__ int sums[33], found[2], counts[2];
  __shared__ int4 warp_c[2][16], cta_c[2 * kMaxCluster];
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
  if (len <= p.budget) {
    for (int j = t; j < cn; j += nt) index[c0 + j] = c0 + j;
    return;
  }
  const int last = len - p.recent;
  // key j of this CTA's share from the weights (0 behind its end)
  auto make_key = [&](int j) {
    const float x = __ldg(w + min(j, cn - 1));
    const int i = c0 + j;
    return j >= cn ? 0u : i < p.sink || i >= last ? kAlways : order_key(x);
  };
  auto key_at = [&](int j) { return HELD ? key_s[j] : make_key(j); };
  const int padded = cn > 0 ? (cn + kBatch * nt - 1) / (kBatch * nt) * (kBatch * nt) : 0;
  if (HELD) {  // (a thread reads back its own keys until the ordered pass)
    for (int j0 = t; j0 < padded; j0 += kBatch * nt) {
      uint32_t k8[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) k8[x] = make_key(j0 + x * nt);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) key_s[j0 + x * nt] = k8[x];
    }
  }
  uint32_t prefix = 0, mask = 0;  // the leading bits of the n-th largest key, found so far
  int left = n;                   // how many of the keys with these bits stay
  // Twelve bits, two at a time, by counting in registers: sign, exponent and three bits of mantissa
  // leave a few percent of the keys (with histograms in shared memory from the first bit on, the
  // atomics of all keys took 40 of 46 us at 512 lists of 4096-8192).
  for (int step = 0; step < 6; ++step) {
    const int shift = 30 - 2 * step;
    int c[4] = {0, 0, 0, 0};  // (keys with digit 0 need no count)
    for (int j0 = t; j0 < padded; j0 += kBatch * nt) {
      uint32_t k8[kBatch], acc = 0;  // a byte per digit
#pragma unroll
      for (int x = 0; x < kBatch; ++x) k8[x] = key_at(j0 + x * nt);
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
        acc += ((k8[x] ^ prefix) & mask) == 0 ? 1u << (8 * ((k8[x] >> shift) & 3u)) : 0u;
#pragma unroll
      for (int d = 1; d < 4; ++d) c[d] += (acc >> (8 * d)) & 255u;
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) c[d] = __reduce_add_sync(0xffffffffu, c[d]);
    // (two sets of slots in turn: one barrier per step)
    if (lane == 0) warp_c[step & 1][warp] = make_int4(0, c[1], c[2], c[3]);
    __syncthreads();
    int4 x = lane < warps ? warp_c[step & 1][lane] : make_int4(0, 0, 0, 0);
    if (cluster > 1) {
      c[1] = __reduce_add_sync(0xffffffffu, x.y);
      c[2] = __reduce_add_sync(0xffffffffu, x.z);
      c[3] = __reduce_add_sync(0xffffffffu, x.w);
      if (t < cluster) cg::this_cluster().map_shared_rank(cta_c, t)[(step & 1) * kMaxCluster + rank] = make_int4(0, c[1], c[2], c[3]);
      cg::this_cluster().sync();
      x = lane < cluster ? cta_c[(step & 1) * kMaxCluster + lane] : make_int4(0, 0, 0, 0);
    }
    const int c3 = __reduce_add_sync(0xffffffffu, x.w), c2 = __reduce_add_sync(0xffffffffu, x.z),
              c1 = __reduce_add_sync(0xffffffffu, x.y);
    uint32_t d = 3;
    if (c3 < left) {
      left -= c3;
      d = 2;
      if (c2 < left) {
        left -= c2;
        d = 1;
        if (c1 < left) { left -= c1; d = 0; }
      }
    }
    prefix |= d << shift;
    mask |= 3u << shift;
  }
  // The other twenty, ten at a time, by histograms of the keys that are left.
  for (int pass = 0; pass < 2; ++pass) {
    const int shift = pass == 0 ? 10 : 0;
    for (int i = t; i < kBins; i += nt) hist[i] = 0;
    __syncthreads();
    // (the lowest key behind the end falls, if anywhere, into bin 0, whose count ends nothing early)
    for (int j0 = t; j0 < padded; j0 += kBatch * nt) {
      uint32_t k8[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) k8[x] = key_at(j0 + x * nt);
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
        if (((k8[x] ^ prefix) & mask) == 0) atomicAdd(&hist[(k8[x] >> shift) & (kBins - 1)], 1);
    }
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    // the bins from the top, two (512 threads) or four to a thread, summed over the cluster
    const int own = kBins / nt, top = kBins - 1 - t * own;
    int c[4] = {0, 0, 0, 0};  // c[i]: bin top - i
    if (cluster > 1) {  // (512 threads: a wide load per CTA, all in flight)
      int2 x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        x[r] = make_int2(0, 0);
        if (r < cluster) x[r] = *reinterpret_cast<const int2 *>(cg::this_cluster().map_shared_rank(hist, r) + top - 1);
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) { c[0] += x[r].y; c[1] += x[r].x; }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < own) c[i] = hist[top - i];
    }
    const int sum = (c[0] + c[1]) + (c[2] + c[3]);
    int total;
    int above = block_scan(sum, sums, total);
    if (above < left && above + sum >= left) {  // (one thread)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
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
    mask |= (uint32_t)(kBins - 1) << shift;
    left = found[1];
  }
  // Keys above `prefix` stay, and the first `left` of those equal to it.  A warp owns a run of the
  // CTA's keys in order: it counts, the counts are summed up (over the cluster too), it writes.
  const int wper = (cn + warps * 32 - 1) / (warps * 32) * 32;
  const int a = min(cn, warp * wper), b = min(cn, a + wper);
  int gt = 0, eq = 0;
#pragma unroll 8
  for (int j = a + lane; j < b; j += 32) {
    const uint32_t key = key_at(j);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
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
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int j0 = a; j0 < b; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < b ? key_at(j) : 0u;
    const unsigned eqs = __ballot_sync(0xffffffffu, j < b && key == prefix);
    const bool keep = j < b && (key > prefix || (key == prefix && eq_at + __popc(eqs & below) < left));
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (keep) index[at + __popc(kept & below)] = c0 + j;
    at += __popc(kept);
    eq_at += __popc(eqs);
  }
  // no CTA leaves while another may still read its counts
  if (cluster > 1) cg::this_cluster().sync();
}

// Kept rows of K, V and the weights.  Grid y = sequence, x = runs of (output row, head) items, heads
// fastest, so that what a block writes is one stretch.  A group of threads copies an item, a thread
// one B-byte piece of its K or V row; four items of each group are in flight (two and eight were as
// fast, one 25% slower; rows moved by bulk copies through shared memory took 248 us where this takes
// TIME_GATHER, at 64 x 2048 of 4096-8192 keys, 8 heads of 128).
constexpr int kUnroll = 4;
template <int B>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p, int rk, int rv, int rounds) {
  using P = typename Piece<B>::type;
  tc::pdl_trigger();
  tc::pdl_wait();
  const int s = blockIdx.y;
  int k0, len;
  if (!evict_seq(p, s, k0, len)) return;
  const int out0 = p.cu_out[s], n = min(len, p.budget);
  if (out0 < 0 || (long long)out0 + n > p.total_out) return;
  // (rows of more than 256 pieces, widths that are no whole 16-byte pieces: the threads go round)
  const int pieces = rk + rv, groups = max(1, 256 / pieces), g = threadIdx.x / min(pieces, 256);
  if (g >= groups) return;
  const long long items = (long long)n * p.h_kv;
  const int dr = groups / p.h_kv, dh = groups % p.h_kv;  // rows and heads from one item to the next
  for (int c0 = (int)threadIdx.x % min(pieces, 256); c0 < pieces; c0 += 256) {
    const bool is_v = c0 >= rk;
    const int width = is_v ? rv : rk, c = is_v ? c0 - rk : c0;
    const P *from = static_cast<const P *>(is_v ? p.v : p.k) + (size_t)k0 * p.h_kv * width + c;
    P *to = static_cast<P *>(is_v ? p.v_out : p.k_out) + (size_t)out0 * p.h_kv * width + c;
    long long i0 = (long long)blockIdx.x * groups * kUnroll * rounds + g;
    int r = (int)(i0 / p.h_kv), h = (int)(i0 % p.h_kv);
    for (int round = 0; round < rounds && i0 < items; ++round, i0 += groups * kUnroll) {
      P x[kUnroll];
      int src[kUnroll], hh[kUnroll], rr[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        // (a plain load: the selection wrote the indices while this kernel may already have been here)
        rr[u] = r;
        hh[u] = h;
        src[u] = r < n ? p.index[(size_t)h * p.total_out + out0 + r] : -1;
        r += dr;
        h += dh;
        if (h >= p.h_kv) { h -= p.h_kv; ++r; }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if ((unsigned)src[u] < (unsigned)len) x[u] = __ldg(from + ((size_t)src[u] * p.h_kv + hh[u]) * width);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if ((unsigned)src[u] < (unsigned)len) {
          to[((size_t)rr[u] * p.h_kv + hh[u]) * width] = x[u];
          if (c0 == 0)
            p.weights_out[(size_t)hh[u] * p.total_out + out0 + rr[u]] =
                __ldg(p.weights + (size_t)hh[u] * p.total_kv + k0 + src[u]);
        }
    }
  }
}

}  // namespace

cudaError_t cache_evict(const EvictParams &p, cudaStream_t st) {
  // CTAs per (sequence, kv head): one per 8192 keys of the longest sequence, eight at most; 512
  // threads each, 256 where their share is small
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)cluster * 8192 < p.max_kv) cluster *= 2;
  const int share = (p.max_kv + cluster - 1) / cluster;
  const int threads = share > 1024 ? 512 : 256, batch = kBatch * threads;
  const bool held = share <= kKeysHeld;
  const int smem = held ? (share + batch - 1) / batch * batch * 4 : 0;
  const void *sel = held ? reinterpret_cast<const void *>(evict_select_kernel<true>)
                         : reinterpret_cast<const void *>(evict_select_kernel<false>);
  cudaError_t e = set_smem_once(sel, smem);
  if (e != cudaSuccess) return e;
  EvictParams a = p;
  void *args[2] = {&a, &cluster};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_seqs * cluster, p.h_kv);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
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
  // rounds of a block: as many, up to eight, as leave eight blocks per SM
  const long long run = std::max(1, 256 / (rk + rv)) * kUnroll, runs = (most * p.h_kv + run - 1) / run;
  int rounds = (int)std::max(1ll, std::min(8ll, runs * p.num_seqs / (152 * 8)));
  const long long x = (runs + rounds - 1) / rounds;
  if (x > 0x7fffffffll) return cudaErrorInvalidValue;
  const void *gather = b == 16 ? reinterpret_cast<const void *>(evict_gather_kernel<16>)
                     : b == 4 ? reinterpret_cast<const void *>(evict_gather_kernel<4>)
                              : reinterpret_cast<const void *>(evict_gather_kernel<2>);
  void *gargs[4] = {&a, &rk, &rv, &rounds};
  e = launch_dependent(gather, dim3((unsigned)x, p.num_seqs), 256, 0, st, gargs);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace vlf
