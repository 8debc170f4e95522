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
// each keeps its share of the keys on chip (one read of the weights from HBM): in registers up to 8 keys
// per thread, beyond that some of them in local memory (64 registers a thread; 36 and 56 bytes of
// spills at 16 keys, 172 and 220 at 32).  The counts are summed through distributed shared memory.  The gather copies the kept rows of K
// and V and is the bulk of the work: bound by HBM, every kept row read once and written once.
// Measured: 64 x 4096-8192 keys of 8 heads of 128 in bf16 cut to 2048, 206 us (gather 175, selection
// 30: the latency of its 6 + 2 counting steps, a read of 12 MB); one list of 131071 keys cut to
// 16384, 55 us (25 of them the selection's cluster barriers, two per counting step; the gather's 30
// are a start, three rounds of loads and an end); 8 x 100-436 keys in one launch, 7 us.
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

// Exclusive prefix sum of x over the block's warps (x: the same in all lanes of a warp), and its total.
__device__ __forceinline__ int warp_scan(int x, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  __syncthreads();  // (sums may still be read from the call before)
  if (lane == 0) sums[warp] = x;
  __syncthreads();
  const int mine = lane < warps ? sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, mine);
  return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
}

// Grid x: sequence * cluster + rank, y: kv head.  A warp owns a run of 32 * K keys in order, lane l
// the keys l, 32 + l, ... of it, in registers (K = 0: more keys than that, read again on each pass).
// What is behind the end counts as the lowest key, which no count below sees.
// COPY: the CTA then copies its rows itself (small problems: one launch).
template <int K, int THREADS, bool COPY>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const EvictParams p, int cluster) {
  namespace cg = cooperative_groups;
  __shared__ __align__(16) int hist[kBins];
  __shared__ int sums[32], found[2], counts[2];
  __shared__ int4 warp_c[2][32], cta_c[2 * kMaxCluster];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster, h = blockIdx.y, t = threadIdx.x;
  constexpr int nt = THREADS, warps = THREADS / 32;
  const int lane = t & 31, warp = t >> 5;
  const bool first = rank == 0 && h == 0 && t == 0;
  // a sequence that cannot be kept leaves -1, and the gather skips it and the one behind it
  auto refuse = [&]() {
    if (rank != 0 || t != 0) return;
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
    if (h == 0) p.cu_out[s + 1] = -1;
  };
  if (s == 0 && first) p.cu_out[0] = 0;
  int k0, len;
  const int prev = COPY ? __ldg(p.cu_kv + max(s - 1, 0)) : 0;
  if (!evict_seq(p, s, k0, len)) {  // (the same for the whole cluster)
    refuse();
    return;
  }
  // Behind a refused sequence no rows are copied, as in the gather.  (One that is refused because it does
  // not fit needs no look: those behind it do not fit either.  A branch around the copy instead of a
  // count of 0 cost 0.4 us of 6.6.)
  const bool behind = COPY && (prev < 0 || prev > k0 || k0 - prev > p.max_kv || (s <= 1 && prev != 0));
  const int n = min(len, p.budget), last = len - p.recent;
  const bool all = len <= p.budget;
  // this CTA's keys [c0, c0 + cn), this warp's [wa, wa + 32 * ke) of them
  const int per = (len + cluster - 1) / cluster, c0 = min(len, rank * per), cn = min(per, len - c0);
  const int ke = K > 0 ? K : (cn + nt - 1) / nt, wa = warp * 32 * ke + lane;
  const float *w = p.weights + (size_t)h * p.total_kv + k0 + c0;
  auto raw = [&](int e) { return __ldg(w + min(wa + 32 * e, cn - 1)); };
  auto make_key = [&](int e, float x) {
    const int j = wa + 32 * e, i = c0 + j;
    return j >= cn ? 0u : i < p.sink || i >= last ? kAlways : order_key(x);
  };
  uint32_t key[K > 0 ? K : 1];
#pragma unroll
  for (int e = 0; e < (K > 0 ? K : 1); ++e) key[e] = 0u;
  if (K > 0 && !all && cn > 0) {
    // (all loads are sent before the first is used)
#pragma unroll
    for (int e = 0; e < K; ++e) key[e] = __float_as_uint(raw(e));
  }
  auto visit = [&](auto &&f) {  // f(key, e) for this lane's keys, in their order
    if constexpr (K > 0) {
#pragma unroll
      for (int e = 0; e < K; ++e) f(key[e], e);
    } else {
#pragma unroll 4
      for (int e = 0; e < ke; ++e) f(make_key(e, raw(e)), e);
    }
  };
  // first output row: what the sequences before this one keep (at most total_kv, an int)
  int before = 0, out0;
  for (int i = t; i < s; i += nt) before += min(max(__ldg(p.cu_kv + i + 1) - __ldg(p.cu_kv + i), 0), p.budget);
  warp_scan(__reduce_add_sync(0xffffffffu, before), sums, out0);
  if ((long long)out0 + n > p.total_out || out0 < 0) {
    refuse();
    return;
  }
  if (first) p.cu_out[s + 1] = out0 + n;
  if (n == 0) return;
  int *index = p.index + (size_t)h * p.total_out + out0;
  // this (sequence, head)'s rows, a 16-byte piece of K or V per thread and turn, four in flight
  auto copy_rows = [&]() {
    __syncthreads();  // (the block's own writes of index)
    const int es = p.dtype == VLF_F32 ? 4 : 2, rk = p.d_qk * es / 16, rv = p.d_v * es / 16, pieces = rk + rv;
    const int rows = behind ? 0 : n;
    for (int r = t; r < rows; r += nt)
      p.weights_out[(size_t)h * p.total_out + out0 + r] = __ldg(p.weights + (size_t)h * p.total_kv + k0 + index[r]);
    const int all_pieces = rows * pieces;
    for (int i0 = t; i0 < all_pieces; i0 += 4 * nt) {
      uint4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * nt, r = i / pieces, c = i % pieces;
        if (i >= all_pieces) continue;
        const size_t row = (size_t)(k0 + index[r]) * p.h_kv + h;
        x[u] = c < rk ? __ldg(static_cast<const uint4 *>(p.k) + row * rk + c)
                      : __ldg(static_cast<const uint4 *>(p.v) + row * rv + c - rk);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * nt, r = i / pieces, c = i % pieces;
        if (i >= all_pieces) continue;
        const size_t row = (size_t)(out0 + r) * p.h_kv + h;
        if (c < rk) static_cast<uint4 *>(p.k_out)[row * rk + c] = x[u];
        else static_cast<uint4 *>(p.v_out)[row * rv + c - rk] = x[u];
      }
    }
  };
  if (all) {
    for (int j = t; j < cn; j += nt) index[c0 + j] = c0 + j;
    if constexpr (COPY) copy_rows();
    return;
  }
  // (no CTA writes another's shared memory before that one has started: awaited at the first write)
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if constexpr (K > 0) {
#pragma unroll
    for (int e = 0; e < K; ++e) key[e] = make_key(e, __uint_as_float(key[e]));
  }
  // Twelve bits of the n-th largest key, two at a time, by counting the keys that reach each of three
  // thresholds: sign, exponent and three bits of mantissa leave a few percent of the keys.  (With
  // histograms from the first bit on, the shared-memory atomics of all keys took most of the time.)
  uint32_t prefix = 0;
  int above = 0;  // keys above every one with these bits
  for (int shift = 30; shift >= 20; shift -= 2) {
    const uint32_t t1 = prefix | 1u << shift, t2 = prefix | 2u << shift, t3 = prefix | 3u << shift;
    int a1 = 0, a2 = 0, a3 = 0;
    visit([&](uint32_t k, int) {
      a1 += k >= t1;
      a2 += k >= t2;
      a3 += k >= t3;
    });
    a1 = __reduce_add_sync(0xffffffffu, a1);
    a2 = __reduce_add_sync(0xffffffffu, a2);
    a3 = __reduce_add_sync(0xffffffffu, a3);
    const int turn = (shift >> 1) & 1;  // (two sets of slots in turn: one barrier per step)
    if (lane == 0) warp_c[turn][warp] = make_int4(a1, a2, a3, 0);
    __syncthreads();
    int4 x = lane < warps ? warp_c[turn][lane] : make_int4(0, 0, 0, 0);
    a1 = __reduce_add_sync(0xffffffffu, x.x);
    a2 = __reduce_add_sync(0xffffffffu, x.y);
    a3 = __reduce_add_sync(0xffffffffu, x.z);
    if (cluster > 1) {
      if (shift == 30) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (t < cluster) cg::this_cluster().map_shared_rank(cta_c, t)[turn * kMaxCluster + rank] = make_int4(a1, a2, a3, 0);
      cg::this_cluster().sync();
      x = lane < cluster ? cta_c[turn * kMaxCluster + lane] : make_int4(0, 0, 0, 0);
      a1 = __reduce_add_sync(0xffffffffu, x.x);
      a2 = __reduce_add_sync(0xffffffffu, x.y);
      a3 = __reduce_add_sync(0xffffffffu, x.z);
    }
    if (a3 >= n) {
      prefix = t3;
    } else if (a2 >= n) {
      prefix = t2;
      above = a3;
    } else if (a1 >= n) {
      prefix = t1;
      above = a2;
    } else {
      above = a1;
    }
  }
  // The other twenty, ten at a time, by histograms of the keys that are left.
  int left = n - above;  // how many of the keys with these bits stay
  for (int shift = 10; shift >= 0; shift -= 10) {
    const uint32_t mask = 0xffffffffu << (shift + 10);
    for (int i = t; i < kBins; i += nt) hist[i] = 0;
    __syncthreads();
    // (the lowest key behind the end falls, if anywhere, into bin 0, whose count ends nothing early)
    visit([&](uint32_t k, int) {
      if (((k ^ prefix) & mask) == 0) atomicAdd(&hist[(k >> shift) & (kBins - 1)], 1);
    });
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    // the bins from the top, four to each of the first 256 threads, summed over the cluster
    const int top = kBins - 1 - 4 * t;
    int4 c = make_int4(0, 0, 0, 0);
    if (t < kBins / 4) {
      if (cluster > 1) {  // (a wide load per CTA, all in flight)
        int4 x[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          x[r] = make_int4(0, 0, 0, 0);
          if (r < cluster) x[r] = *reinterpret_cast<const int4 *>(cg::this_cluster().map_shared_rank(hist, r) + top - 3);
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) { c.x += x[r].x; c.y += x[r].y; c.z += x[r].z; c.w += x[r].w; }
      } else {
        c = *reinterpret_cast<const int4 *>(hist + top - 3);
      }
    }
    const int sum = (c.x + c.y) + (c.z + c.w);
    int inc = sum, total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    int over = warp_scan(__shfl_sync(0xffffffffu, inc, 31), sums, total) + inc - sum;
    if (over < left && over + sum >= left) {  // (one thread)
      const int bins[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (over < left && over + bins[i] >= left) {
          found[0] = top - i;
          found[1] = left - over;
        }
        over += bins[i];
      }
    }
    // every CTA has read the histograms before any of them starts the next one
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    left = found[1];
  }
  // Keys above `prefix` stay, and the first `left` of those equal to it: the warps count, the counts
  // are summed up (over the cluster too), each warp writes its run.
  int gt = 0, eq = 0, all_eq, all_gt;
  visit([&](uint32_t k, int e) {
    gt += k > prefix;
    eq += k == prefix && wa + 32 * e < cn;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  int eq_at = warp_scan(eq, sums, all_eq), gt_at = warp_scan(gt, sums, all_gt);
  if (cluster > 1) {
    if (t == 0) { counts[0] = all_eq; counts[1] = all_gt; }
    cg::this_cluster().sync();
    // (lane r reads rank r's, of the ranks before this one)
    const int *c = cg::this_cluster().map_shared_rank(counts, min(lane, cluster - 1));
    eq_at += __reduce_add_sync(0xffffffffu, lane < rank ? c[0] : 0);
    gt_at += __reduce_add_sync(0xffffffffu, lane < rank ? c[1] : 0);
  }
  int at = gt_at + min(eq_at, left);  // this warp's first output
  if (gt + eq > 0) {
    const unsigned below = (1u << lane) - 1u;
    visit([&](uint32_t k, int e) {
      const int j = wa + 32 * e;
      const bool is_eq = k == prefix && j < cn;
      const unsigned eqs = __ballot_sync(0xffffffffu, is_eq);
      const bool keep = k > prefix || (is_eq && eq_at + __popc(eqs & below) < left);
      const unsigned kept = __ballot_sync(0xffffffffu, keep);
      if (keep) index[at + __popc(kept & below)] = c0 + j;
      at += __popc(kept);
      eq_at += __popc(eqs);
    });
  }
  // no CTA leaves while another may still read its counts
  if (cluster > 1) cg::this_cluster().sync();
  if constexpr (COPY) copy_rows();
}

// Kept rows of K, V and the weights.  Grid y = sequence, x = runs of (output row, head) items, heads
// fastest, so that what a block writes is one stretch.  A group of threads copies an item, a thread
// one B-byte piece of its K or V row; four items of each group are in flight (two and eight were as
// fast, one 25% slower; rows moved by bulk copies through shared memory took 248 us where this takes
// 175 us = 92% of the copy rate, at 64 x 2048 of 4096-8192 keys, 8 heads of 128).
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
  const int es = p.dtype == VLF_F32 ? 4 : 2;
  const bool whole = p.d_qk * es % 16 == 0 && p.d_v * es % 16 == 0;
  const long long most = std::min(p.max_kv, p.budget);
  // CTAs per (sequence, kv head): one per 8192 keys of the longest sequence, eight at most.  Threads
  // and keys per thread by the share of a CTA and by how many lists there are: 256 threads up to 1024
  // keys, and up to 8192 where there are more lists than two per SM (four CTAs to an SM: 64 x 8 lists
  // of 4-8k keys, rows copied, 206 us; 216 with 1024 threads each), else 1024 (7 lists of 2-7k keys
  // 16.5 us, with 256 threads 20.6; 46 x 2 lists 29 and 33).  Lists of at most
  // 1024 keys whose rows are whole pieces are copied by the CTA that selected them, as long as one CTA
  // has at most 256 KB to move: the second launch would cost more.
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)cluster * 8192 < p.max_kv) cluster *= 2;
  const int share = (p.max_kv + cluster - 1) / cluster;
  const bool copy = share <= 1024 && whole && most * (p.d_qk + p.d_v) * es <= 262144;
  int threads = 1024;
  const void *sel;
  const bool few = (long long)p.num_seqs * p.h_kv <= 152 * 2;
  if (share <= 1024) {
    threads = 256;
    sel = copy ? reinterpret_cast<const void *>(evict_select_kernel<4, 256, true>)
               : reinterpret_cast<const void *>(evict_select_kernel<4, 256, false>);
  } else if (share <= 8192 && few) {
    sel = share <= 4096 ? reinterpret_cast<const void *>(evict_select_kernel<4, 1024, false>)
                        : reinterpret_cast<const void *>(evict_select_kernel<8, 1024, false>);
  } else if (share <= 8192) {
    threads = 256;
    sel = share <= 4096 ? reinterpret_cast<const void *>(evict_select_kernel<16, 256, false>)
                        : reinterpret_cast<const void *>(evict_select_kernel<32, 256, false>);
  } else if (share <= 16384) {
    sel = reinterpret_cast<const void *>(evict_select_kernel<16, 1024, false>);
  } else {
    sel = share <= 32768 ? reinterpret_cast<const void *>(evict_select_kernel<32, 1024, false>)
                         : reinterpret_cast<const void *>(evict_select_kernel<0, 1024, false>);
  }
  EvictParams a = p;
  void *args[2] = {&a, &cluster};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_seqs * cluster, p.h_kv);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelExC(&cfg, sel, args);
  if (e != cudaSuccess) {
    cudaGetLastError();  // (reported here: not left behind for a later check)
    return e;
  }
  count_launch();
  if (copy || most == 0 || p.total_out == 0) return cudaSuccess;
  const int b = whole ? 16 : es;
  int rk = p.d_qk * es / b, rv = p.d_v * es / b;
  // rounds of a block: as many, up to eight, as leave a grid of eight blocks per SM (four are resident,
  // by their 64 registers a thread)
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
