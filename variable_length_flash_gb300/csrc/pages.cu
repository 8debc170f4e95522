// A cache of pages: keys and values of a layer held in e4m3 as [num_pages][h_kv][page][d], with one fp32
// scale for each page and head ([num_pages][h_kv]), reached through the sequences' page tables.  Here are
// the kernels that write tokens into pages, copy pages, and keep the tables: which pages the sequences of
// the next step have (fork), and the pages in use moved to the front (compact).
#include <type_traits>

#include "e4m3.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ writing
// A value rounds to nearest e4m3 of x / scale.  The scale is a power of two, so a page whose scale grows
// loses nothing but what falls below e4m3's least step: bytes already there are multiplied by
// old / new and rounded again.  (A scale that is not a power of two, 448 / amax say, would round the whole
// page anew with each token that raises it.)
//
// Bound: HBM, each token read once, a byte written for it.  A block has one page of one head, of K or of
// V: it keeps the rows in registers between the maximum and the rounding.  Measured: 66k tokens of 8 heads of
// 128 in bf16, 74 us (81% of the copy rate; 300 us with values kept in fp32 and places found by division), in fp32
// 110 (91%); 64 single tokens 3.6 us, which is a launch.
constexpr int kKeep = 8;  // chunks a thread keeps; what is behind them is read again

// V values as they are read.
template <typename T, int V> struct Values {
  static constexpr int W = V == 1 ? 1 : V * sizeof(T) / 16;
  typename std::conditional<V == 1, T, uint4>::type r[W];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = reinterpret_cast<decltype(&r[0])>(const_cast<T *>(p))[i];
  }
  // The bits of an infinity, and of a number that 16 bits hold.
  static constexpr uint32_t kInf = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  static __device__ __forceinline__ float number(uint32_t b) {
    return tc::unpack2(b, std::is_same<T, __nv_bfloat16>::value).x;
  }
  // The larger of m and the values' sizes, as bits (of two 16-bit values at a time, m in both halves).
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 4) return max(m, __float_as_uint(r[0]) & 0x7fffffffu);
      else return max(m, (uint32_t)(*reinterpret_cast<const uint16_t *>(&r[0]) & 0x7fffu));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 4) m = max(m, w[e] & 0x7fffffffu);
          else m = __vmaxu2(m, w[e] & 0x7fff7fffu);
        }
      }
      return m;
    }
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
    if constexpr (V == 1) {
      x[0] = to_f32<T>(r[0]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 4) {
            x[4 * i + e] = __uint_as_float(w[e]);
          } else {
            const float2 f = tc::unpack2(w[e], std::is_same<T, __nv_bfloat16>::value);
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
          }
        }
      }
    }
  }
};

// The unit blockIdx.x of a call: sequence s has the units from cu[s] / page + 2 s on, at least as many as
// its tokens touch pages.
template <typename T, int V, int NT>
__global__ void __launch_bounds__(NT) pages_write_kernel(const PagesWriteParams p) {
  __shared__ uint32_t top[NT / 32];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int unit = blockIdx.x, head = blockIdx.y >> 1, is_v = blockIdx.y & 1;
  int s = 0, hi = p.num_seqs;
  while (hi - s > 1) {
    const int mid = (s + hi) / 2;
    if ((ld(p.cu + mid) >> p.log2_page) + 2 * mid <= unit) s = mid;
    else hi = mid;
  }
  const int t0 = ld(p.cu + s), t1 = ld(p.cu + s + 1), len = ld(p.kv_lens + s);
  if (t0 < 0 || t0 > t1 || t1 > p.total || len < t1 - t0 || (len > 0 && (len - 1) >> p.log2_page >= p.max_pages)) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_BAD_SEQLENS);
    return;
  }
  if (t0 == t1) return;
  const int first = len - (t1 - t0), nth = unit - ((t0 >> p.log2_page) + 2 * s);
  const int index = (first >> p.log2_page) + nth;
  if (nth < 0 || index > (len - 1) >> p.log2_page) return;
  const int page = ld(p.table + (long long)s * p.max_pages + index);
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_BAD_PAGES);
    return;
  }
  // slots [a, b) of the page take tokens t .. t + b - a
  const int base = index << p.log2_page, a = max(first - base, 0), b = min(len - base, p.page);
  const long long t = (long long)t0 + (base + a - first);
  const int d = is_v ? p.d_v : p.d_qk;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  const T *x = static_cast<const T *>(is_v ? p.v : p.k) + t * stride + (long long)head * d;
  const long long slot = (long long)page * p.h_kv + head;
  uint8_t *bytes = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages) + slot * p.page * d;
  float *scale = (is_v ? p.v_scale : p.k_scale) + slot;
  const float was = *scale;

  // a thread has one chunk of V columns of every R-th row
  const int chunks = d / V, R = NT / chunks, r0 = threadIdx.x / chunks, rows = r0 < R ? b - a : 0;
  const int c0 = (threadIdx.x - r0 * chunks) * V;
  const T *const mine = x + (long long)r0 * stride + c0;
  Values<T, V> kept[kKeep];
  // f(row, chunk) for this thread's rows: the ones it keeps, then the others, read again
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (r0 + k * R < rows) f(r0 + k * R, kept[k]);
    for (int r = r0 + kKeep * R; r < rows; r += R) {
      Values<T, V> v;
      v.load(x + (long long)r * stride + c0);
      f(r, v);
    }
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (r0 + k * R < rows) kept[k].load(mine + (long long)(k * R) * stride);
  // the largest size, as bits: those of numbers are ordered as the numbers are, and infinities and NaN are
  // above them all (16-bit values two at a time)
  auto block_max = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (NT > 32) {
      __syncthreads();
      if (threadIdx.x % 32 == 0) top[threadIdx.x / 32] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) m = max(m, top[i]);
    }
    return m;
  };
  uint32_t bits = 0;
  each([&](int, const Values<T, V> &v) { bits = v.most(bits); });
  if constexpr (sizeof(T) == 2) bits = max(bits & 0xffffu, bits >> 16);
  bits = block_max(bits);
  const bool odd = bits >= Values<T, V>::kInf;
  if (odd) {  // without what is not finite
    bits = 0;
    each([&](int, const Values<T, V> &v) {
      float y[V];
      v.get(y);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (fabsf(y[e]) <= 3.402823466e38f) bits = max(bits, __float_as_uint(fabsf(y[e])));
    });
    bits = block_max(bits);
  }
  const float m = odd || sizeof(T) == 4 ? __uint_as_float(bits) : Values<T, V>::number(bits);
  float now = page_scale(m);
  if (a > 0 && was >= now) now = was;  // (slot 0 begins a page: what its scale was does not count)
  const float inv = 1.f / now;
  if (a > 0 && now != was) {
    const float ratio = was / now;
    for (int i = threadIdx.x; i < p.page * d / 2; i += NT) {
      const int c0 = 2 * i / d;
      // (pairs of bytes: d may be odd, but a page has an even number of rows)
      uint16_t *at2 = reinterpret_cast<uint16_t *>(bytes) + i;
      if (c0 >= a && (2 * i + 1) / d < b) continue;
      const float2 f = e4m3_pair(*at2);
      *at2 = (uint16_t)e4m3x2(f.x * ratio, f.y * ratio);
    }
    if constexpr (NT > 32) __syncthreads();
    else __syncwarp();
  }
  uint8_t *const out = bytes + a * d + c0;
  auto store = [&](int r, const Values<T, V> &v) {
    uint8_t *to = out + r * d;
    float x[V];
    v.get(x);
    if constexpr (V == 1) {
      *to = (uint8_t)e4m3_byte(x[0], inv);
    } else {
      uint32_t w[2] = {0, 0};
      if (odd) {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e / 4] |= e4m3_byte(x[e], inv) << 8 * (e % 4);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[e] = e4m3x2(x[4 * e] * inv, x[4 * e + 1] * inv) | e4m3x2(x[4 * e + 2] * inv, x[4 * e + 3] * inv) << 16;
      }
      *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    }
  };
  each(store);
  if (threadIdx.x == 0 && now != was) *scale = now;
}

// A launch that starts as the one ahead of it in the stream ends (its kernel waits for that one first).
cudaError_t launch_step(const void *kern, dim3 grid, int threads, cudaStream_t st, void **args) {
  const cudaError_t e = launch_dependent(kern, grid, threads, 0, st, args);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t write(PagesWriteParams p, cudaStream_t st) {
  constexpr int A = 16 / sizeof(T);
  const bool vec = p.d_qk % 8 == 0 && p.d_v % 8 == 0 && p.k_stride % A == 0 && p.v_stride % A == 0;
  // one warp where a sequence has a few tokens (a decode step), else enough threads to keep a page
  const bool few = (long long)p.total <= 4ll * p.num_seqs;
  const int nt = few ? 32 : p.page * max(p.d_qk, p.d_v) <= 8 * kKeep * 128 ? 128 : 256;
  const void *kern = vec ? (nt == 32    ? (const void *)pages_write_kernel<T, 8, 32>
                            : nt == 128 ? (const void *)pages_write_kernel<T, 8, 128>
                                        : (const void *)pages_write_kernel<T, 8, 256>)
                         : (const void *)pages_write_kernel<T, 1, 256>;
  const dim3 grid((unsigned)((p.total >> p.log2_page) + 2 * p.num_seqs), (unsigned)(2 * p.h_kv));
  void *args[1] = {&p};
  return launch_step(kern, grid, vec ? nt : 256, st, args);
}

// ------------------------------------------------------------------------------ copying
// Bound: HBM.  Pair i is page src[i] over page dst[i], all heads; a block has `chunk` pairs' segments of
// 16 KB, four wide loads a thread in flight.  Measured: 4368 of 8723 pairs, pages of 128 KB, 173 us (97% of the copy
// rate; with chunks of 32 189, of 2 177, of 1 194).
constexpr int kSegment = 16384;

__global__ void __launch_bounds__(256) pages_copy_kernel(const PagesCopyParams p) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const long long kb = (long long)p.h_kv * p.page * p.d_qk, vb = (long long)p.h_kv * p.page * p.d_v;
  const int ks = (int)((kb + kSegment - 1) / kSegment);
  const bool is_v = (int)blockIdx.y >= ks;
  const long long at = (long long)(is_v ? blockIdx.y - ks : blockIdx.y) * kSegment;
  const long long size = is_v ? vb : kb;
  const int n = (int)((min(size, at + kSegment) - at) / 16);  // (a page has 16 rows or more)
  uint8_t *pages = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
  float *scale = is_v ? p.v_scale : p.k_scale;
  const int i0 = blockIdx.x * p.chunk, i1 = min(i0 + p.chunk, p.n);
  for (int i = i0; i < i1; ++i) {
    const int src = ld(p.src + i), dst = ld(p.dst + i);
    if (src < 0) continue;
    if (src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
      if (threadIdx.x == 0) set_error(p.err, VLF_ERR_BAD_PAGES);
      continue;
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(pages + (long long)src * size + at);
    uint4 *to = reinterpret_cast<uint4 *>(pages + (long long)dst * size + at);
    uint4 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (threadIdx.x + 256 * k < n) r[k] = from[threadIdx.x + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (threadIdx.x + 256 * k < n) to[threadIdx.x + 256 * k] = r[k];
    if (at == 0)
      for (int h = threadIdx.x; h < p.h_kv; h += 256)
        scale[(long long)dst * p.h_kv + h] = scale[(long long)src * p.h_kv + h];
  }
}

// ------------------------------------------------------------------------------ tables
// Bound: latency; a call is three or four dependent steps, each a launch that starts while the one before ends
// (its blocks are there already, and wait).  256 rows of up to 1041 pages on 256 others, with their copies: 15.5 us,
// of which the entries and counts are 1 us at the memory's rate; 21.1 with a warp for each row in the last step
// instead of a block (a row's entries are 33 loads one behind another then), 66 as one cluster of eight CTAs with its
// barriers between the steps (eight SMs look at a quarter of a million entries).  Tables of few entries
// take one block (below).
constexpr int kChunk = 1024;  // pages of a block that counts

__device__ __forceinline__ int pages_of(int len, int log2_page) { return (int)(((long long)len + (1 << log2_page) - 1) >> log2_page); }
__device__ __forceinline__ void step_begins() {
  tc::pdl_trigger();
  tc::pdl_wait();
}

// Sum over a block of 256 threads; every thread gets it.
__device__ __forceinline__ long long block_sum(long long x) {
  __shared__ long long red[8];
  for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  x = 0;
  for (int i = 0; i < 8; ++i) x += red[i];
  return x;
}
// How many of the flags of a chunk's pages are set, as each thread has four of them in a row: before its own, and in all.
__device__ __forceinline__ int chunk_before(int mine, int &all) {
  __shared__ int red[8];
  const int lane = threadIdx.x % 32;
  int y = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) red[threadIdx.x / 32] = y;
  __syncthreads();
  int before = y - mine;
  all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    before += i < (int)threadIdx.x / 32 ? red[i] : 0;
    all += red[i];
  }
  return before;
}

// A new row's parent, its length and the whole pages in it.
struct Row {
  int parent, len, whole;
  bool part;
};
__device__ __forceinline__ Row row_of(const PagesForkParams &p, int s) {
  Row r{ld(p.parents + s), 0, 0, false};
  if (r.parent >= 0 && r.parent < p.num_in) r.len = max(0, ld(p.lens + r.parent));
  r.whole = r.len >> p.log2_page;
  r.part = (r.len & ((1 << p.log2_page) - 1)) != 0;
  return r;
}
// Holders of page i once the new rows have what they share or keep.
__device__ __forceinline__ int held(const PagesForkParams &p, int i) {
  const int n = p.outside[i] + p.whole[i];
  return n == 0 && p.owner[i] != 0x7fffffff ? 1 : n;
}
// The page that a new row goes on in, and whether it keeps it (else it takes a copy).
__device__ __forceinline__ int part_of(const PagesForkParams &p, const Row &r, int s, bool &keeps) {
  keeps = false;
  if (!r.part || r.whole >= p.max_pages) return -1;
  const int page = ld(p.table + (long long)r.parent * p.max_pages + r.whole);
  if (page < 0 || page >= p.num_pages) return -1;
  keeps = p.outside[page] + p.whole[page] == 0 && p.owner[page] == s;
  return page;
}

// Fork.  outside[p]: holders of p that are no row of the old table; whole[p]: new rows that have it whole;
// owner[p]: the first new row that goes on inside it; list: each chunk's free pages in order; counts: how many;
// need[s]: new pages of the rows before row s in its 256; group: those of each 256 rows; state: an
// error, free pages, new pages.
__global__ void __launch_bounds__(256) fork_begin_kernel(const PagesForkParams p) {
  step_begins();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i < p.num_pages) {
    p.outside[i] = p.refs[i];
    p.whole[i] = 0;
    p.owner[i] = 0x7fffffff;
  }
  if (i < 4) p.state[i] = 0;
}

// The old rows' holds and the new ones'.  Grid y: rows, the old ones first; x: runs of 256 entries.
__global__ void __launch_bounds__(256) fork_count_kernel(const PagesForkParams p) {
  step_begins();
  const int j = blockIdx.x * 256 + threadIdx.x;
  for (int y = blockIdx.y; y < p.num_in + p.num_out; y += gridDim.y) {
    const bool old = y < p.num_in;
    const int s = y - p.num_in;
    Row r{y, 0, 0, false};
    if (old) {
      r.len = ld(p.lens + y);
      if (r.len < 0 || pages_of(r.len, p.log2_page) > p.max_pages) {
        if (j == 0) p.state[0] = VLF_ERR_BAD_SEQLENS;
        continue;
      }
    } else {
      r = row_of(p, s);
      const int grow = ld(p.grow + s);
      if (j == 0 && r.parent >= p.num_in) p.state[0] = VLF_ERR_BAD_PAGES;
      if (grow < 0 || (long long)r.len + grow > (long long)p.max_pages << p.log2_page) {
        if (j == 0) p.state[0] = VLF_ERR_BAD_SEQLENS;
        continue;
      }
    }
    if (j >= min(pages_of(r.len, p.log2_page), p.max_pages)) continue;
    const int page = ld(p.table + (long long)r.parent * p.max_pages + j);
    if (page < 0 || page >= p.num_pages) p.state[0] = VLF_ERR_BAD_PAGES;
    else if (old) atomicSub(p.outside + page, 1);
    else if (j < r.whole) atomicAdd(p.whole + page, 1);
    else atomicMin(p.owner + page, s);
  }
}

// The free pages of a chunk (a block each); the blocks behind them: what new rows need, 256 a block.
__global__ void __launch_bounds__(256) fork_free_kernel(const PagesForkParams p) {
  step_begins();
  int n = 0;
  if ((int)blockIdx.x < p.chunks) {
    const long long i0 = (long long)blockIdx.x * kChunk + 4 * threadIdx.x;
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = i0 + k < p.num_pages;
      if (in && (p.outside[i0 + k] < 0 || p.refs[i0 + k] < 0)) p.state[0] = VLF_ERR_BAD_PAGES;
      mine |= (uint32_t)(in && held(p, (int)i0 + k) == 0) << k;
    }
    int *at = p.list + (long long)blockIdx.x * kChunk + chunk_before(__popc(mine), n);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (mine >> k & 1) *at++ = (int)i0 + k;
    if (threadIdx.x == 0) {
      p.counts[blockIdx.x] = n;
      atomicAdd(p.state + 1, n);
    }
    return;
  }
  const int s = (blockIdx.x - p.chunks) * 256 + threadIdx.x;
  if (s < p.num_out) {
    const Row r = row_of(p, s);
    bool keeps;
    const int page = part_of(p, r, s, keeps);
    const long long to = min((long long)r.len + max(0, ld(p.grow + s)), (long long)p.max_pages << p.log2_page);
    n = pages_of((int)to, p.log2_page) - pages_of(r.len, p.log2_page) + (page >= 0 && !keeps);
  }
  int sum;
  const int before = chunk_before(n, sum);  // (may wrap only where the call asks for more pages than there are)
  if (s < p.num_out) p.need[s] = before;
  const long long all = block_sum(n);
  if (threadIdx.x == 0) p.group[blockIdx.x - p.chunks] = sum;
  if (threadIdx.x == 0) atomicAdd(reinterpret_cast<unsigned long long *>(p.state + 2), (unsigned long long)all);
}

// The new counts (a block for each chunk), and the new rows (a block each; its first warp finds the new pages).
__global__ void __launch_bounds__(256) fork_end_kernel(const PagesForkParams p) {
  step_begins();
  const int bad = p.state[0], free = p.state[1], lane = threadIdx.x % 32;
  const long long need = *reinterpret_cast<const long long *>(p.state + 2);
  const bool ok = bad == 0 && need <= free;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (bad) set_error(p.err, bad);
    *p.left = bad ? (int)0x80000000 : (int)max((long long)free - need, -0x7fffffffll);
  }
  if ((int)blockIdx.x < p.chunks) {
    long long before = 0;
    for (int c = threadIdx.x; c < (int)blockIdx.x; c += 256) before += p.counts[c];
    const int at = (int)block_sum(before);  // free pages in front of the chunk
    const long long i0 = (long long)blockIdx.x * kChunk + 4 * threadIdx.x;
    int holds[4], mine = 0;  // of this thread's four pages
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      holds[k] = i0 + k < p.num_pages ? held(p, (int)i0 + k) : 1;
      mine += holds[k] == 0;
    }
    int all, rank = at + chunk_before(mine, all);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long i = i0 + k;
      if (i >= p.num_pages) continue;
      // the pages given out are the first `need` free ones
      if (!ok) p.refs_out[i] = p.refs[i];
      else if (holds[k] == 0) p.refs_out[i] = rank++ < need;
      else p.refs_out[i] = holds[k];
    }
    return;
  }
  const int s = blockIdx.x - p.chunks;
  if (s >= p.num_out) return;  // (a call without rows)
  long long sum = 0;
  for (int g = threadIdx.x; g < s / 256; g += 256) sum += p.group[g];
  sum = block_sum(sum) + p.need[s];  // new pages of the rows before
  const Row r = row_of(p, s);
  bool keeps;
  const int part = part_of(p, r, s, keeps);
  const bool copy = ok && part >= 0 && !keeps;
  const int len = ok ? r.len + ld(p.grow + s) : 0, has = pages_of(len, p.log2_page);
  const int32_t *row = p.table + (long long)r.parent * p.max_pages;
  int *out = p.table_out + (long long)s * p.max_pages;
  const int shared = ok ? r.whole + (keeps ? 1 : 0) : 0;  // entries that stay
  for (int j0 = threadIdx.x; j0 < p.max_pages; j0 += 4 * 256) {
    int x[4];  // (loads in flight together: a store between them would hold the next one up)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = j0 + 256 * k < min(r.whole, has) ? ld(row + j0 + 256 * k) : part;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 256 * k;
      if (j < p.max_pages && (j < shared || j >= has)) out[j] = j >= has ? -1 : x[k];
    }
  }
  if (threadIdx.x >= 32) return;
  // the new pages are the free ones of ranks sum, sum + 1, ...; a lane looks at eight chunks
  const long long end = sum + has - shared;
  int first = -1;
  long long base = 0;
  for (int c0 = 0; c0 < p.chunks && base < end && has > shared; c0 += 256) {
    const int c = c0 + 8 * lane;
    int n[8], y = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = c + i < p.chunks ? p.counts[c + i] : 0;
      y += n[i];
    }
    const int own = y;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    const long long at = base + y - own;
    for (uint32_t m = __ballot_sync(0xffffffffu, at < end && at + own > sum); m; m &= m - 1) {
      const int from = __ffs(m) - 1;
      long long lo = __shfl_sync(0xffffffffu, at, from);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = __shfl_sync(0xffffffffu, n[i], from);
        const int *list = p.list + (long long)(c0 + 8 * from + i) * kChunk - lo;
        for (long long g = max(lo, sum) + lane; g < min(lo + k, end); g += 32) {
          const int page = list[g];
          out[shared + (int)(g - sum)] = page;
          if (g == sum) first = page;
        }
        lo += k;
      }
    }
    base += __shfl_sync(0xffffffffu, y, 31);
  }
  first = __reduce_max_sync(0xffffffffu, first);  // (one lane met it)
  if (lane == 0) {
    p.lens_out[s] = len;
    p.src[s] = copy ? part : -1;
    p.dst[s] = copy ? first : -1;
  }
}

// Small calls as one block of 1024 threads, counters and free pages in shared memory: 32 rows of 16 pages on 8 others
// take 6.8 us with their copies, the steps above 10.7 and a cluster of eight CTAs 13.1; the host spends 5.7 us on
// the call instead of 11.9.
constexpr int kSmallPages = 4096, kSmallRows = 1024, kSmallEntries = 32768;

// The sum of x over the threads before this one, and over all (1024 threads).
__device__ __forceinline__ int before_1024(int x, int &all) {
  __shared__ int red[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) red[warp] = y;
  __syncthreads();
  const int r = red[lane];
  all = __reduce_add_sync(0xffffffffu, r);
  return y - x + __reduce_add_sync(0xffffffffu, lane < warp ? r : 0);
}

__global__ void __launch_bounds__(1024) fork_small_kernel(PagesForkParams p) {
  extern __shared__ int dyn[];
  __shared__ int begin[kSmallRows], bad;
  step_begins();
  const int t = threadIdx.x, warp = t / 32, lane = t % 32;
  int *const list = dyn + 3 * p.num_pages;
  p.outside = dyn;
  p.whole = dyn + p.num_pages;
  p.owner = dyn + 2 * p.num_pages;
  for (int i = t; i < p.num_pages; i += 1024) {
    p.outside[i] = p.refs[i];
    p.whole[i] = 0;
    p.owner[i] = 0x7fffffff;
  }
  if (t == 0) bad = 0;
  __syncthreads();
  for (int y = warp; y < p.num_in + p.num_out; y += 32) {
    const int s = y - p.num_in;
    Row r{y, 0, 0, false};
    if (s < 0) {
      r.len = ld(p.lens + y);
      if (r.len < 0 || pages_of(r.len, p.log2_page) > p.max_pages) {
        if (lane == 0) bad = VLF_ERR_BAD_SEQLENS;
        continue;
      }
    } else {
      r = row_of(p, s);
      const int grow = ld(p.grow + s);
      if (lane == 0 && r.parent >= p.num_in) bad = VLF_ERR_BAD_PAGES;
      if (grow < 0 || (long long)r.len + grow > (long long)p.max_pages << p.log2_page) {
        if (lane == 0) bad = VLF_ERR_BAD_SEQLENS;
        continue;
      }
    }
    const int n = min(pages_of(r.len, p.log2_page), p.max_pages);
    const int32_t *row = p.table + (long long)r.parent * p.max_pages;
    for (int j = lane; j < n; j += 32) {
      const int page = ld(row + j);
      if (page < 0 || page >= p.num_pages) bad = VLF_ERR_BAD_PAGES;
      else if (s < 0) atomicSub(p.outside + page, 1);
      else if (j < r.whole) atomicAdd(p.whole + page, 1);
      else atomicMin(p.owner + page, s);
    }
  }
  __syncthreads();
  // the free pages in order, and where each new row's new pages begin among them
  int free = 0, need = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += 1024) {
    const int i = i0 + t;
    const bool in = i < p.num_pages, is = in && held(p, i) == 0;
    if (in && (p.outside[i] < 0 || p.refs[i] < 0)) bad = VLF_ERR_BAD_PAGES;
    int all;
    const int at = free + before_1024(is, all);
    if (is) list[at] = i;
    free += all;
  }
  bool keeps = false;
  Row mine{-1, 0, 0, false};
  int part = -1, more = 0;
  if (t < p.num_out) {
    mine = row_of(p, t);
    part = part_of(p, mine, t, keeps);
    const long long to = min((long long)mine.len + max(0, ld(p.grow + t)), (long long)p.max_pages << p.log2_page);
    more = pages_of((int)to, p.log2_page) - pages_of(mine.len, p.log2_page) + (part >= 0 && !keeps);
  }
  const int at = before_1024(more, need);  // (at most kSmallEntries pages)
  if (t < p.num_out) begin[t] = at;
  __syncthreads();
  const bool ok = bad == 0 && need <= free;
  if (t == 0) {
    if (bad) set_error(p.err, bad);
    *p.left = bad ? (int)0x80000000 : free - need;
  }
  if (t < p.num_out) {
    const bool copy = ok && part >= 0 && !keeps;
    p.lens_out[t] = ok ? mine.len + ld(p.grow + t) : 0;
    p.src[t] = copy ? part : -1;
    p.dst[t] = copy ? list[at] : -1;
  }
  for (int i = t; i < p.num_pages; i += 1024) {
    if (!ok) p.refs_out[i] = p.refs[i];
    else if (const int n = held(p, i)) p.refs_out[i] = n;
  }
  if (ok)
    for (int i = t; i < free; i += 1024) p.refs_out[list[i]] = i < need;
  for (int s = warp; s < p.num_out; s += 32) {
    const Row r = row_of(p, s);
    bool keep;
    const int page = part_of(p, r, s, keep);
    const int has = ok ? pages_of(r.len + ld(p.grow + s), p.log2_page) : 0, stay = r.whole + (keep ? 1 : 0);
    const int32_t *row = p.table + (long long)r.parent * p.max_pages;
    int *out = p.table_out + (long long)s * p.max_pages;
    for (int j = lane; j < p.max_pages; j += 32)
      out[j] = j >= has ? -1 : j < r.whole ? ld(row + j) : j < stay ? page : list[begin[s] + j - stay];
  }
}

// Compact.  Of the U pages in use the ones behind the first U pages move into the free ones among them, the
// first into the first.
__global__ void __launch_bounds__(256) compact_count_kernel(const PagesCompactParams p) {
  step_begins();
  int n = 0;
#pragma unroll
  for (int k = 0; k < kChunk / 256; ++k) {
    const long long i = (long long)blockIdx.x * kChunk + k * 256 + threadIdx.x;
    if (i >= p.num_pages) continue;
    n += p.refs[i] > 0;
    if (i < p.num_pages / 2) p.src[i] = p.dst[i] = -1;
  }
  n = (int)block_sum(n);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = n;
}
// order[p]: which of the moving pages p is (-1: none).
__global__ void __launch_bounds__(256) compact_list_kernel(const PagesCompactParams p) {
  step_begins();
  long long before = 0, total = 0;
  for (int c = threadIdx.x; c < p.chunks; c += 256) {
    const int n = p.counts[c];
    before += c < (int)blockIdx.x ? n : 0;
    total += n;
  }
  const int at = (int)block_sum(before), used = (int)block_sum(total);
  // pages in use among the first `used`
  long long front = 0;
  for (int c = threadIdx.x; c < used / kChunk; c += 256) front += p.counts[c];
  for (int i = used / kChunk * kChunk + threadIdx.x; i < used; i += 256) front += p.refs[i] > 0;
  front = block_sum(front);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.used = used;
  bool is[4];
  int mine = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long i = (long long)blockIdx.x * kChunk + 4 * threadIdx.x + k;
    is[k] = i < p.num_pages && p.refs[i] > 0;
    mine += is[k];
  }
  int all, rank = at + chunk_before(mine, all);  // pages in use before this one
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = (int)(blockIdx.x * kChunk + 4 * threadIdx.x + k);
    if (i >= p.num_pages) continue;
    p.order[i] = -1;
    if (is[k] && i >= used) {
      p.order[i] = rank - (int)front;
      p.src[rank - (int)front] = i;
    } else if (!is[k] && i < used) {
      p.dst[i - rank] = i;
    }
    rank += is[k];
  }
}
__global__ void __launch_bounds__(256) compact_end_kernel(const PagesCompactParams p) {
  step_begins();
  const long long step = (long long)gridDim.x * 256;
  auto moved = [&](int i) {  // where the page i in use is afterwards
    const int o = p.order[i];
    return o < 0 ? i : p.dst[o];
  };
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.num_pages; i += step) {
    const int n = p.refs[i], to = n > 0 ? moved((int)i) : -1;
    p.to[i] = to;
    if (n > 0) p.refs_out[to] = n;
    if (i >= *p.used) p.refs_out[i] = 0;
  }
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.entries; i += step) {
    const int page = p.table[i];
    p.table_out[i] = page >= 0 && page < p.num_pages && p.refs[page] > 0 ? moved(page) : -1;
  }
}

// The same for few pages and entries, as one block: src, dst and order in shared memory.
__global__ void __launch_bounds__(1024) compact_small_kernel(const PagesCompactParams p) {
  __shared__ short order[kSmallPages], dst[kSmallPages / 2];
  step_begins();
  const int t = threadIdx.x;
  int used = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += 1024) used += __syncthreads_count(i0 + t < p.num_pages && p.refs[i0 + t] > 0);
  int rank0 = 0, front = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += 1024) front += __syncthreads_count(i0 + t < used && p.refs[i0 + t] > 0);
  for (int i = t; i < p.num_pages / 2; i += 1024) p.src[i] = p.dst[i] = -1;
  __syncthreads();
  for (int i0 = 0; i0 < p.num_pages; i0 += 1024) {
    const int i = i0 + t;
    const bool in = i < p.num_pages, is = in && p.refs[i] > 0;
    int all;
    const int rank = rank0 + before_1024(is, all);  // pages in use before this one
    rank0 += all;
    if (!in) continue;
    order[i] = -1;
    if (is && i >= used) {
      order[i] = (short)(rank - front);
      p.src[rank - front] = i;
    } else if (!is && i < used) {
      dst[i - rank] = (short)i;
      p.dst[i - rank] = i;
    }
  }
  __syncthreads();
  auto moved = [&](int i) { return order[i] < 0 ? i : (int)dst[order[i]]; };
  for (int i = t; i < p.num_pages; i += 1024) {
    const int n = p.refs[i], to = n > 0 ? moved(i) : -1;
    p.to[i] = to;
    if (n > 0) p.refs_out[to] = n;
    if (i >= used) p.refs_out[i] = 0;
  }
  for (int i0 = t; i0 < (int)p.entries; i0 += 4 * 1024) {
    int page[4];  // (loads in flight together: a store between them would hold the next one up)
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = i0 + 1024 * k < (int)p.entries ? ld(p.table + i0 + 1024 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = page[k] >= 0 && page[k] < p.num_pages && ld(p.refs + page[k]) > 0 ? moved(page[k]) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + 1024 * k < (int)p.entries) p.table_out[i0 + 1024 * k] = page[k];
  }
  if (t == 0) *p.used = used;
}

size_t ints(long long n) { return ((size_t)n * 4 + 255) & ~(size_t)255; }
int chunks_of(int num_pages) { return (int)(((long long)num_pages + kChunk - 1) / kChunk); }
}  // namespace

cudaError_t pages_write(const PagesWriteParams &p, cudaStream_t st) {
  if (p.dtype == VLF_F32) return write<float>(p, st);
  if (p.dtype == VLF_BF16) return write<__nv_bfloat16>(p, st);
  return write<__half>(p, st);
}

cudaError_t pages_copy(PagesCopyParams p, cudaStream_t st) {
  auto segments = [&](int d) { return ((long long)p.h_kv * p.page * d + kSegment - 1) / kSegment; };
  const long long segs = segments(p.d_qk) + segments(p.d_v);
  // pairs per block: one where the call is small, eight where blocks of one are more than are resident (pairs
  // that are not to be copied cost a block each then; 32 leave the SMs unequal work)
  p.chunk = (int)max(1ll, min(8ll, (long long)p.n * segs / (152 * 8)));
  void *args[1] = {&p};
  return launch_step((const void *)pages_copy_kernel, dim3((unsigned)((p.n + p.chunk - 1) / p.chunk), (unsigned)segs), 256,
                     st, args);
}

size_t pages_fork_workspace(int num_pages, int num_out) {
  const int chunks = chunks_of(num_pages);
  return 3 * ints(num_pages) + ints((long long)chunks * kChunk) + ints(chunks) + ints(num_out) + ints((num_out + 255ll) / 256) + ints(4);
}
cudaError_t pages_fork(PagesForkParams p, void *workspace, cudaStream_t st) {
  char *w = static_cast<char *>(workspace);
  auto take = [&](long long n) {
    int *r = reinterpret_cast<int *>(w);
    w += ints(n);
    return r;
  };
  p.chunks = chunks_of(p.num_pages);
  p.outside = take(p.num_pages);
  p.whole = take(p.num_pages);
  p.owner = take(p.num_pages);
  p.list = take((long long)p.chunks * kChunk);
  p.counts = take(p.chunks);
  p.need = take(p.num_out);
  p.group = take((p.num_out + 255ll) / 256);
  p.state = take(4);
  void *args[1] = {&p};
  const int rows = p.num_in + p.num_out;
  if (p.num_pages <= kSmallPages && p.num_out <= kSmallRows && (long long)rows * p.max_pages <= kSmallEntries) {
    const int bytes = 4 * p.num_pages * (int)sizeof(int);
    cudaError_t e = set_smem_once((const void *)fork_small_kernel, bytes);
    if (e == cudaSuccess) e = launch_dependent((const void *)fork_small_kernel, dim3(1), 1024, bytes, st, args);
    if (e == cudaSuccess) count_launch();
    return e;
  }
  auto step = [&](const void *kern, dim3 grid) { return launch_step(kern, grid, 256, st, args); };
  cudaError_t e = step((const void *)fork_begin_kernel, dim3((unsigned)(((long long)max(p.num_pages, 4) + 255) / 256)));
  if (e == cudaSuccess && rows > 0)
    e = step((const void *)fork_count_kernel, dim3((unsigned)max(1, (p.max_pages + 255) / 256), (unsigned)min(rows, 65535)));
  const int behind = (int)((p.num_out + 255ll) / 256);
  if (e == cudaSuccess && p.chunks + behind > 0) e = step((const void *)fork_free_kernel, dim3((unsigned)(p.chunks + behind)));
  if (e == cudaSuccess) e = step((const void *)fork_end_kernel, dim3((unsigned)max(1ll, (long long)p.chunks + p.num_out)));
  return e;
}

size_t pages_compact_workspace(int num_pages) { return ints(chunks_of(num_pages)) + ints(num_pages); }
cudaError_t pages_compact(PagesCompactParams p, void *workspace, cudaStream_t st) {
  p.chunks = chunks_of(p.num_pages);
  p.counts = static_cast<int *>(workspace);
  p.order = reinterpret_cast<int *>(static_cast<char *>(workspace) + ints(p.chunks));
  void *args[1] = {&p};
  if (p.num_pages <= kSmallPages && p.entries <= kSmallEntries)
    return launch_step((const void *)compact_small_kernel, dim3(1), 1024, st, args);
  auto step = [&](const void *kern, long long blocks) { return launch_step(kern, dim3((unsigned)blocks), 256, st, args); };
  cudaError_t e = step((const void *)compact_count_kernel, p.chunks);
  if (e == cudaSuccess) e = step((const void *)compact_list_kernel, p.chunks);
  if (e == cudaSuccess)
    e = step((const void *)compact_end_kernel, min((max(p.entries, (long long)p.num_pages) + 255) / 256, 152ll * 8));
  return e;
}

}  // namespace vlf
