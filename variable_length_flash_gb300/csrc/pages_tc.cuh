// What the tensor-core kernels over pages share (pages_tc.cu, pages_rows.cu): the items of a call and the equal
// runs of key tiles that they are cut into, parts of items and their join.
#pragma once

#include <type_traits>

#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace pages {

using namespace tc;

constexpr float kLn2 = 0.69314718055994531f;

struct TcParams {
  PagesAttnParams a;
  float *part;  // [2 grid][columns (D + 2)]
  int4 *rec;    // [grid][2] {sequence, kv head, query tile, units behind the run's end} of the item that a CTA begins and
                // leaves open (-1: none); then {units of the call (64 bits), CTAs with a run}
  int rows;     // query rows of a query tile
  int splits;   // query tiles of a row (a group with more heads than columns), else 1
  int magic;    // magic_of(group)
};
// c / group is c * this >> 16 for c < 256 (c * group < 2^16); where there are more heads it is not asked for.
inline int magic_of(int group) { return 65536 / group + 1; }

// The key tiles (of KEYS keys) of the items from one on, in order.
template <int KEYS> struct Walk {
  const TcParams *at;
  int s, head, qt;                // sequence, kv head, query tile
  int q0, q_len, len, tiles_q;    // of the sequence; tiles_q = 0: nothing to do
  int r0, r1, lo, hi, t0, nt;     // of the item: its rows, the keys they see, its key tiles (none: nt = 0)

  __device__ __forceinline__ explicit Walk(const TcParams &x) : at(&x) {}
  __device__ __forceinline__ bool load(int seq) {  // false: bad lengths
    s = seq;
    const TcParams &p = *at;
    const Params &b = p.a.p;
    const int x = ld(b.cu_q + s), y = ld(b.cu_q + s + 1);
    len = ld(p.a.kv_lens + s);
    q0 = x;
    q_len = y - x;
    tiles_q = 0;
    if (x < 0 || x > y || y > b.total_q || q_len > b.max_q || len < 0 ||
        (len > 0 && (len - 1) >> p.a.log2_page >= p.a.max_pages))
      return false;
    tiles_q = p.splits > 1 ? q_len * p.splits : (q_len + p.rows - 1) / p.rows;
    return true;
  }
  __device__ __forceinline__ void item() {
    const TcParams &p = *at;
    r0 = p.splits > 1 ? qt / p.splits : qt * p.rows;
    r1 = min(r0 + p.rows, q_len);
    kv_band(r0, r1, q_len, len, p.a.p.causal, p.a.p.window, lo, hi);
    t0 = lo / KEYS;
    nt = hi > lo ? (hi + KEYS - 1) / KEYS - t0 : 0;
  }
  __device__ __forceinline__ int units() const { return max(nt, 1); }
  // units of one head of the sequence
  __device__ __forceinline__ long long head_units() {
    long long n = 0;
    for (qt = 0; qt < tiles_q; ++qt) {
      item();
      n += units();
    }
    return n;
  }
  // to a unit of sequence seq; returns the unit within the item
  __device__ __forceinline__ int seek(int seq, long long unit) {
    load(seq);
    const long long per = head_units();
    head = (int)(unit / per);
    unit -= head * per;
    for (qt = 0;; ++qt) {
      item();
      if (unit < units()) return (int)unit;
      unit -= units();
    }
  }
  __device__ __forceinline__ void next() {
    if (++qt >= tiles_q) {
      qt = 0;
      if (++head >= at->a.p.h_kv) {
        head = 0;
        do {  // (there is another one: the caller has units left)
          if (s + 1 >= at->a.p.num_seqs) return;
          load(s + 1);
        } while (tiles_q == 0);
      }
    }
    item();
  }
};
// The query row and head of column c; false where there is none.
template <typename W>
__device__ __forceinline__ bool column_of(const TcParams &p, int nc, const W &w, int c, int &row, int &head) {
  const int group = p.a.p.group;
  if (p.splits > 1) {
    const int h = w.qt % p.splits * nc + c;
    row = w.r0;
    head = w.head * group + h;
    return h < group;
  }
  const int r = c * p.magic >> 16;
  row = w.r0 + r;
  head = w.head * group + c - r * group;
  return row < w.r1;
}

// Values that a wait has made good: what uses them is not scheduled ahead of it.
template <int N> __device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// N consecutive columns (no wait).
template <int N> __device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t *r) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr) : "memory");
  } else {
    tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r));
  }
}
// A CTA's run of units.
struct Run {
  bool any;
  long long total, grid, f0, f1;  // units of the call, CTAs with a run, this one's [f0, f1)
  int seq;                        // f0 is unit `unit` of sequence seq
  long long unit;
};
// Units of all sequences, then this CTA's run of them and where it begins: the THREADS threads take a sequence
// each.  red: THREADS / 32 + 2 numbers of shared memory.  Every thread comes here.
template <int KEYS, int THREADS>
__device__ __forceinline__ Run run_of(const TcParams &p, long long *red) {
  constexpr int WARPS = THREADS / 32;
  const Params &b = p.a.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Walk<KEYS> w(p);
  auto units_of = [&](int s, bool tell) -> long long {
    if (s >= b.num_seqs) return 0;
    if (!w.load(s)) {
      if (tell && blockIdx.x == 0) set_error(b.err, VLF_ERR_BAD_SEQLENS);
      return 0;
    }
    return w.head_units() * b.h_kv;
  };
  Run r{};
  long long mine = 0;
  for (int s0 = 0; s0 < b.num_seqs; s0 += THREADS) {
    mine = units_of(s0 + threadIdx.x, true);
    long long x = mine;
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    for (int i = 0; i < WARPS; ++i) r.total += red[i];
  }
  // (CTAs with a run, be it of one tile: 24 tiles of three short caches take 10.6 us, 13.7 with two tiles each)
  r.grid = max(1ll, min((long long)gridDim.x, r.total));
  r.any = r.total > 0 && blockIdx.x < r.grid;
  if (!r.any) return r;
  r.f0 = r.total * blockIdx.x / r.grid;
  r.f1 = r.total * (blockIdx.x + 1) / r.grid;
  long long *const start = red + WARPS;
  long long before = 0;
  for (int s0 = 0; s0 < b.num_seqs; s0 += THREADS) {
    const long long x = b.num_seqs <= THREADS ? mine : units_of(s0 + threadIdx.x, false);
    long long y = x;
    for (int o = 1; o < 32; o *= 2) {
      const long long z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    __syncthreads();
    if (lane == 31) red[warp] = y;
    __syncthreads();
    y += before;
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) y += red[i];
      before += red[i];
    }
    if (x > 0 && y - x <= r.f0 && r.f0 < y) {
      start[0] = s0 + threadIdx.x;
      start[1] = r.f0 - (y - x);
    }
    if (before > r.f0) break;
  }
  __syncthreads();
  r.seq = (int)start[0];
  r.unit = start[1];
  return r;
}
// The record of an item that has `rest` units behind the end of a run that begins it; none.
template <typename W> __device__ __forceinline__ void open_item(const TcParams &p, const Run &r, const W &w, int rest) {
  p.rec[2 * blockIdx.x] = make_int4(w.s, w.head, w.qt, rest);
  p.rec[2 * blockIdx.x + 1] = make_int4((int)(uint32_t)r.total, (int)(r.total >> 32), (int)r.grid, 0);
}
__device__ __forceinline__ void no_item(const TcParams &p) { p.rec[2 * blockIdx.x] = make_int4(-1, 0, 0, 0); }

// Joins the parts of the item that CTA blockIdx.x of the launch before began and others ended: out = sum_i f_i O_i /
// sum_i f_i l_i with f_i = 2^(reference_i - the largest).  A warp has a column of the item (grid y: runs of them),
// its lanes the parts' references and sums, then their D / 32 columns of O.
constexpr int kJoinWarps = 8;

template <int D, int NC, int KEYS, bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) pages_join_kernel(const TcParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using V = typename std::conditional<D == 128, float4, float2>::type;
  constexpr int PART = NC * (D + 2), FLY = 8;
  pdl_wait();
  pdl_trigger();
  const int4 rec = p.rec[2 * blockIdx.x];
  const int c = blockIdx.y * kJoinWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (rec.x < 0 || c >= NC) return;
  Walk<KEYS> w(p);
  w.load(rec.x);
  w.head = rec.y;
  w.qt = rec.z;
  w.item();
  int row, head;
  if (!column_of(p, NC, w, c, row, head)) return;
  // the last CTA with a part: the one that has the item's last unit
  const int4 of = p.rec[2 * blockIdx.x + 1];
  const long long total = (long long)(uint32_t)of.x | (long long)of.y << 32, grid = of.z;
  const long long end = total * (blockIdx.x + 1) / grid + rec.w;
  const int n = (int)((end * grid - 1) / total) - (int)blockIdx.x + 1;
  auto part = [&](int i) { return p.part + (2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * PART; };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float *x = part(i) + NC * D + c;
    if (x[NC] != 0.f) top = fmaxf(top, x[0]);
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float f = 0.f;  // (a part that saw nothing has no weight; a NaN sum stays one)
    if (i0 + lane < n) {
      const float *x = part(i0 + lane) + NC * D + c;
      const float l = x[NC];
      f = l == 0.f ? 0.f : ex2(x[0] - top);
      if (l != 0.f) sum = fmaf(f, l, sum);
    }
    for (int i = 0; i < 32 && i0 + i < n; i += FLY) {
      V x[FLY];
#pragma unroll
      for (int k = 0; k < FLY; ++k)
        if (i0 + i + k < n) x[k] = *reinterpret_cast<const V *>(part(i0 + i + k) + c * D + lane * (D / 32));
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, i + k);
        if (i0 + i + k >= n || fk == 0.f) continue;
        const float *y = reinterpret_cast<const float *>(&x[k]);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(fk, y[e], acc[e]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T y[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) y[e] = from_f32<T>(sum == 0.f ? 0.f : acc[e] * inv);
  T *out = static_cast<T *>(p.a.p.out) + ((long long)(w.q0 + row) * p.a.p.h_q + head) * D + lane * (D / 32);
  if constexpr (D == 128) *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<uint2 *>(y);
  else *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<uint32_t *>(y);
  if (lane == 0 && p.a.p.lse)
    p.a.p.lse[(long long)head * p.a.p.total_q + w.q0 + row] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * kLn2;
}

}  // namespace pages
}  // namespace vlf
