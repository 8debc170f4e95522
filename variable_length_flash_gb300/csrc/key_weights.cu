// Attention weight received by each key:
//   weights[g, j] = prev[g, j] + sum over the query rows i that see key j and the heads h of kv
//                   head g of exp(scale * q_i,h . k_j,g - lse[h, i]),
// the column sums of the attention matrix, recomputed from the forward's log-sum-exp.  A row whose
// lse is -inf (it sees no key) gives nothing.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

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
  KeyWeightParams a = kp;
  void *args[1] = {&a};
  return launch_plain(reinterpret_cast<const void *>(simt_key_weights_kernel<T>), grid, kThreads, smem, st, args);
}

cudaError_t simt_key_weights(const KeyWeightParams &kp, cudaStream_t st) {
  if (kp.p.dtype == VLF_F32) return launch_simt<float>(kp, st);
  if (kp.p.dtype == VLF_BF16) return launch_simt<__nv_bfloat16>(kp, st);
  return launch_simt<__half>(kp, st);
}

// ------------------------------------------------------------------------------ tensor-core kernel
// 16-bit data, widths 64, 96, 128 and 192.  S^T = K Q^T with the keys as the 128 rows of the MMA:
// a TMEM lane is a key, its columns are (query row, head) pairs, so a key's sum is the sum of one
// thread's registers -- no reduction across threads, no atomics, a fixed order.  The scores never
// leave TMEM; per score the epilogue does half a packed FMA, one ex2 and half a packed add.
//
// Two shapes of the same pipeline (TMA producer warp, MMA warp, a warp that fetches the columns' lse,
// two warpgroups that take the score tiles in turn, a TMEM buffer each):
//  * STREAM_K, where all rows of a (sequence, kv head) make at most 128 columns (decode steps, a
//    window of rows): Q stays in shared memory, a CTA streams a run of key tiles through a ring and
//    each tile's 128 weights are complete at once.  Bound: HBM, K read once.
//  * otherwise (whole prompts): the key tile stays, the column tiles stream, the sums stay in
//    registers until the last.  Where the key tiles alone leave SMs idle, the column tiles are cut
//    into parts whose sums a second kernel adds in order.
// Measured, bf16 / fp16, width 128: 64 decode rows of 32 heads against 1-8k keys of 8 kv heads 95 us
// (97% of the copy rate); 4 x 32 rows against 12-32k keys 37 us (77%: the rest is the CTAs' start and
// end, one wave of them); 4 x 4096 causal rows, 32 heads, 271 us against 145 us of products: tensor
// pipe 47% of its cycles, exponentials 47%, issue slots 56%, and per score tile two CTAs of an SM
// wait for one another's products, TMEM loads and exponentials in turn.  Tried and slower: score
// buffers released in halves of 64 columns (295), four warpgroups of sums (419), the key tile in TMEM
// as the MMA's A operand, which leaves room for 96 columns (277); as fast: fragments of four keys per
// thread (tcgen05.ld 16x256b), which read each -lse once for four keys.
// Columns: Gb heads (the largest divisor of the group that is at most 128) x R rows, column
// c = row c / Gb, head c mod Gb, one TMA box.  Rows and keys of other sequences that a box holds
// are masked by selection, so that nothing in them reaches a sum.
using namespace tc;

struct KwMaps {
  CUtensorMap q, k;
};

struct KwPlan {
  int stream_k;
  int gb, nhb;      // heads per column tile, column tiles per row block
  int rows;         // query rows per column tile
  int ncol;         // MMA N: rows * gb rounded up to 16
  int slots;        // ring slots of the streamed operand
  int run;          // STREAM_K: key tiles per CTA
  int splits;       // otherwise: parts of the column tiles
  int smem;
  int k_bytes, q_bytes, q_blk;
};

constexpr int kKwThreads = 352;  // producer, MMA issuer, lse warp, eight epilogue warps
constexpr int kKwMisc = 1024;  // barriers, flags
constexpr int kMaxSlots = 8;
constexpr int kLseBytes = 5 * 128 * 4;  // four buffers in turn, and the second warpgroup's sums

template <int D, bool BF16, bool STREAM_K>
__global__ void __launch_bounds__(kKwThreads, D <= 128 ? 2 : 1)
tc_key_weights_kernel(const __grid_constant__ KwMaps maps, const KeyWeightParams kp, const KwPlan pl,
                      float *parts) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_trigger();
  pdl_wait();
  const Params &p = kp.p;
  constexpr int KB = (D + 63) / 64, KBLK = 128 * 128;
  const int s = STREAM_K ? (int)blockIdx.z : (int)blockIdx.z / pl.splits, hk = blockIdx.y;
  Seq sq;
  if (!load_seq(p, s, sq)) return;
  if (s == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_kv) != 0)) set_error(p.err, VLF_ERR_BAD_SEQLENS);
  if (s == p.num_seqs - 1 && (sq.q0 + sq.q_len != p.total_q || sq.k0 + sq.kv_len != p.total_kv))
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
  // key tiles [t0, t1) of this CTA (one where the columns stream)
  const int ntiles = (sq.kv_len + 127) / 128;
  const int t0 = STREAM_K ? (int)blockIdx.x * pl.run : (int)blockIdx.x;
  const int t1 = min(ntiles, STREAM_K ? t0 + pl.run : t0 + 1);
  if (t0 >= t1) return;
  const int off = sq.kv_len - sq.q_len;
  // the rows that see some key of tile t
  auto band = [&](int t, int &lo, int &hi) {
    q_band(t * 128, min(t * 128 + 128, sq.kv_len), sq.q_len, sq.kv_len, p.causal, p.window, lo, hi);
  };
  // column tiles [c0, c1): row block c / nhb, head block c mod nhb
  int c0 = 0, c1 = 0;
  if (!STREAM_K) {
    int lo, hi;
    band(t0, lo, hi);
    if (hi > lo) {
      c0 = lo / pl.rows * pl.nhb;
      c1 = ((hi + pl.rows - 1) / pl.rows) * pl.nhb;
      const int part = (int)blockIdx.z % pl.splits, per = (c1 - c0 + pl.splits - 1) / pl.splits;
      c0 = min(c1, c0 + part * per);
      c1 = min(c1, c0 + per);
    }
  }
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_ALIGN);
    return;
  }
  const int nk = STREAM_K ? pl.slots : 1, nq = STREAM_K ? 1 : pl.slots;
  const uint32_t sK = base, sQ = sK + nk * pl.k_bytes, sM = sQ + nq * pl.q_bytes;
  // barriers: fixed operand, ring full / empty, score buffers full / empty, drain
  auto bar = [&](int i) { return sM + 8u * (uint32_t)i; };
  constexpr int B_FIX = 0, B_RF = 1, B_RE = B_RF + kMaxSlots, B_SF = B_RE + kMaxSlots, B_SE = B_SF + 2,
                B_DRAIN = B_SE + 2;
  uint8_t *misc = smem_raw + (sM - base);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(misc + 512);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 516);
  volatile int *dead_s = reinterpret_cast<volatile int *>(misc + 528);  // [score tile mod 4]: see below
  float *lse_s = reinterpret_cast<float *>(misc + kKwMisc);  // [score tile mod 4][128], then [128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(B_FIX), 1);
    for (int i = 0; i < pl.slots; ++i) { mbar_init(bar(B_RF + i), 1); mbar_init(bar(B_RE + i), 1); }
    // (a score buffer is ready with its product and its columns' lse)
    for (int i = 0; i < 2; ++i) { mbar_init(bar(B_SF + i), 2); mbar_init(bar(B_SE + i), 4); }
    mbar_init(bar(B_DRAIN), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  // two score buffers of ncol columns (an allocation is a power of two, 32 at least)
  const int half = pl.ncol <= 16 ? 16 : pl.ncol <= 32 ? 32 : pl.ncol <= 64 ? 64 : 128;
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 2 * half);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_holder;
  // The walk, the same for every role: score tiles n = 0, 1, ...; STREAM_K: the key tiles that some
  // row sees; otherwise the column tiles.
  const int first = STREAM_K ? t0 : c0, last = STREAM_K ? t1 : c1;
  auto live = [&](int t) {
    if (!STREAM_K) return true;
    int lo, hi;
    band(t, lo, hi);
    return hi > lo;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t q_tx = (uint32_t)(KB * pl.gb * pl.rows * 128);
      auto load_k = [&](int t, uint32_t dst, uint32_t b) {
        mbar_expect_tx(b, KB * KBLK);
        for (int c = 0; c < KB; ++c)
          tma_load_2d(dst + c * KBLK, &maps.k, hk * D + 64 * c, sq.k0 + t * 128, b);
      };
      auto load_q = [&](int c, uint32_t dst, uint32_t b) {
        mbar_expect_tx(b, q_tx);
        for (int x = 0; x < KB; ++x)
          tma_load_3d(dst + x * pl.q_blk, &maps.q, 64 * x, hk * p.group + c % pl.nhb * pl.gb,
                      sq.q0 + c / pl.nhb * pl.rows, b);
      };
      bool fixed = false, ok = true;
      int n = 0;
      for (int t = first; t < last && ok; ++t) {
        if (!live(t)) continue;
        if (!fixed) {
          if (STREAM_K) load_q(0, sQ, bar(B_FIX));
          else load_k(t0, sK, bar(B_FIX));
          fixed = true;
        }
        const int sl = n % pl.slots;
        if (n >= pl.slots) ok = mbar_wait(bar(B_RE + sl), (n / pl.slots - 1) & 1, abort_flag, p.err);
        if (!ok) break;
        if (STREAM_K) load_k(t, sK + sl * pl.k_bytes, bar(B_RF + sl));
        else load_q(t, sQ + sl * pl.q_bytes, bar(B_RF + sl));
        ++n;
      }
      // no copy may still be landing when the CTA leaves
      if (fixed) drain_wait(bar(B_FIX), 0);
      for (int i = 0; i < pl.slots && i < n; ++i)
        drain_wait(bar(B_RF + i), ((n - 1 - i) / pl.slots) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t id = idesc_f16(BF16 ? 1 : 0, 128, (uint32_t)pl.ncol, 0, 0);
    const uint64_t dk0 = sdesc_sw128(sK, 16, 1024), dq0 = sdesc_sw128(sQ, 16, 1024);
    bool ok = true, fixed = false;
    int n = 0;
    for (int t = first; t < last && ok; ++t) {
      if (!live(t)) continue;
      const int sl = n % pl.slots, b = n & 1;
      if (!fixed) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_FIX), 0, abort_flag, p.err));
        if (!ok) break;
        fixed = true;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar(B_RF + sl), (n / pl.slots) & 1, abort_flag, p.err));
      if (!ok) break;
      if (n >= 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_SE + b), ((n >> 1) - 1) & 1, abort_flag, p.err));
        if (!ok) break;
      }
      fence_after();
      const uint64_t dk = dk0 + (uint64_t)((STREAM_K ? sl * pl.k_bytes : 0) >> 4);
      const uint64_t dq = dq0 + (uint64_t)((STREAM_K ? 0 : sl * pl.q_bytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t ok_ = (uint64_t)(((kk >> 2) * KBLK + (kk & 3) * 32) >> 4);
        const uint64_t oq = (uint64_t)(((kk >> 2) * pl.q_blk + (kk & 3) * 32) >> 4);
        mma_ss_w(tmem + half * b, dk + ok_, dq + oq, id, kk > 0);
      }
      mma_commit_w(bar(B_SF + b));
      mma_commit_w(bar(B_RE + sl));
      ++n;
    }
    mma_commit_w(bar(B_DRAIN));
    drain_wait(bar(B_DRAIN), 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ -lse of the columns
    // One warp fetches it for all: the loads of the next tile pass under this one.
    const int valid = pl.rows * pl.gb;  // columns that hold a (row, head) pair
    const bool one_hb = pl.nhb == 1;    // (saves the divisions)
    int ri[4], hi_[4];                  // row and head of this lane's four columns
#pragma unroll
    for (int e = 0; e < 4; ++e) { ri[e] = (lane + 32 * e) / pl.gb; hi_[e] = (lane + 32 * e) % pl.gb; }
    auto fetch = [&](int c, float (&x)[4]) {  // (-inf where there is no row)
      const int rb = one_hb ? c : c / pl.nhb, r0 = rb * pl.rows;
      const int h0 = hk * p.group + (one_hb ? 0 : (c - rb * pl.nhb) * pl.gb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = -INFINITY;
        if (lane + 32 * e < valid && r0 + ri[e] < sq.q_len)
          x[e] = __ldg(kp.lse + (size_t)(h0 + hi_[e]) * p.total_q + sq.q0 + r0 + ri[e]);
      }
    };
    float next[4];
    bool ok = true;
    int n = 0;
    if (first < last) fetch(STREAM_K ? 0 : first, next);
    for (int t = first; t < last; ++t) {
      if (!live(t)) continue;
      const int b = n & 1;
      if (n >= 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_SE + b), ((n >> 1) - 1) & 1, abort_flag, p.err));
        if (!ok) break;
      }
      // Four buffers: this one's last reader has since released a later score tile.
      if (!STREAM_K || n < 4) {  // (STREAM_K: the same columns for every tile)
#pragma unroll
        for (int e = 0; e < 4; ++e)  // what the exponent adds; -inf takes the column out
          lse_s[128 * (n & 3) + lane + 32 * e] = next[e] == -INFINITY ? -INFINITY : -next[e] * kLog2e;
        // (a row without an lse is passed over by selection: its logits may be NaN)
        const int dead = __any_sync(0xffffffffu, next[0] == -INFINITY || next[1] == -INFINITY ||
                                                 next[2] == -INFINITY || next[3] == -INFINITY);
        if (lane == 0) dead_s[n & 3] = dead;
        if (!STREAM_K && t + 1 < last) fetch(t + 1, next);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_SF + b));
      ++n;
    }
  } else {
    // ------------------------------------------------------------------ sums
    const int wg = (warp - 3) >> 2, quarter = warp & 3, tid = 32 * quarter + lane;
    const uint32_t s_addr = tmem + half * wg + ((uint32_t)(32 * quarter) << 16);
    const uint32_t la0 = smem_u32(lse_s);
    const int valid = pl.rows * pl.gb;
    const bool one_hb = pl.nhb == 1;
    const float sl2 = p.scale_log2;
    const uint64_t scale2 = f2pack(sl2, sl2);
    float total = 0.f;
    bool ok = true;
    int lo = 0, hi = 0;  // the rows that see this thread's key
    if (!STREAM_K) visible_rows(min(t0 * 128 + tid, sq.kv_len - 1), off, sq.q_len, p.causal, p.window, lo, hi);
    int n = 0;  // score tiles so far, both warpgroups'
    for (int t = first; t < last; ++t) {
      const bool is_live = live(t);
      if (!is_live ? (t & 1) != wg : (n & 1) != wg) {
        n += is_live;
        continue;
      }
      // this thread's key, and the columns that see it
      const int j = (STREAM_K ? t : t0) * 128 + tid;
      const size_t at = (size_t)hk * p.total_kv + sq.k0 + j;
      float before = 0.f;
      if (STREAM_K && kp.prev && j < sq.kv_len) before = kp.prev[at];  // (kernel may write in place)
      float sum = 0.f;
      if (is_live) {
        if (STREAM_K) visible_rows(min(j, sq.kv_len - 1), off, sq.q_len, p.causal, p.window, lo, hi);
        const int r0 = STREAM_K ? 0 : (one_hb ? t : t / pl.nhb) * pl.rows;
        const int clo = min(max(lo - r0, 0), pl.rows) * pl.gb, chi = min(max(hi - r0, 0), pl.rows) * pl.gb;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_SF + wg), (n >> 1) & 1, abort_flag, p.err));
        if (!ok) break;
        fence_after();
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        const uint32_t la = la0 + 512 * (n & 3);
        auto release = [&]() {  // the score buffer may be overwritten
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_SE + wg));
        };
        // Adds the W columns from c on, loaded into v; FULL: every key of the warp sees all of them, and
        // all have an lse.  (All 128: groups of 3, 5, 6 and 7 heads, whose tiles hold 125 or 126 rows, go
        // through the selects on every tile.)
        auto add = [&](auto width, auto whole, const uint32_t *v, int c) {
          constexpr int W = decltype(width)::value;
          constexpr bool FULL = decltype(whole)::value;
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            uint64_t l0, l1;  // two pairs of -lse
            lds_b64x2(la + 4 * (c + e), l0, l1);
            float2 a = f2unpack(fma2(f2pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), scale2, l0));
            float2 b = f2unpack(fma2(f2pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), scale2, l1));
            if constexpr (!FULL) {
              const int x = c + e;
              const float2 la = f2unpack(l0), lb = f2unpack(l1);
              a.x = x >= clo && x < chi && la.x != -INFINITY ? a.x : -INFINITY;
              a.y = x + 1 >= clo && x + 1 < chi && la.y != -INFINITY ? a.y : -INFINITY;
              b.x = x + 2 >= clo && x + 2 < chi && lb.x != -INFINITY ? b.x : -INFINITY;
              b.y = x + 3 >= clo && x + 3 < chi && lb.y != -INFINITY ? b.y : -INFINITY;
            }
            acc0 = add2(acc0, f2pack(ex2(a.x), ex2(a.y)));
            acc1 = add2(acc1, f2pack(ex2(b.x), ex2(b.y)));
          }
        };
        constexpr std::integral_constant<int, 32> w32{};
        __syncwarp();
        if (half == 16) {
          uint32_t v[16];
          tmem_ld16(s_addr, v);
          tmem_ld_wait();
          release();
          add(std::integral_constant<int, 16>{}, std::false_type{}, v, 0);
        } else if (__all_sync(0xffffffffu, clo <= 0 && chi >= 128 && dead_s[n & 3] == 0)) {
          // 32 columns are added while the next 32 load
          uint32_t v0[32], v1[32];
          tmem_ld32(s_addr, v0);
          tmem_ld_wait_for(v0);
          tmem_ld32(s_addr + 32, v1);
          add(w32, std::true_type{}, v0, 0);
          tmem_ld_wait_for(v1);
          tmem_ld32(s_addr + 64, v0);
          add(w32, std::true_type{}, v1, 32);
          tmem_ld_wait_for(v0);
          tmem_ld32(s_addr + 96, v1);
          add(w32, std::true_type{}, v0, 64);
          tmem_ld_wait_for(v1);
          release();
          add(w32, std::true_type{}, v1, 96);
        } else {
#pragma unroll 1
          for (int c = 0; c < valid; c += 32) {
            // (a chunk that no key of the warp sees is passed over)
            if (!__any_sync(0xffffffffu, c < chi && c + 32 > clo)) continue;
            uint32_t v[32];
            tmem_ld32(s_addr + c, v);
            tmem_ld_wait_for(v);
            add(w32, std::false_type{}, v, c);
          }
          release();
        }
        const float2 f0 = f2unpack(acc0), f1 = f2unpack(acc1);
        sum = (f0.x + f0.y) + (f1.x + f1.y);
        ++n;
      }
      if (STREAM_K) {
        if (j < sq.kv_len) kp.weights[at] = kp.prev ? before + sum : sum;
      } else {
        total += sum;
      }
    }
    if (!STREAM_K) {
      // the two warpgroups' sums of each key
      if (wg == 1) lse_s[512 + tid] = total;
      named_sync(1, 256);
      const int j = t0 * 128 + tid;
      if (wg == 0 && j < sq.kv_len && ok) {
        const float w = total + lse_s[512 + tid];
        const size_t at = (size_t)hk * p.total_kv + sq.k0 + j;
        if (parts) parts[(size_t)((int)blockIdx.z % pl.splits) * p.h_kv * p.total_kv + at] = w;
        else kp.weights[at] = kp.prev ? kp.prev[at] + w : w;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, 2 * half);
  }
}

// weights = prev + the parts, in their order.
__global__ void __launch_bounds__(256) key_weights_join_kernel(const float *parts, int splits, size_t n,
                                                               const float *prev, float *weights) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float w = 0.f;
  for (int x = 0; x < splits; ++x) w += parts[(size_t)x * n + i];
  weights[i] = prev ? prev[i] + w : w;
}

bool tc_shape(int d, int dtype, unsigned flags) {
  return (dtype == VLF_F16 || dtype == VLF_BF16) && !(flags & VLF_FLAG_FORCE_SIMT) &&
         (d == 64 || d == 96 || d == 128 || d == 192);
}

KwPlan make_plan(int num_seqs, int max_q, int max_kv, int h_q, int h_kv, int d, int num_sms) {
  KwPlan pl{};
  const int group = h_q / h_kv, kb = (d + 63) / 64;
  pl.gb = std::min(group, 128);
  while (group % pl.gb) --pl.gb;
  pl.nhb = group / pl.gb;
  pl.stream_k = pl.nhb == 1 && (long long)max_q * group <= 128;
  pl.rows = pl.stream_k ? max_q : 128 / pl.gb;
  pl.ncol = (pl.rows * pl.gb + 15) / 16 * 16;
  pl.k_bytes = kb * 128 * 128;
  pl.q_blk = pl.ncol * 128;
  pl.q_bytes = kb * pl.q_blk;
  // ring slots: what fits beside the fixed operand in half an SM's shared memory (two CTAs per SM:
  // one's start and end run under the other's loop), else in all of it
  const int fixed = (pl.stream_k ? pl.q_bytes : pl.k_bytes) + kKwMisc + kLseBytes;
  const int slot = pl.stream_k ? pl.k_bytes : pl.q_bytes;
  pl.slots = (115712 - fixed) / slot;
  if (pl.slots < 2) pl.slots = (232448 - fixed) / slot;
  pl.slots = std::min(pl.slots, kMaxSlots);
  pl.smem = fixed + pl.slots * slot;
  const long long tiles = (long long)((max_kv + 127) / 128), ctas = tiles * h_kv * num_seqs;
  const long long room = 2ll * num_sms;  // CTAs resident
  pl.run = 1;
  pl.splits = 1;
  if (pl.stream_k) {
    // One wave of CTAs where that takes at most 32 tiles each (a CTA's start and end cost about three
    // tiles), else runs of at most 16, whose many waves even out ragged lengths.  Measured: 4 x 32
    // rows against up to 32k keys 35 us in one wave (27 tiles), 38 with 6 or 13 tiles, 43 with 3 or 16;
    // 64 decode rows against up to 8k keys 95 us with 13 tiles, 98 with 16 or more, 109 with 64.  The rule
    // has a step where one wave ends, which costs: 64 decode rows, 8 kv heads, against 2432 keys each 53 us
    // with 32 tiles, against 2500 keys 61 us with 4 (6230 and 5530 GB/s); from 3500 keys on (5 tiles,
    // 76 us) the rate is back, at 4096 keys (6 tiles) 86 us, at 8192 (13 tiles) 165 us.
    const long long wave = (ctas + room - 1) / room;
    pl.run = (int)(wave <= 32 ? wave : std::min(16ll, std::max(1ll, ctas / (8 * room))));
  } else if (ctas < room) {
    const long long cols = ((long long)max_q + pl.rows - 1) / pl.rows * pl.nhb;
    pl.splits = (int)std::max<long long>(1, std::min({room / ctas, cols / 4, 65535ll / num_seqs, 32ll}));
  }
  return pl;
}

template <int D>
cudaError_t launch_tc(const KeyWeightParams &kp, const KwPlan &pl, float *parts, cudaStream_t st) {
  const Params &p = kp.p;
  KwMaps maps;
  const int bf = p.dtype == VLF_BF16;
  const uint64_t kc = (uint64_t)p.h_kv * D;
  if (!make_tmap_16bit(&maps.k, p.k, p.total_kv, kc, kc, 128, bf) ||
      !make_tmap_q3(&maps.q, p.q, p.total_q, p.h_q, D, pl.gb, pl.rows, bf))
    return cudaErrorInvalidValue;
  const void *kern = pl.stream_k ? (bf ? (const void *)tc_key_weights_kernel<D, true, true>
                                       : (const void *)tc_key_weights_kernel<D, false, true>)
                                 : (bf ? (const void *)tc_key_weights_kernel<D, true, false>
                                       : (const void *)tc_key_weights_kernel<D, false, false>);
  cudaError_t e = set_smem_once(kern, pl.smem);
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)((p.max_kv + 127) / 128);
  const dim3 grid(pl.stream_k ? (tiles + pl.run - 1) / pl.run : tiles, p.h_kv, (unsigned)p.num_seqs * pl.splits);
  float *out = pl.splits > 1 ? parts : nullptr;
  KeyWeightParams a = kp;
  KwPlan b = pl;
  void *args[4] = {&maps, &a, &b, &out};
  e = launch_kernel(kern, grid, kKwThreads, pl.smem, st, args);
  if (e != cudaSuccess) return e;
  count_launch();
  if (pl.splits > 1) {
    const size_t n = (size_t)p.h_kv * p.total_kv;
    if ((n + 255) / 256 > 0x7fffffffull) return cudaErrorInvalidValue;
    const float *in = parts;
    int splits = pl.splits;
    size_t all = n;
    void *jargs[5] = {&in, &splits, &all, &a.prev, &a.weights};
    e = launch_plain((const void *)key_weights_join_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, st, jargs);
  }
  return e;
}

}  // namespace

size_t key_weights_workspace(int num_seqs, int total_kv, int max_q, int max_kv, int h_q, int h_kv, int d,
                             int dtype, unsigned flags, int num_sms) {
  if (num_seqs < 1 || total_kv < 1 || max_q < 1 || max_kv < 1 || h_kv < 1 || h_q < 1 || h_q % h_kv ||
      num_sms < 1 || !tc_shape(d, dtype, flags))
    return 0;
  const KwPlan pl = make_plan(num_seqs, max_q, max_kv, h_q, h_kv, d, num_sms);
  return pl.splits > 1 ? (size_t)pl.splits * h_kv * total_kv * sizeof(float) : 0;
}

cudaError_t key_weights(const KeyWeightParams &kp, void *workspace, int num_sms, cudaStream_t st) {
  const Params &p = kp.p;
  // (without rows or keys there is nothing to stage: the sums are empty)
  if (!tc_shape(p.d_qk, p.dtype, p.flags) || p.total_q == 0 || p.total_kv == 0 || p.max_q == 0)
    return simt_key_weights(kp, st);
  const KwPlan pl = make_plan(p.num_seqs, p.max_q, p.max_kv, p.h_q, p.h_kv, p.d_qk, num_sms);
  float *parts = static_cast<float *>(workspace);
  if (p.d_qk == 64) return launch_tc<64>(kp, pl, parts, st);
  if (p.d_qk == 96) return launch_tc<96>(kp, pl, parts, st);
  if (p.d_qk == 128) return launch_tc<128>(kp, pl, parts, st);
  return launch_tc<192>(kp, pl, parts, st);
}

}  // namespace vlf
