// Attention of a batch whose sequences all start with the same keys: the keys of sequence s are the
// shared prefix [0, P) followed by its own kv_len keys,
//   logit(i, j) = scale * q_i . k_j,   j < P: prefix key j;  j >= P: own key j - P,
// with the end-aligned causal and window rules over the P + kv_len keys (row i stands at key
// i + P + kv_len - q_len).  out and lse are those of the forward on the concatenated keys.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace vlf {
namespace {

// ------------------------------------------------------------------------------ fp32 FMA kernel
// Every type and head width up to 256.  A block of 128 threads owns 16 query rows of one (sequence,
// head); thread t works on row t / 8 and every 8th column, over tiles of 32 keys -- the prefix's,
// then the sequence's own (a tile never crosses the two).  Shared rows stay apart from their
// neighbours: a key or value behind the segment's end is staged as zero, never read.
constexpr int kRows = 16, kTile = 32, kThreads = 128;

__device__ __forceinline__ float lanes8_max(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float lanes8_sum(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
__device__ __forceinline__ void stage(float *dst, int ld, const T *src, long long row0, int n, int cap,
                                      int heads, int head, int d) {
  for (int idx = threadIdx.x; idx < cap * d; idx += kThreads) {
    const int r = idx / d, c = idx - r * d;
    dst[r * ld + c] = r < n ? to_f32<T>(src[((size_t)(row0 + r) * heads + head) * d + c]) : 0.f;
  }
}

template <typename T, int DVPT>
__global__ void __launch_bounds__(kThreads) simt_prefix_kernel(const PrefixParams pp) {
  extern __shared__ float smem[];
  const Params &p = pp.p;
  const int s = blockIdx.z, h = blockIdx.y, hk = h / p.group;
  Seq sq;
  if (!load_seq(p, s, sq)) return;
  if (s == 0 && (ld(p.cu_q) != 0 || ld(p.cu_kv) != 0)) set_error(p.err, VLF_ERR_BAD_SEQLENS);
  if (s == p.num_seqs - 1 && (sq.q0 + sq.q_len != p.total_q || sq.k0 + sq.kv_len != p.total_kv))
    set_error(p.err, VLF_ERR_BAD_SEQLENS);
  const int r0 = blockIdx.x * kRows;
  if (r0 >= sq.q_len) return;
  const int r1 = min(r0 + kRows, sq.q_len);
  const int P = pp.prefix_len, keys = P + sq.kv_len;
  const int dq = p.d_qk, dv = p.d_v, ldq = dq + 1;
  float *Qs = smem;                // [kRows][ldq]
  float *Ks = Qs + kRows * ldq;    // [kTile][ldq]
  float *Vs = Ks + kTile * ldq;    // [kTile][dv]
  float *Ps = Vs + kTile * dv;     // [kRows][kTile + 1]
  const int t = threadIdx.x, r = t >> 3, sub = t & 7, i = r0 + r;
  const bool row_ok = i < r1;
  const int off = keys - sq.q_len;
  int vlo, vhi;  // this row's visible keys
  visible_range(i, off, keys, p.causal, p.window, vlo, vhi);
  if (!row_ok) vhi = vlo;
  int lo, hi;    // the block's
  kv_band(r0, r1, sq.q_len, keys, p.causal, p.window, lo, hi);
  stage<T>(Qs, ldq, static_cast<const T *>(p.q), sq.q0 + r0, r1 - r0, kRows, p.h_q, h, dq);

  float m = -INFINITY, l = 0.f, o[DVPT];
#pragma unroll
  for (int u = 0; u < DVPT; ++u) o[u] = 0.f;
#pragma unroll 1
  for (int seg = 0; seg < 2; ++seg) {
    const int a = seg == 0 ? 0 : P, b = seg == 0 ? P : keys;  // the segment's keys
    const T *k = static_cast<const T *>(seg == 0 ? pp.k_pre : p.k);
    const T *v = static_cast<const T *>(seg == 0 ? pp.v_pre : p.v);
    const long long base = seg == 0 ? 0 : (long long)sq.k0 - P;  // packed row of key j: base + j
    const int e = min(b, hi);
#pragma unroll 1
    for (int kt = a + max(0, lo - a) / kTile * kTile; kt < e; kt += kTile) {
      const int nk = min(kTile, b - kt);
      __syncthreads();  // the tile before is consumed
      stage<T>(Ks, ldq, k, base + kt, nk, kTile, p.h_kv, hk, dq);
      stage<T>(Vs, dv, v, base + kt, nk, kTile, p.h_kv, hk, dv);
      __syncthreads();
      float sc[4], tmax = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int jj = sub + 8 * x, j = kt + jj;
        float y = -INFINITY;
        if (jj < nk && j >= vlo && j < vhi) {
          float acc = 0.f;
          for (int c = 0; c < dq; ++c) acc = fmaf(Qs[r * ldq + c], Ks[jj * ldq + c], acc);
          y = p.scale * acc;
        }
        sc[x] = y;
        tmax = fmaxf(tmax, y);
      }
      const float m_new = fmaxf(m, lanes8_max(tmax));
      // (no maximum yet: masked keys, whose weight is 0 from any reference, or NaN logits, which fmaxf
      // passes over and which have to reach the sums)
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = expf(m - ref);  // m = -inf: 0 (and a NaN sum stays NaN)
      float psum = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sc[x] = expf(sc[x] - ref);  // masked: 0
        psum += sc[x];
      }
      l = l * alpha + lanes8_sum(psum);
      m = m_new;
#pragma unroll
      for (int x = 0; x < 4; ++x) Ps[r * (kTile + 1) + sub + 8 * x] = sc[x];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < DVPT; ++u) o[u] *= alpha;
#pragma unroll 2
      for (int jj = 0; jj < nk; ++jj) {
        const float pj = Ps[r * (kTile + 1) + jj];
        const float *vrow = Vs + jj * dv;
#pragma unroll
        for (int u = 0; u < DVPT; ++u)
          if (sub + 8 * u < dv) o[u] = fmaf(pj, vrow[sub + 8 * u], o[u]);
      }
    }
  }
  if (!row_ok) return;
  const size_t grow = (size_t)sq.q0 + i;
  T *out = static_cast<T *>(p.out) + (grow * p.h_q + h) * dv;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int u = 0; u < DVPT; ++u)
    if (sub + 8 * u < dv) out[sub + 8 * u] = from_f32<T>(o[u] * inv);
  if (p.lse && sub == 0) p.lse[(size_t)h * p.total_q + grow] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T, int DVPT>
cudaError_t launch_simt(const PrefixParams &pp, cudaStream_t st) {
  const Params &p = pp.p;
  const int smem = (int)sizeof(float) * ((kRows + kTile) * (p.d_qk + 1) + kTile * p.d_v + kRows * (kTile + 1));
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(simt_prefix_kernel<T, DVPT>), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.max_q + kRows - 1) / kRows), p.h_q, p.num_seqs);
  PrefixParams a = pp;
  void *args[1] = {&a};
  return launch_plain(reinterpret_cast<const void *>(simt_prefix_kernel<T, DVPT>), grid, kThreads, smem, st, args);
}

template <typename T>
cudaError_t simt_by_width(const PrefixParams &pp, cudaStream_t st) {
  if (pp.p.d_v <= 64) return launch_simt<T, 8>(pp, st);
  if (pp.p.d_v <= 128) return launch_simt<T, 16>(pp, st);
  return launch_simt<T, 32>(pp, st);
}

cudaError_t simt_prefix(const PrefixParams &pp, cudaStream_t st) {
  if (pp.p.dtype == VLF_F32) return simt_by_width<float>(pp, st);
  if (pp.p.dtype == VLF_BF16) return simt_by_width<__nv_bfloat16>(pp, st);
  return simt_by_width<__half>(pp, st);
}

// ------------------------------------------------------------------------------ tensor-core kernel
// 16-bit data, widths 64, 96 and 128.  The pipeline of the forward's one-tile kernel: a CTA owns a
// 128-row tile (R query rows x Gb heads of a kv head, row r = query row r / Gb, head r mod Gb) and
// walks key tiles of 64 through TMA rings; one warp issues S = Q K^T, another O += P V with P read
// from TMEM, four warps run the online softmax, a thread per row.  What differs:
//  * Key tiles come from two tensors.  Tile j < np holds prefix keys 64 j ..., tile j >= np the
//    sequence's own keys 64 (j - np) ...; a tile never crosses the two, and keys are counted from the
//    prefix's first one, so that one interval of visible keys per row masks both.
//  * Two ways to cut the work.  Shared: the prefix part runs with tiles packed from the rows of ALL
//    sequences -- the prefix is read once per 128 / Gb rows of the batch, not once per sequence --
//    and the own keys run per sequence; a second kernel merges the parts' fp32 results by their
//    log-sum-exps.  Per sequence: each row tile walks prefix and own keys in one go (cut into parts
//    only where the row tiles are too few to fill the GPU).  Shared pays where a sequence's rows fill
//    less than a tile (decode steps): make_plan below.
//  * Quarter tiles (quad) where the rows -- a sequence's, or all of a small batch's against the prefix --
//    fill at most a quarter of a row tile (decode steps).
//    A softmax warp can only read its own 32 TMEM lanes, so with one row tile a single warp would walk
//    all 64 columns of each key tile and set the pace.  The rows are loaded four times instead, once
//    per quarter, and quarter w takes keys 16 w ... 16 w + 15 of each tile: four softmaxes over disjoint
//    keys, a quarter of the work each, joined at the end in shared memory.  The product for 16 keys
//    writes the lanes of their quarter alone: weights of zero in the others would make NaN of an
//    infinite value that a row sees.
//  * Measured, width 128, 32 heads on 8: 64 decode rows behind 16384 shared keys and 100-1024 own ones
//    50 us (floor 32 us of HBM; a CTA's start and end and about 1 us per key tile); 16 x 64-436 rows
//    behind 8192 and 436-2048, 530 us (floor 322 us of products; tensor pipe 63%): a key tile's S reads
//    48 KB of shared memory and its PV 16 KB while TMA writes 32 KB, 768 of the 1000 cycles it takes at
//    128 bytes a cycle.  3 decode rows behind 1000 keys 9 us, two launches.  Tried and slower: two
//    warps per quarter of the rows, 32 columns each (609 and 58 us).
//  * Values behind a sequence's last key belong to the next sequence: they are zeroed in shared memory
//    before the product, so that an infinity or NaN there (0 x inf) cannot reach this one.
using namespace tc;

struct PfxMaps {
  CUtensorMap q, q_own, k, v, kp, vp;
};

constexpr int kBN = 64;  // keys per tile
constexpr float kLn2f = 0.6931471805599453f;
constexpr float kMoveMax = 8.0f;  // the reference max moves once a row's max has grown by 2^8

struct PfxPlan {
  int shared;
  int gb, nhb;         // heads per row tile, row tiles per kv head's group
  int quad_pre, rows;  // shared prefix part: quarter tiles, query rows per row tile
  int quad, rows_own;  // the sequences' own CTAs: the same
  int np;              // prefix key tiles
  int heads;           // h_kv * nhb
  int rb_pre, rb_own;  // row blocks: of the batch (shared prefix part), of a sequence
  int parts_pre, parts_own;
  int parts;           // results per row to merge (0: written directly)
  unsigned n_pre, n_all;  // CTAs
};

template <int D>
struct PfxCfg {
  static constexpr int KB = (D + 63) / 64, NPAD = KB * 64;
  static constexpr int QBLK = 128 * 128, KVBLK = kBN * 128;
  static constexpr int Q_BYTES = KB * QBLK, T_BYTES = KB * KVBLK;
  static constexpr int NK = 3, NV = D == 64 ? 3 : 2;
  static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + NK * T_BYTES, OFF_BAR = OFF_V + NV * T_BYTES;
  static constexpr int B_Q = 0, B_KF = 1, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + NV;
  static constexpr int B_S = B_VE + NV, B_P = B_S + 2, B_O = B_P + 2, B_DRAIN = B_O + 2, NBAR = B_DRAIN + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tmem address, abort flag, band lo / hi
  static constexpr int OFF_SEQ = OFF_MISC + 16;         // uint16 [128]: the sequence of each row
  static constexpr int SMEM = OFF_SEQ + 256;
  static constexpr uint32_t O_COL = 128, TMEM_COLS = 256;
  static_assert(SMEM <= 115712, "two CTAs per SM");
};

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(256, 2)
tc_prefix_kernel(const __grid_constant__ PfxMaps maps, const PrefixParams pp, const PfxPlan pl, float *o_part,
                 float *lse_part) {
  using C = PfxCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_trigger();
  pdl_wait();
  const Params &p = pp.p;
  const int P = pp.prefix_len;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int is_bf16 = BF16 ? 1 : 0;

  // ---- this CTA's rows and key tiles
  // The shared prefix part's CTAs (bound by the tensor cores) and the own keys' (bound by HBM) take
  // turns, so that an SM holds one of each, while there are both.
  const unsigned both = 2 * min(pl.n_pre, pl.n_all - pl.n_pre), bid = blockIdx.x;
  const bool pre = SPLIT && (bid < both ? (bid & 1) == 0 : pl.n_pre > both / 2);
  const unsigned nth = bid < both ? bid / 2 : bid - both / 2;  // among its kind
  int hd, rb, part, slot;
  Seq sq{0, 0, 0, 0};
  if (pre) {
    // row blocks fastest: CTAs that read the same prefix tiles run together
    int x = (int)nth;
    rb = x % pl.rb_pre;
    x /= pl.rb_pre;
    hd = x % pl.heads;
    part = slot = x / pl.heads;
  } else {
    int x = (int)nth;
    part = x % pl.parts_own;
    x /= pl.parts_own;
    rb = x % pl.rb_own;
    x /= pl.rb_own;
    hd = x % pl.heads;
    const int s = x / pl.heads;
    if (!load_seq(p, s, sq)) return;
    if (s == 0 && (ld(p.cu_q) != 0 || ld(p.cu_kv) != 0)) set_error(p.err, VLF_ERR_BAD_SEQLENS);
    if (s == p.num_seqs - 1 && (sq.q0 + sq.q_len != p.total_q || sq.k0 + sq.kv_len != p.total_kv))
      set_error(p.err, VLF_ERR_BAD_SEQLENS);
    if (p.causal) rb = pl.rb_own - 1 - rb;  // the rows that see most first
    if (rb * pl.rows_own >= sq.q_len) return;
    slot = pl.parts_pre + part;
  }
  const int hk = hd / pl.nhb, h0 = hk * p.group + hd % pl.nhb * pl.gb;
  const bool quad = pre ? pl.quad_pre : pl.quad;
  const int rows = pre ? pl.rows : pl.rows_own;
  const int row0 = pre ? rb * rows : sq.q0 + rb * rows;                    // packed row of tile row 0
  const int nrows = min(rows, (pre ? p.total_q : sq.q0 + sq.q_len) - row0);  // query rows of the tile
  const int keys = P + sq.kv_len, off = keys - sq.q_len;                      // (per-sequence CTAs)
  // Softmax warps that hold a row.  The others have nothing to do: what they leave in P stands in
  // rows of O that nobody reads (a decode step's tile is mostly such rows).
  const int live_warps = quad ? 4 : (nrows * pl.gb + 31) / 32;

  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) set_error(p.err, VLF_ERR_ALIGN);
    return;
  }
  const uint32_t sQ = base, sK = base + C::OFF_K, sV = base + C::OFF_V;
  auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem_raw + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + C::OFF_MISC + 4);
  int *band = reinterpret_cast<int *>(smem_raw + C::OFF_MISC + 8);
  uint16_t *seq_of = reinterpret_cast<uint16_t *>(smem_raw + C::OFF_SEQ);

  if (threadIdx.x == 0) {
    mbar_init(bar(C::B_Q), 1);
    for (int i = 0; i < C::NK; ++i) { mbar_init(bar(C::B_KF + i), 1); mbar_init(bar(C::B_KE + i), 1); }
    for (int i = 0; i < C::NV; ++i) { mbar_init(bar(C::B_VF + i), 1); mbar_init(bar(C::B_VE + i), 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_S + i), 1);
      mbar_init(bar(C::B_P + i), 32 * live_warps);
      mbar_init(bar(C::B_O + i), 1);
      mbar_init(bar(C::B_DRAIN + i), 1);
    }
    *abort_flag = 0;
    band[0] = P;
    band[1] = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  }
  int lo, hi;  // key tiles
  if (pre) {
    // which sequence each row belongs to: the threads look at a sequence each (one round of loads),
    // and at what its rows in this tile see of the prefix
    if (threadIdx.x < 128) seq_of[threadIdx.x] = 0xffff;
    __syncthreads();
    for (int s = threadIdx.x; s < p.num_seqs; s += 256) {
      const int a = ld(p.cu_q + s), b = ld(p.cu_q + s + 1);
      const int c = ld(p.cu_kv + s), d = ld(p.cu_kv + s + 1);
      if (a < 0 || a > b || b > p.total_q || b - a > p.max_q || c < 0 || c > d || d > p.total_kv || d - c > p.max_kv)
        continue;  // (recorded by that sequence's own CTAs)
      const int x = max(a, row0), y = min(b, row0 + nrows);
      if (x >= y) continue;
      for (int i = x; i < y; ++i) seq_of[i - row0] = (uint16_t)s;
      int klo, khi;
      kv_band(x - a, y - a, b - a, P + d - c, p.causal, p.window, klo, khi);
      khi = min(khi, P);
      if (khi > klo) { atomicMin(&band[0], klo); atomicMax(&band[1], khi); }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (pre) {
    lo = band[1] > band[0] ? band[0] / kBN : 0;
    hi = band[1] > band[0] ? (band[1] + kBN - 1) / kBN : 0;
  } else {
    int klo, khi;
    kv_band(rb * rows, rb * rows + nrows, sq.q_len, keys, p.causal, p.window, klo, khi);
    lo = klo < P ? klo / kBN : pl.np + (klo - P) / kBN;
    hi = khi <= P ? (khi + kBN - 1) / kBN : pl.np + (khi - P + kBN - 1) / kBN;
    if (SPLIT && pl.shared) lo = max(lo, pl.np);  // the prefix part has CTAs of its own
    if (khi <= klo || hi < lo) hi = lo;
  }
  if (SPLIT) {
    // this part's share (possibly none: it then writes O = 0 and LSE = -inf)
    const int n = pre ? pl.parts_pre : pl.parts_own, per = (hi - lo + n - 1) / n;
    lo = min(hi, lo + part * per);
    hi = min(hi, lo + per);
  }
  const uint32_t tmem = *tmem_holder;
  // first key of tile j, and the end of the keys that its tensor holds for this CTA
  auto key_of = [&](int j) { return j < pl.np ? j * kBN : P + (j - pl.np) * kBN; };
  auto end_of = [&](int j) { return j < pl.np ? P : keys; };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0 && hi > lo) {
      mbar_expect_tx(bar(C::B_Q), (quad ? 4 : 1) * C::KB * pl.gb * rows * 128);
      for (int c = 0; c < C::KB; ++c)
        for (int x = 0; x < (quad ? 4 : 1); ++x)
          tma_load_3d(sQ + c * C::QBLK + x * 32 * 128, pre ? &maps.q : &maps.q_own, 64 * c, h0, row0, bar(C::B_Q));
      auto load = [&](const CUtensorMap *pm, const CUtensorMap *om, int j, uint32_t dst, uint32_t b) {
        const CUtensorMap *m = j < pl.np ? pm : om;
        const int y = j < pl.np ? j * kBN : sq.k0 + (j - pl.np) * kBN;
        mbar_expect_tx(b, C::T_BYTES);
        for (int c = 0; c < C::KB; ++c) tma_load_2d(dst + c * C::KVBLK, m, hk * D + 64 * c, y, b);
      };
      bool ok = true;
      int nk = 0, nv = 0;
      for (int j = lo; j < hi + 1 && ok; ++j) {  // K leads V by one tile
        if (j < hi) {
          const int sl = nk % C::NK;
          if (nk >= C::NK) ok = mbar_wait(bar(C::B_KE + sl), (nk / C::NK - 1) & 1, abort_flag, p.err);
          if (!ok) break;
          load(&maps.kp, &maps.k, j, sK + sl * C::T_BYTES, bar(C::B_KF + sl));
          ++nk;
        }
        if (j > lo) {
          const int sl = nv % C::NV;
          if (nv >= C::NV) ok = mbar_wait(bar(C::B_VE + sl), (nv / C::NV - 1) & 1, abort_flag, p.err);
          if (!ok) break;
          load(&maps.vp, &maps.v, j - 1, sV + sl * C::T_BYTES, bar(C::B_VF + sl));
          ++nv;
        }
      }
      // no copy may still be landing when the CTA leaves
      drain_wait(bar(C::B_Q), 0);
      for (int i = 0; i < C::NK && i < nk; ++i) drain_wait(bar(C::B_KF + i), ((nk - 1 - i) / C::NK) & 1);
      for (int i = 0; i < C::NV && i < nv; ++i) drain_wait(bar(C::B_VF + i), ((nv - 1 - i) / C::NV) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    if (hi > lo) {
      const uint32_t id = idesc_f16(is_bf16, 128, kBN, 0, 0);
      const uint64_t dq = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024);
      bool ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_Q), 0, abort_flag, p.err));
      for (int n = 0; n < hi - lo && ok; ++n) {
        const int b = n & 1, sl = n % C::NK;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_KF + sl), (n / C::NK) & 1, abort_flag, p.err));
        if (!ok) break;
        if (n >= 2) {  // S(n) overwrites the buffer that P(n - 2) was read from
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O + b), ((n - 2) >> 1) & 1, abort_flag, p.err));
          if (!ok) break;
        }
        fence_after();
        const uint64_t dk = dk0 + (uint64_t)((sl * C::T_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_w(tmem + 64 * b, dq + (uint64_t)(((kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                   dk + (uint64_t)(((kk >> 2) * C::KVBLK + (kk & 3) * 32) >> 4), id, kk > 0);
        mma_commit_w(bar(C::B_S + b));
        mma_commit_w(bar(C::B_KE + sl));
      }
      mma_commit_w(bar(C::B_DRAIN));
      drain_wait(bar(C::B_DRAIN), 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ O += P V
    if (hi > lo) {
      const uint32_t id = idesc_f16(is_bf16, 128, C::NPAD, 0, 1);  // V is MN-major
      const uint64_t dv0 = sdesc_sw128(sV, C::KVBLK, 1024);
      bool ok = true;
      for (int n = 0; n < hi - lo && ok; ++n) {
        const int b = n & 1, sl = n % C::NV, j = lo + n;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_VF + sl), (n / C::NV) & 1, abort_flag, p.err));
        if (!ok) break;
        const int have = end_of(j) - key_of(j);
        if (j >= pl.np && have < kBN) {
          // the rows behind the sequence's last key: zero
          for (int c = 0; c < C::KB; ++c) {
            const uint32_t a = sV + sl * C::T_BYTES + c * C::KVBLK;
            for (int x = have * 128 + lane * 16; x < kBN * 128; x += 512) sts_v4(a + x, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_P + b), (n >> 1) & 1, abort_flag, p.err));
        if (!ok) break;
        fence_after();
        const uint64_t dv = dv0 + (uint64_t)((sl * C::T_BYTES) >> 4);
        // (two loops: with a choice in each step the common one's operands left the uniform registers,
        // 545 us where prefix extensions take 530)
        if (quad) {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts_quarter_w(tmem + C::O_COL, tmem + 64 * b + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id,
                             n > 0 ? 1u : 0u, kk);
        } else {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts_w(tmem + C::O_COL, tmem + 64 * b + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id,
                     (n > 0 || kk > 0) ? 1u : 0u);
        }
        mma_commit_w(bar(C::B_O + b));
        mma_commit_w(bar(C::B_VE + sl));
      }
      mma_commit_w(bar(C::B_DRAIN + 1));
      drain_wait(bar(C::B_DRAIN + 1), 0);
    }
  } else if (warp >= 4 && warp - 4 < live_warps) {
    // ------------------------------------------------------------------ softmax / epilogue
    const int quarter = warp & 3, r = quad ? lane : 32 * quarter + lane, tok = r / pl.gb;
    const int head = h0 + r % pl.gb, grow = row0 + tok;
    bool row_ok = tok < nrows;
    int vlo = 0, vhi = 0;  // this row's visible keys
    if (pre) {
      const int s = seq_of[row_ok ? tok : 0];
      row_ok = row_ok && s != 0xffff;
      if (row_ok) {
        const int q0 = ld(p.cu_q + s), ql = ld(p.cu_q + s + 1) - q0;
        const int ks = P + ld(p.cu_kv + s + 1) - ld(p.cu_kv + s);
        visible_range(grow - q0, ks - ql, ks, p.causal, p.window, vlo, vhi);
      }
    } else if (row_ok) {
      visible_range(grow - sq.q0, off, keys, p.causal, p.window, vlo, vhi);
    }
    const uint32_t s_addr = tmem + ((uint32_t)(32 * quarter) << 16), o_addr = s_addr + C::O_COL;
    const float sl2 = p.scale_log2;
    // l: sum of the rounded P that the MMA multiplies (normalises O); lf: the fp32 sum (LSE)
    float m_ref = -INFINITY, l = 0.f, lf = 0.f;
    const int nt = hi - lo;
    bool ok = true;
    for (int n = 0; quad && n < nt; ++n) {
      // quarter tiles: columns c0 ... c0 + 15
      const int j = lo + n, b = n & 1, c0 = 16 * quarter;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S + b), (n >> 1) & 1, abort_flag, p.err));
      if (!ok) break;
      fence_after();
      const uint32_t sb = s_addr + 64 * b;
      const int kb = key_of(j) + c0, elo = vlo - kb, ehi = min(vhi, end_of(j)) - kb;
      uint32_t v[16];
      __syncwarp();
      tmem_ld16(sb + c0, v);
      tmem_ld_wait();
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = e >= elo && e < ehi ? __uint_as_float(v[e]) * sl2 : -INFINITY;
        v[e] = __float_as_uint(x);
        mx = fmaxf(mx, x);
      }
      const float m_new = fmaxf(m_ref, mx);
      const bool move = m_new != -INFINITY && m_new > m_ref + kMoveMax;
      const float alpha = move ? ex2(m_ref - m_new) : 1.f;  // m_ref = -inf: 0
      if (__any_sync(0xffffffffu, move && n > 0 && l > 0.f)) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag, p.err));
        if (!ok) break;
        fence_after();
        const float a = l > 0.f ? alpha : 1.f;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(o_addr + ch * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st32(o_addr + ch * 32, o);
        }
      }
      if (move) {
        l *= alpha;
        lf *= alpha;
        m_ref = m_new;
      }
      const float m0 = m_ref == -INFINITY ? 0.f : m_ref;
      uint32_t pk[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float pa = ex2(__uint_as_float(v[2 * e]) - m0), pb = ex2(__uint_as_float(v[2 * e + 1]) - m0);
        pk[e] = pack2(pa, pb, is_bf16);
        lf += pa + pb;
        l = add_halves(l, pk[e], is_bf16);
      }
      __syncwarp();
      tmem_st8(sb + 8 * quarter, pk);  // (this quarter's product reads these columns alone)
      tmem_st_wait();
      fence_before();
      mbar_arrive(bar(C::B_P + b));
    }
    for (int n = 0; !quad && n < nt; ++n) {
      const int j = lo + n, b = n & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S + b), (n >> 1) & 1, abort_flag, p.err));
      if (!ok) break;
      fence_after();
      const uint32_t sb = s_addr + 64 * b;
      const int kb = key_of(j), elo = vlo - kb, ehi = min(vhi, end_of(j)) - kb;
      const bool full = elo <= 0 && ehi >= kBN;
      uint32_t v[kBN];
      __syncwarp();
      tmem_ld32_at(sb + 0, v, 0);
      tmem_ld32_at(sb + 32, v, 32);
      tmem_ld_wait();
      // P = 2^(logit2 - m_ref), two at a time, in 16 bits over the S buffer's first 32 columns, with
      // the fp32 sum and the sum of the rounded P
      float sumr = 0.f, lsum = 0.f;
      auto exp_pass = [&](float scale, float neg_m) {
        const uint64_t scale2 = f2pack(scale, scale), negm2 = f2pack(neg_m, neg_m);
        uint64_t sf0 = f2pack(0.f, 0.f), sf1 = sf0;
        float sr0 = 0.f, sr1 = 0.f;
#pragma unroll
        for (int ch = 0; ch < kBN / 32; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 32 * ch + 2 * e;
            const float2 x = f2unpack(fma2(f2pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), scale2, negm2));
            const float pa = ex2(x.x), pb = ex2(x.y);
            pk[e] = pack2(pa, pb, is_bf16);
            if (e & 1) {
              sf1 = add2(sf1, f2pack(pa, pb));
              sr1 = add_halves(sr1, pk[e], is_bf16);
            } else {
              sf0 = add2(sf0, f2pack(pa, pb));
              sr0 = add_halves(sr0, pk[e], is_bf16);
            }
          }
          __syncwarp();
          tmem_st16(sb + ch * 16, pk);
        }
        const float2 f0 = f2unpack(sf0), f1 = f2unpack(sf1);
        lsum = (f0.x + f0.y) + (f1.x + f1.y);
        sumr = sr0 + sr1;
      };
      auto row_max = [&]() {
        float m8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float *f = reinterpret_cast<const float *>(v) + 8 * q;
          m8[q] = fmax3(fmax3(f[0], f[1], f[2]), fmax3(f[3], f[4], f[5]), fmaxf(f[6], f[7]));
        }
        return fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
      };
      // Unmasked tile and a reference max in every row of the warp: P with that reference, the row
      // max beside it; only a max beyond the threshold goes through the general pass.  (Lanes that hold
      // no row, the last two or three with groups of 3, 5, 6 or 7 heads, have neither: their warp takes
      // the general pass on every tile.)
      bool done = false;
      if (__all_sync(0xffffffffu, full && m_ref != -INFINITY)) {
        exp_pass(sl2, -m_ref);
        done = !__any_sync(0xffffffffu, row_max() * sl2 > m_ref + kMoveMax);
        if (!done) tmem_st_wait();  // (the general pass rewrites P)
      }
      if (!done) {
        float mx;
        if (full) {
          mx = row_max() * sl2;
        } else {
          mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < kBN; ++e) {
            const float x = e >= elo && e < ehi ? __uint_as_float(v[e]) * sl2 : -INFINITY;
            v[e] = __float_as_uint(x);
            mx = fmaxf(mx, x);
          }
        }
        const float m_new = fmaxf(m_ref, mx);
        float alpha = 1.f;
        const bool move = m_new != -INFINITY && m_new > m_ref + kMoveMax;
        if (move) alpha = ex2(m_ref - m_new);  // m_ref = -inf: 0
        const bool need = move && n > 0 && l > 0.f;
        if (__any_sync(0xffffffffu, need)) {
          // O is rescaled once the product before (so every earlier one) has completed
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag, p.err));
          if (!ok) break;
          fence_after();
          const float a = need ? alpha : 1.f;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld32(o_addr + ch * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st32(o_addr + ch * 32, o);
          }
        }
        if (move) {
          l *= alpha;
          lf *= alpha;
          m_ref = m_new;
        }
        exp_pass(full ? sl2 : 1.f, m_ref == -INFINITY ? 0.f : -m_ref);
      }
      l += sumr;
      lf += lsum;
      __syncwarp();
      tmem_st_wait();
      fence_before();
      mbar_arrive(bar(C::B_P + b));
    }
    if (ok && nt > 0) ok = mbar_wait(bar(C::B_O + ((nt - 1) & 1)), ((nt - 1) >> 1) & 1, abort_flag, p.err);
    ok = __all_sync(0xffffffffu, ok);
    if (quad) {
      // Join the quarters.  Weights f_w = 2^(m_w - max m); the sums by them, and O in runs of 32
      // columns through shared memory (the K ring: every product has completed): thread t sums columns
      // of row t / 4.  (All four warps come here, also after a wait that gave up.)
      constexpr int LD = 36;  // floats per row: 16-byte rows, banks apart
      float *buf = reinterpret_cast<float *>(smem_raw + C::OFF_K), *st = buf + 128 * LD;  // st [4][32][3]
      fence_after();
      const int tid = 32 * quarter + lane;
      st[3 * tid] = m_ref;
      st[3 * tid + 1] = l;
      st[3 * tid + 2] = lf;
      named_sync(1, 128);
      const int jr = tid >> 2, jt = jr / pl.gb;  // row and columns that this thread writes
      const size_t at = (size_t)(row0 + jt) * p.h_q + h0 + jr % pl.gb;
      float m = -INFINITY, f[4], ls = 0.f, lfs = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) m = fmaxf(m, st[3 * (32 * x + jr)]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float *q = st + 3 * (32 * x + jr);
        f[x] = m == -INFINITY ? 0.f : ex2(q[0] - m);
        ls = fmaf(f[x], q[1], ls);
        lfs = fmaf(f[x], q[2], lfs);
      }
      const float inv = ls == 0.f ? 0.f : 1.f / ls;  // (a NaN logit leaves a NaN sum, and a NaN row)
      const bool wr = ok && jt < nrows;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t v[32];
        if (nt > 0) {
          __syncwarp();
          tmem_ld32(o_addr + ch * 32, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        // (rows of nobody hold whatever the tile held; they are not summed)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4 *>(buf + tid * LD + 4 * q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        named_sync(1, 128);
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!(f[x] > 0.f)) continue;
          const float *q = buf + (32 * x + jr) * LD + 8 * (tid & 3);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(f[x], q[e], o[e]);
        }
        named_sync(1, 128);
        if (!wr) continue;
        const int c = 32 * ch + 8 * (tid & 3);
        if (SPLIT) {
          float4 *dst = reinterpret_cast<float4 *>(o_part + ((size_t)slot * p.total_q * p.h_q + at) * D + c);
          dst[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
          dst[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
        } else {
          *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + (at * D + c) * 2) =
              make_uint4(pack2(o[0] * inv, o[1] * inv, is_bf16), pack2(o[2] * inv, o[3] * inv, is_bf16),
                         pack2(o[4] * inv, o[5] * inv, is_bf16), pack2(o[6] * inv, o[7] * inv, is_bf16));
        }
      }
      if (wr && (tid & 3) == 0) {
        const float lse = lfs == 0.f ? -INFINITY : (m + lg2(lfs)) * kLn2f;
        if (SPLIT) lse_part[(size_t)slot * p.total_q * p.h_q + at] = lse;
        else if (p.lse) p.lse[(size_t)(h0 + jr % pl.gb) * p.total_q + row0 + jt] = lse;
      }
    } else if (ok) {
      fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = lf == 0.f ? -INFINITY : (m_ref + lg2(lf)) * kLn2f;
      const size_t at = (size_t)grow * p.h_q + head;  // (row, head)
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t v[32];
        if (nt > 0) {
          __syncwarp();
          tmem_ld32(o_addr + ch * 32, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if (!row_ok) continue;
        if (SPLIT) {
          float4 *dst = reinterpret_cast<float4 *>(o_part + ((size_t)slot * p.total_q * p.h_q + at) * D) + ch * 8;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(__uint_as_float(v[4 * q]) * inv, __uint_as_float(v[4 * q + 1]) * inv,
                                 __uint_as_float(v[4 * q + 2]) * inv, __uint_as_float(v[4 * q + 3]) * inv);
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + at * D * 2) + ch * 4;
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = pack2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv, is_bf16);
#pragma unroll
          for (int q = 0; q < 4; ++q) dst[q] = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
        }
      }
      if (row_ok) {
        if (SPLIT) lse_part[(size_t)slot * p.total_q * p.h_q + at] = lse;
        else if (p.lse) p.lse[(size_t)head * p.total_q + grow] = lse;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merges the parts: LSE = log sum_s exp(L_s), O = sum_s exp(L_s - LSE) O_s.  A warp per (row, head);
// a lane holds four columns of a part (width 64: half a warp per part), the weights sit in the lanes.
// Rows of no sequence are left alone.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const Params p, int parts, const float *o_part,
                                                           const float *lse_part) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  pdl_trigger();
  pdl_wait();
  const size_t pairs = (size_t)p.total_q * p.h_q;
  const size_t w = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= pairs || w / p.h_q >= (size_t)max(0, ld(p.cu_q + p.num_seqs))) return;
  constexpr int NL = D / 4;                // lanes per part
  constexpr int PER = NL <= 16 ? 2 : 1;    // parts at a time
  constexpr int FLY = 12;                  // their loads in flight, together with the log-sum-exps'
  const int sub = PER == 2 ? lane >> 4 : 0, c = PER == 2 ? lane & 15 : lane;
  auto fetch = [&](int s0, float4 (&x)[FLY]) {
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int s = s0 + i * PER + sub;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < parts && c < NL) x[i] = *reinterpret_cast<const float4 *>(o_part + (s * pairs + w) * D + 4 * c);
    }
  };
  float4 x[FLY];
  fetch(0, x);
  // (64 parts at most: two per lane)
  const float l0 = lane < parts ? lse_part[lane * pairs + w] : -INFINITY;
  const float l1 = 32 + lane < parts ? lse_part[(32 + lane) * pairs + w] : -INFINITY;
  float m = fmaxf(l0, l1);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mm = m == -INFINITY ? 0.f : m;
  const float e0 = expf(l0 - mm), e1 = expf(l1 - mm);
  float sum = e0 + e1;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += FLY * PER) {
    if (s0 > 0) fetch(s0, x);
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int s = s0 + i * PER + sub;
      const float wa = __shfl_sync(0xffffffffu, e0, s & 31), wb = __shfl_sync(0xffffffffu, e1, s & 31);
      const float wgt = s < 32 ? wa : wb;
      if (s >= parts || wgt == 0.f) continue;  // (a NaN weight stays)
      acc.x = fmaf(wgt, x[i].x, acc.x);
      acc.y = fmaf(wgt, x[i].y, acc.y);
      acc.z = fmaf(wgt, x[i].z, acc.z);
      acc.w = fmaf(wgt, x[i].w, acc.w);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (PER == 2) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (c < NL && sub == 0) {
    T y[4] = {from_f32<T>(acc.x * inv), from_f32<T>(acc.y * inv), from_f32<T>(acc.z * inv), from_f32<T>(acc.w * inv)};
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + w * D + 4 * c) = *reinterpret_cast<uint2 *>(y);
  }
  if (lane == 0 && p.lse)
    p.lse[(w % p.h_q) * p.total_q + w / p.h_q] = sum == 0.f ? -INFINITY : mm + logf(sum);
}

bool tc_shape(int d_qk, int d_v, int dtype, unsigned flags) {
  return (dtype == VLF_F16 || dtype == VLF_BF16) && !(flags & VLF_FLAG_FORCE_SIMT) && d_qk == d_v &&
         (d_qk == 64 || d_qk == 96 || d_qk == 128);
}

// How the work is cut, by sizes alone (the lengths are on the device: every sequence counts with the
// longest length, so that a loose bound or one long sequence makes fewer prefix parts, or none: the 64
// decode rows below get 6 of them with a bound of 1024 own keys, 3 with 4096, no shared part with 16384).
// Costs in tenths of a
// microsecond: a key tile takes a CTA about 1 us whatever else runs (10; 4 with quarter tiles), the
// busiest of the resident CTA slots (two per SM) sets the time, and merging costs a launch and the
// traffic of the parts (30 and 1 per 0.6 MB).
//  * per sequence: row tiles walk the prefix and their own keys; cut into parts, four tiles each at
//    least, where the row tiles leave slots empty;
//  * shared: the batch's rows packed against the prefix, and the own keys apart, in parts of what a
//    slot gets where that is one wave of CTAs, else of twice that: the own keys' CTAs fill up beside
//    and behind them, and fewer parts cost less to write and merge (64 decode rows, 16k shared keys:
//    50 us; 53, 54, 58 us with runs of 1.5, 1 and 0.75 times a slot's share, 54 and 58 us with 2.5 and
//    3).  Taken where it saves a fifth.
PfxPlan make_plan(int num_seqs, int total_q, int max_q, int max_kv, int prefix, int h_q, int h_kv, int d, int num_sms) {
  constexpr long long kTile = 10, kQuad = 4, kMerge = 30;
  PfxPlan pl{};
  const int group = h_q / h_kv;
  pl.gb = std::min(group, 128);
  while (group % pl.gb) --pl.gb;
  pl.nhb = group / pl.gb;
  pl.quad_pre = (long long)total_q * pl.gb <= 32;
  pl.rows = (pl.quad_pre ? 32 : 128) / pl.gb;
  pl.quad = (long long)max_q * pl.gb <= 32;
  pl.rows_own = (pl.quad ? 32 : 128) / pl.gb;
  pl.heads = h_kv * pl.nhb;
  pl.np = (prefix + kBN - 1) / kBN;
  const long long no = ((long long)max_kv + kBN - 1) / kBN, slots = 2ll * num_sms;
  pl.rb_own = (max_q + pl.rows_own - 1) / pl.rows_own;
  pl.rb_pre = (total_q + pl.rows - 1) / pl.rows;
  // row tiles of the sequences one by one, as far as the sizes tell
  const long long own_tiles =
      std::min((long long)num_seqs * pl.rb_own, (long long)(total_q + pl.rows_own - 1) / pl.rows_own + num_seqs);
  const long long own = std::max(1ll, own_tiles * pl.heads), pre = (long long)pl.rb_pre * pl.heads;
  const long long tile = pl.quad ? kQuad : kTile, tile_pre = pl.quad_pre ? kQuad : kTile;
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  auto merge = [&](long long parts) { return kMerge + parts * total_q * h_q * d * 8 / 600000; };
  const long long all = pl.np + no;
  const long long cut = std::max(1ll, std::min({slots / own, all / 4, 64ll}));
  const long long whole = std::max(own * all / slots, all) * tile, in_parts = up(all, cut) * tile + merge(cut);
  const long long work = pre * pl.np * tile_pre + own * no * tile;  // of the shared cut
  long long run;
  int parts_pre, parts_own;
  auto cut_shared = [&](long long share) {
    run = std::max(4 * std::min(tile, tile_pre), share);
    parts_pre = (int)std::min(up(pl.np * tile_pre, run), 48ll);
    parts_own = (int)std::max(1ll, std::min(up(no * tile, run), 16ll));
  };
  cut_shared(work / slots);
  if (pre * parts_pre + own * parts_own > slots) cut_shared(2 * work / slots);
  pl.parts_own = cut > 1 && in_parts < whole ? (int)cut : 1;
  const long long apart = std::max(work / slots, run) + merge(parts_pre + parts_own);
  pl.shared = pl.np > 0 && apart * 5 < (pl.parts_own > 1 ? in_parts : whole) * 4;
  pl.parts_pre = pl.shared ? parts_pre : 0;
  if (pl.shared) pl.parts_own = parts_own;
  pl.parts = pl.parts_pre + pl.parts_own;
  if (pl.parts == 1) pl.parts = 0;
  const long long n_pre = pre * pl.parts_pre, n_own = (long long)num_seqs * pl.heads * pl.rb_own * pl.parts_own;
  pl.n_pre = (unsigned)n_pre;
  pl.n_all = n_pre + n_own <= 0x7fffffffll ? (unsigned)(n_pre + n_own) : 0u;
  return pl;
}

size_t parts_bytes(const PfxPlan &pl, int total_q, int h_q, int d) {
  const size_t pairs = (size_t)pl.parts * total_q * h_q;
  return ((pairs * d * sizeof(float) + 255) & ~(size_t)255) + ((pairs * sizeof(float) + 255) & ~(size_t)255);
}

template <int D>
cudaError_t launch_tc(const PrefixParams &pp, PfxPlan pl, void *workspace, cudaStream_t st) {
  const Params &p = pp.p;
  using C = PfxCfg<D>;
  PfxMaps maps;
  const int bf = p.dtype == VLF_BF16;
  const uint64_t kc = (uint64_t)p.h_kv * D;
  const bool have_p = pp.prefix_len > 0, have_o = p.total_kv > 0;
  if (!make_tmap_q3(&maps.q, p.q, p.total_q, p.h_q, D, pl.gb, pl.rows, bf) ||
      !make_tmap_q3(&maps.q_own, p.q, p.total_q, p.h_q, D, pl.gb, pl.rows_own, bf))
    return cudaErrorInvalidValue;
  if (have_p && (!make_tmap_16bit(&maps.kp, pp.k_pre, pp.prefix_len, kc, kc, kBN, bf) ||
                 !make_tmap_16bit(&maps.vp, pp.v_pre, pp.prefix_len, kc, kc, kBN, bf)))
    return cudaErrorInvalidValue;
  if (have_o && (!make_tmap_16bit(&maps.k, p.k, p.total_kv, kc, kc, kBN, bf) ||
                 !make_tmap_16bit(&maps.v, p.v, p.total_kv, kc, kc, kBN, bf)))
    return cudaErrorInvalidValue;
  if (!have_p) { maps.kp = maps.k; maps.vp = maps.v; }  // (never read: no tile comes from it)
  if (!have_o) { maps.k = maps.kp; maps.v = maps.vp; }
  float *o_part = nullptr, *lse_part = nullptr;
  if (pl.parts) {
    o_part = static_cast<float *>(workspace);
    lse_part = reinterpret_cast<float *>(
        static_cast<uint8_t *>(workspace) +
        (((size_t)pl.parts * p.total_q * p.h_q * D * sizeof(float) + 255) & ~(size_t)255));
  }
  const void *kern = pl.parts ? (bf ? (const void *)tc_prefix_kernel<D, true, true>
                                    : (const void *)tc_prefix_kernel<D, false, true>)
                              : (bf ? (const void *)tc_prefix_kernel<D, true, false>
                                    : (const void *)tc_prefix_kernel<D, false, false>);
  cudaError_t e = set_smem_once(kern, C::SMEM);
  if (e != cudaSuccess) return e;
  PrefixParams a = pp;
  void *args[5] = {&maps, &a, &pl, &o_part, &lse_part};
  e = launch_kernel(kern, dim3(pl.n_all), 256, C::SMEM, st, args);
  if (e != cudaSuccess) return e;
  count_launch();
  if (pl.parts) {
    Params pm = p;
    void *margs[4] = {&pm, &pl.parts, &o_part, &lse_part};
    const size_t blocks = ((size_t)p.total_q * p.h_q + 7) / 8;
    e = launch_dependent(bf ? (const void *)prefix_merge_kernel<D, true> : (const void *)prefix_merge_kernel<D, false>,
                         dim3((unsigned)blocks), 256, 0, st, margs);
    if (e == cudaSuccess) count_launch();
  }
  return e;
}

}  // namespace

size_t prefix_workspace(int num_seqs, int total_q, int max_q, int max_kv, int prefix, int h_q, int h_kv, int d_qk,
                        int d_v, int dtype, unsigned flags, int num_sms) {
  if (num_seqs < 1 || total_q < 1 || max_q < 1 || max_kv < 0 || prefix < 0 || h_kv < 1 || h_q < 1 || h_q % h_kv ||
      num_sms < 1 || !tc_shape(d_qk, d_v, dtype, flags))
    return 0;
  const PfxPlan pl = make_plan(num_seqs, total_q, max_q, max_kv, prefix, h_q, h_kv, d_v, num_sms);
  return pl.parts ? parts_bytes(pl, total_q, h_q, d_v) : 0;
}

cudaError_t prefix_forward(const PrefixParams &pp, void *workspace, int num_sms, cudaStream_t st) {
  const Params &p = pp.p;
  // (without rows or keys there is nothing to stage)
  if (!tc_shape(p.d_qk, p.d_v, p.dtype, p.flags) || p.total_q == 0 || (p.total_kv == 0 && pp.prefix_len == 0))
    return simt_prefix(pp, st);
  const PfxPlan pl = make_plan(p.num_seqs, p.total_q, p.max_q, p.max_kv, pp.prefix_len, p.h_q, p.h_kv, p.d_v, num_sms);
  if (pl.n_all == 0) return cudaErrorInvalidValue;
  if (p.d_qk == 64) return launch_tc<64>(pp, pl, workspace, st);
  if (p.d_qk == 96) return launch_tc<96>(pp, pl, workspace, st);
  return launch_tc<128>(pp, pl, workspace, st);
}

}  // namespace vlf
