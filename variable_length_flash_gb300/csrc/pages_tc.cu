// Attention over pages in e4m3 on the tensor cores (16-bit queries, widths 64 and 128).
//
// The bytes are multiplied as they are: both products are tcgen05 kind::f8f6f4, with the page as operand A
// from shared memory, where TMA puts it, and nothing is converted.  Keys are the rows of a tile:
//     S^T[key, column] = sum_c K[key, c] Q[column, c],       O^T[c, column] += sum_key V[key, c] P[key, column],
// 128 keys a tile; a column is one query row of one head of the kv head's group.  So each of the 128
// softmax threads has a key, whose scale (its page's) is one number of its, and a step with few
// columns, a decode step's four or eight, still has 128 threads to share its exponentials.
//
// Eight bits are not enough for Q and P; each is a sum of several numbers of eight bits, exact enough:
//  * Q, brought to [128, 256) by a power of two for each column, as two e4m3 terms (bf16) or three (fp16):
//    x = t0 + t1 + t2, each the rest's nearest e4m3.  A term holds 4 bits and a sign, so bf16's 8 and fp16's
//    11 bits are exact down to where the last term meets e4m3's least step, 2^-18 of the column's largest.
//  * P, as three e5m2 terms: 3 bits each and two signs are 11 bits, half a step of fp16; the first term is
//    the high byte of P in fp16.  e5m2 reaches from 2^-16 to 57344: with the column's largest P between 2^7 and
//    2^15, what a key loses is below 2^-24 of the largest weight.  (Two e4m3 terms hold 9 bits, but reach
//    down to 2^-18 only: a long tail of small weights behind one large one would vanish.)
// The terms of Q are added by the accumulator; those of P are columns of their own, added at the end: the
// matrix pipe reads each byte of V once for all of them.
//
// A key's scale multiplies its logits.  A value's scale goes into the exponent, P = 2^(logit + log2 scale -
// reference), so that the reference follows the weights as they meet the values; the sum of the weights
// takes P / scale.  The reference of a column moves when a P would pass 2^15 (a vote of the 128 threads on
// each tile), and O is rescaled then.
//
// Work is cut evenly, whatever the lengths: the (sequence, kv head, query tile) items' key tiles, laid end to
// end, are shared out to the resident CTAs in equal runs.  A run that holds a whole item writes it; one that
// starts or ends inside an item leaves its part (two at most), which a second launch joins.  Loads run on
// across items, so nothing starts or drains but at the two ends.  Nothing about the lengths is needed on the
// host, and a loose bound costs nothing.
//
// Roles of a CTA: warps 0-3 softmax (thread = key) and the output (thread = column of V), warp 4 page loads,
// warp 5 both products.
//
// Bound: HBM, each byte of the cache read once.  64 single rows on caches of 1000 to 16384 keys, 32 heads over 8 of
// 128: 180 us (93% of the copy rate), 181 with pages of 16 tokens, 192 with groups of 8 heads, 227 with 4 rows
// a sequence; width 64 in fp16 107 us (79%: a tile's softmax steps take longer than its bytes then, and the CTAs'
// roles fetch instructions past the cache); one cache of 131071 keys 56 us (71%: 40 us of bytes, the
// ends of the runs and the join).  Three short caches 10.7 us, which is latency.
#include "e4m3.cuh"
#include "pages_tc.cuh"

namespace vlf {
namespace {

using namespace pages;

constexpr int kKeys = 128;         // keys of a tile
constexpr float kNoRef = -1e30f;   // reference of a column that has met no key
constexpr float kTop = 15.f;       // log2 of the largest P
constexpr float kSet = 7.f;        // log2 of the largest P when the reference is set
constexpr int kScales = 8;         // tiles whose scales are held (more than the rings let loads run ahead)

// NC: columns of a tile.
template <int D, int NC> struct Cfg {
  static constexpr int NS = NC < 16 ? 16 : NC;              // columns of S (the least N of the product)
  static constexpr int NP = (3 * NC + 15) / 16 * 16;        // columns of P and O: three terms
  static constexpr int T_BYTES = kKeys * D;
  static constexpr int KST = 3, VST = D == 128 && NC >= 32 ? 2 : 3;
  static constexpr int PB = NC >= 16 ? 1 : 2;               // buffers of P
  static constexpr int Q_TERM = NS * D, P_BYTES = NP * kKeys;
  static constexpr int OFF_K = 0, OFF_V = OFF_K + KST * T_BYTES, OFF_Q = OFF_V + VST * T_BYTES, OFF_P = OFF_Q + 3 * Q_TERM;
  static constexpr int OFF_COL = OFF_P + PB * P_BYTES;      // float2 (scale, -reference)[2][NC]
  static constexpr int OFF_LIM = OFF_COL + 2 * NC * 8;      // int2 (first, end)[2][NC]
  static constexpr int OFF_WM = OFF_LIM + 2 * NC * 8;       // float[4][NC]
  static constexpr int OFF_FAC = OFF_WM + 4 * NC * 4;       // float[NC]
  static constexpr int OFF_SC = OFF_FAC + NC * 4;           // float2 (k, v scale)[kScales][8]
  static constexpr int OFF_RED = OFF_SC + kScales * 8 * 8;  // long long[8]
  static constexpr int OFF_BAR = OFF_RED + 64;
  static constexpr int B_KF = 0, B_KE = B_KF + KST, B_VF = B_KE + KST, B_VE = B_VF + VST, B_SF = B_VE + VST, B_SE = B_SF + 2,
                       B_PF = B_SE + 2, B_PE = B_PF + PB, B_Q = B_PE + PB, B_OF = B_Q + 1, B_OE = B_OF + 1, B_SC = B_OE + 1,
                       B_DRAIN = B_SC + kScales, BARS = B_DRAIN + 1;
  static constexpr int OFF_END = OFF_BAR + BARS * 8 + 16;   // then the TMEM address and the abort flag
  static constexpr int SMEM = OFF_END + 1024;               // (to start on 1024 bytes)
  static constexpr int O_COL = 2 * NS;
  static constexpr int TMEM = O_COL + NP <= 64 ? 64 : O_COL + NP <= 128 ? 128 : 256;
  // resident CTAs per SM: by shared memory (227 KB) and TMEM (512 columns)
  static constexpr int CTAS = (227 * 1024) / (SMEM + 1024) < 512 / TMEM ? (227 * 1024) / (SMEM + 1024) : 512 / TMEM;
  static constexpr int PART = NC * (D + 2);                 // floats of a part
};

__device__ __forceinline__ uint32_t idesc_f8(uint32_t b_type, uint32_t n, uint32_t mn) {
  // D fp32; A e4m3 (0), B e4m3 (0) or e5m2 (1); both K-major or both MN-major; M = 128
  return (1u << 4) | (b_type << 10) | (mn << 15) | (mn << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
// Shared-memory descriptor with a swizzle code (0 none, 2 128 bytes, 4 64 bytes).
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 |
         (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}
__device__ __forceinline__ void mma_f8_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Barrier of the 128 softmax threads; whether any of them says x.
__device__ __forceinline__ bool any_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// NC columns.
template <int NC> __device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[NC]) {
  if constexpr (NC <= 16) {
    tmem_ld<NC>(taddr, r);
  } else {
#pragma unroll
    for (int i = 0; i < NC; i += 16) tmem_ld<16>(taddr + i, r + i);
  }
}

template <int D, int NC, bool BF16>
__global__ void __launch_bounds__(192, Cfg<D, NC>::CTAS)
    pages_tc_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                    const __grid_constant__ TcParams p) {
  using C = Cfg<D, NC>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int QT = BF16 ? 2 : 3;  // terms of Q
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t base = (smem_u32(smem_dyn) + 1023u) & ~1023u;
  uint8_t *const smem = smem_dyn + (base - smem_u32(smem_dyn));
  const uint32_t sK = base + C::OFF_K, sV = base + C::OFF_V, sQ = base + C::OFF_Q, sP = base + C::OFF_P;
  float2 *const col = reinterpret_cast<float2 *>(smem + C::OFF_COL);
  int2 *const lim = reinterpret_cast<int2 *>(smem + C::OFF_LIM);
  float *const wm = reinterpret_cast<float *>(smem + C::OFF_WM), *const fac = reinterpret_cast<float *>(smem + C::OFF_FAC);
  float2 *const scales = reinterpret_cast<float2 *>(smem + C::OFF_SC);
  long long *const red = reinterpret_cast<long long *>(smem + C::OFF_RED);
  auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
  uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + C::BARS * 8);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Params &b = p.a.p;
  int *const err = b.err;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KST; ++i) { mbar_init(bar(C::B_KF + i), 1); mbar_init(bar(C::B_KE + i), 1); }
    for (int i = 0; i < C::VST; ++i) { mbar_init(bar(C::B_VF + i), 1); mbar_init(bar(C::B_VE + i), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(bar(C::B_SF + i), 1); mbar_init(bar(C::B_SE + i), 128); }
    for (int i = 0; i < C::PB; ++i) { mbar_init(bar(C::B_PF + i), 128); mbar_init(bar(C::B_PE + i), 1); }
    mbar_init(bar(C::B_Q), 128);
    mbar_init(bar(C::B_OF), 1);
    mbar_init(bar(C::B_OE), 128);
    for (int i = 0; i < kScales; ++i) mbar_init(bar(C::B_SC + i), 1);
    mbar_init(bar(C::B_DRAIN), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  pdl_wait();
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM);
    tmem_relinquish();
  }

  const Run run = run_of<kKeys, 192>(p, red);
  Walk<kKeys> w(p);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_holder;

  if (!run.any) {
    if (threadIdx.x == 0) no_item(p);
  } else if (warp == 4) {
    // ------------------------------------------------------------------ pages
    int off = w.seek(run.seq, run.unit);
    const int page = min(p.a.page, kKeys), npt = kKeys / page;  // slots and pages of a tile
    const int log2_page = p.a.log2_page, none = p.a.num_pages * b.h_kv;
    bool ok = true;
    long long left = run.f1 - run.f0;
    int nk = 0, nv = 0;
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        const int j0 = (w.t0 + off) * kKeys, first = j0 >> log2_page;  // the first page of the run's tiles
        const int last = (min(w.hi, j0 + n * kKeys) - 1) >> log2_page;
        const int32_t *row = p.a.table + (long long)w.s * p.a.max_pages;
        // a lane has a page of the next 32, and one of the 32 behind them
        auto id_of = [&](int i) {
          if (i > last || i < w.lo >> log2_page) return -2;  // no key of the run's in it
          return max(ld(row + i), -1);
        };
        auto real = [&](int id) { return id >= 0 && id < p.a.num_pages; };
        int id = id_of(first + lane), id_next = id_of(first + 32 + lane);
        auto scale_of = [&](int i) {
          if (!real(i)) return make_float2(0.f, -1.f);  // (keys of no weight, below)
          const long long at = (long long)i * b.h_kv + w.head;
          return make_float2(ld(p.a.k_scale + at), ld(p.a.v_scale + at));
        };
        float2 sc = scale_of(id), sc_next = make_float2(0.f, 0.f);
        for (int m = 0; m < n && ok; ++m) {
          // page index of the tile's first page among the run's (a page of 256 has two tiles)
          const int at = ((j0 + m * kKeys) >> log2_page) - first, in = at % 32;
          if (in == 0 && m > 0 && ((j0 + m * kKeys) & (p.a.page - 1)) == 0) {
            id = id_next;
            sc = sc_next;
            id_next = id_of(first + at + 32 + lane);
          }
          if (in == 16) sc_next = scale_of(id_next);  // (every run of 32 pages has a tile that begins there)
          const int mine_id = __shfl_sync(0xffffffffu, id, in + lane % npt);
          const bool have = lane < npt && mine_id != -2;
          if (have && !real(mine_id)) set_error(err, VLF_ERR_BAD_PAGES);
          const int z = real(mine_id) ? mine_id * b.h_kv + w.head : none;  // (outside: zeros, so that nothing is a NaN)
          const int bytes = __popc(__ballot_sync(0xffffffffu, have)) * page * D;
          const int y = p.a.page > kKeys ? (j0 + m * kKeys) & (p.a.page - 1) : 0;
          const int ks = nk % C::KST, vs = nv % C::VST;
          if (nk >= C::KST) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_KE + ks), (nk / C::KST - 1) & 1, abort_flag, err));
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(C::B_KF + ks), bytes);
          __syncwarp();
          if (have) tma_load_3d(sK + ks * C::T_BYTES + lane * page * D, &k_map, 0, y, z, bar(C::B_KF + ks));
          const float2 mine_sc = make_float2(__shfl_sync(0xffffffffu, sc.x, in + lane % npt),
                                             __shfl_sync(0xffffffffu, sc.y, in + lane % npt));
          if (lane < npt) scales[nk % kScales * 8 + lane] = mine_sc;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_SC + nk % kScales));
          ++nk;
          if (nv >= C::VST) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_VE + vs), (nv / C::VST - 1) & 1, abort_flag, err));
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(C::B_VF + vs), bytes);
          __syncwarp();
          if (have) tma_load_3d(sV + vs * C::T_BYTES + lane * page * D, &v_map, 0, y, z, bar(C::B_VF + vs));
          ++nv;
        }
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0) {
      for (int i = 0; i < C::KST && i < nk; ++i) drain_wait(bar(C::B_KF + i), ((nk - 1 - i) / C::KST) & 1);
      for (int i = 0; i < C::VST && i < nv; ++i) drain_wait(bar(C::B_VF + i), ((nv - 1 - i) / C::VST) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------------ products
    int off = w.seek(run.seq, run.unit);
    const uint32_t id_s = idesc_f8(0, C::NS, 0), id_o = idesc_f8(1, C::NP, 1);
    constexpr uint32_t SW = D == 128 ? 2 : 4;
    // K and Q: rows of D bytes, eight to a swizzle atom.  V: 128 (64: twice the same 64) columns of a key in a
    // row, eight keys to an atom.  P: 16 columns of a key in 16 bytes, 128 keys, then the next 16 columns.
    const uint64_t dk0 = sdesc(sK, 16, 8 * D, SW), dq0 = sdesc(sQ, 16, 8 * D, SW), dv0 = sdesc(sV, 0, 8 * D, SW);
    const uint64_t dp0 = sdesc(sP, 128, 16 * kKeys, 0);
    bool ok = true;
    int ns = 0, np = 0, seg = 0;  // tiles of S and of O issued, items begun
    auto wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, abort_flag, err)); };
    auto issue_s = [&]() {
      const int ks = ns % C::KST, sb = ns & 1;
      ok = wait(C::B_KF + ks, ns / C::KST);
      if (ok && ns >= 2) ok = wait(C::B_SE + sb, ns / 2 - 1);
      if (!ok) return;
      fence_after();
      const uint64_t dk = dk0 + (uint64_t)((ks * C::T_BYTES) >> 4);
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_f8_w(tmem + C::NS * sb, dk + 2 * kk, dq0 + (uint64_t)((t * C::Q_TERM + 32 * kk) >> 4), id_s, t > 0 || kk > 0);
      mma_commit_w(bar(C::B_SF + sb));
      mma_commit_w(bar(C::B_KE + ks));
      ++ns;
    };
    long long left = run.f1 - run.f0;
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        ok = wait(C::B_Q, seg);
        if (ok) issue_s();
        for (int m = 0; m < n && ok; ++m) {
          if (m + 1 < n) issue_s();
          if (!ok) break;
          const int vs = np % C::VST, pb = np % C::PB;
          ok = wait(C::B_VF + vs, np / C::VST) && wait(C::B_PF + pb, np / C::PB);
          if (ok && m == 0 && seg > 0) ok = wait(C::B_OE, seg - 1);
          if (!ok) break;
          fence_after();
          const uint64_t dv = dv0 + (uint64_t)((vs * C::T_BYTES) >> 4), dp = dp0 + (uint64_t)((pb * C::P_BYTES) >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk)
            mma_f8_w(tmem + C::O_COL, dv + (uint64_t)((kk * 32 * D) >> 4), dp + (uint64_t)((kk * 512) >> 4), id_o, m > 0 || kk > 0);
          mma_commit_w(bar(C::B_VE + vs));
          mma_commit_w(bar(C::B_PE + pb));
          if (m + 1 == n) mma_commit_w(bar(C::B_OF));
          ++np;
        }
        ++seg;
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
    mma_commit_w(bar(C::B_DRAIN));
    drain_wait(bar(C::B_DRAIN), 0);
  } else if (warp < 4) {
    // ------------------------------------------------------------------ softmax / output
    const int tid = threadIdx.x;  // the key of a tile, or the column of V
    const uint32_t t_addr = tmem + ((uint32_t)(32 * warp) << 16);
    int off = w.seek(run.seq, run.unit);
    int seg = 0, ns = 0;  // items with tiles begun, tiles
    bool bad = false;     // a wait gave up (all four warps leave together)
    auto wait = [&](int i, int parity) {
      if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, abort_flag, err));
    };
    // The item's queries in terms, its columns' scales, references and limits.  A warp has every fourth column,
    // its lanes D / 32 elements each.
    auto prepare = [&](int par) {
      named_sync(1, 128);
      constexpr int E = D / 32, PER = C::NS / 4;
      uint32_t raw[PER][E / 2];  // (all loads in flight at once)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        int row = 0, head = 0;
        const int c = warp + 4 * i;
        const bool have = c < NC && column_of(p, NC, w, c, row, head);
        const T *q = static_cast<const T *>(b.q) + ((long long)(w.q0 + row) * b.h_q + head) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) raw[i][e] = have ? ld(reinterpret_cast<const uint32_t *>(q) + e) : 0;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        int row = 0, head = 0;
        const int c = warp + 4 * i;
        const bool have = c < NC && column_of(p, NC, w, c, row, head);
        float x[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 f = unpack2(raw[i][e / 2], BF16);
          x[e] = f.x;
          x[e + 1] = f.y;
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const bool odd = top >= 0x7f800000u;  // a query that is not finite: every logit of the row is NaN
        const int ex = min(max((int)(top >> 23) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23), down = __uint_as_float((uint32_t)(127 - 7 + ex) << 23);
        uint32_t word[3];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = odd ? 0.f : x[e] * up;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          word[t] = 0;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t two = e4m3x2(x[e], x[e + 1]);
            const float2 f = e4m3_pair(two);
            x[e] -= f.x;
            x[e + 1] -= f.y;
            word[t] |= two << 8 * e;
          }
          // row c: D bytes, 16-byte chunks swizzled by the row
          const int chunk = lane * E / 16, in = lane * E % 16;
          const uint32_t to = sQ + t * C::Q_TERM + c * D + ((D == 128 ? chunk ^ (c & 7) : chunk ^ (c >> 1 & 3)) << 4) + in;
          if constexpr (E == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(word[t]) : "memory");
          else asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"((uint16_t)word[t]) : "memory");
        }
        if (lane == 0 && c < NC) {
          const float nan = __uint_as_float(0x7fffffffu);
          // (a column of nobody: P = 0)
          col[par * NC + c] = make_float2(odd ? nan : down * b.scale_log2, have ? -kNoRef : kNoRef);
          int a = 0, e = 0;
          if (have) visible_range(row, w.len - w.q_len, w.len, b.causal, b.window, a, e);
          lim[par * NC + c] = make_int2(a, e);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::B_Q));
      named_sync(1, 128);
    };
    long long left = run.f1 - run.f0;
    while (left > 0 && !bad) {
      const int n = (int)min((long long)(w.units() - off), left), units = w.units();
      const bool whole = off == 0 && n == units;
      if (w.nt == 0) {
        // rows that see no key
        for (int c = 0; c < NC; ++c) {
          int row, head;
          if (!column_of(p, NC, w, c, row, head)) continue;
          const long long at = (long long)(w.q0 + row) * b.h_q + head;
          if (tid < D) static_cast<T *>(b.out)[at * D + tid] = from_f32<T>(0.f);
          if (tid == 0 && b.lse) b.lse[(long long)head * b.total_q + w.q0 + row] = -INFINITY;
        }
      } else {
        const int par = seg & 1;
        prepare(par);
        float l[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] = 0.f;
        // keys that every column sees
        int all_lo, all_hi, x;
        visible_range(w.r1 - 1, w.len - w.q_len, w.len, b.causal, b.window, all_lo, x);
        visible_range(w.r0, w.len - w.q_len, w.len, b.causal, b.window, x, all_hi);
        for (int m = 0; m < n; ++m, ++ns) {
          const int j0 = (w.t0 + off + m) * kKeys, j = j0 + tid;
          const int sb = ns & 1, pb = ns % C::PB, sc = ns % kScales;
          wait(C::B_SF + sb, ns / 2);
          wait(C::B_SC + sc, ns / kScales);
          uint32_t acc[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[c] = 0;
          if (!bad) {
            fence_after();
            __syncwarp();
            tmem_ld_cols<NC>(t_addr + C::NS * sb, acc);
            tmem_ld_wait();
            pin(acc);
            fence_before();
            mbar_arrive(bar(C::B_SE + sb));
          }
          const float2 s2 = scales[sc * 8 + (tid >> min(p.a.log2_page, 7))];
          const float vs = fminf(fmaxf(s2.y, 0x1p-100f), 0x1p120f);  // (a scale of zero or no number: of no weight)
          const float lv = s2.y < 0.f ? -INFINITY : lg2(vs), over = 1.f / vs;  // (a page outside the pool: passed over)
          const bool in = j >= w.lo && j < w.hi;
          const bool full = j0 >= all_lo && j0 + kKeys <= all_hi;
          if (j0 < w.lo || j0 + kKeys > w.hi) {
            // slots that hold no key of the item: zero times them would be NaN if they held one
            wait(C::B_VF + ns % C::VST, ns / C::VST);
            if (!in && !bad) {
              const uint32_t to = sV + ns % C::VST * C::T_BYTES + tid * D;
#pragma unroll
              for (int i = 0; i < D; i += 16) sts_v4(to + i, 0, 0, 0, 0);
            }
          }
          // y = log2 of P, with the references as they are; -inf where the key is not seen
          float y[NC], most = -INFINITY;
          auto logits = [&]() {
            most = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
              const float4 f = *reinterpret_cast<const float4 *>(col + par * NC + c);
              y[c] = fmaf(__uint_as_float(acc[c]) * s2.x, f.x, lv + f.y);
              y[c + 1] = fmaf(__uint_as_float(acc[c + 1]) * s2.x, f.z, lv + f.w);
            }
            if (!full) {
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                const int2 r = lim[par * NC + c];
                if (j < r.x || j >= r.y) y[c] = -INFINITY;
              }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) most = fmaxf(most, y[c]);
          };
          logits();
          if (any_of_128(most > kTop || bad)) {
            if (any_of_128(bad)) {
              bad = true;
              break;
            }
            // the columns' largest logits, and a new reference where one is passed
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              float t = y[c];
#pragma unroll
              for (int o = 16; o > 0; o /= 2) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
              if (lane == 0) wm[warp * NC + c] = t;
            }
            named_sync(1, 128);
            if (tid < NC) {
              const float t = fmaxf(fmaxf(wm[tid], wm[NC + tid]), fmaxf(wm[2 * NC + tid], wm[3 * NC + tid]));
              // (t is less the reference, and tells nothing where there was none)
              const float2 now = col[par * NC + tid];
              float f = 1.f;
              if (t > kTop) {
                const bool none = now.y == -kNoRef;
                col[par * NC + tid].y = none ? 0.f : now.y - (t - kSet);
                f = none ? 0.f : ex2(kSet - t);
              }
              fac[tid] = f;
            }
            named_sync(1, 128);
            bool first = false;
#pragma unroll
            for (int c = 0; c < NC; ++c) first |= fac[c] == 0.f;
            if (first) {
              // columns that had no reference: their logits as they are, then the reference from them
              logits();
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                float t = y[c];
#pragma unroll
                for (int o = 16; o > 0; o /= 2) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                if (lane == 0) wm[warp * NC + c] = t;
              }
              named_sync(1, 128);
              if (tid < NC && fac[tid] == 0.f) {
                const float t = fmaxf(fmaxf(wm[tid], wm[NC + tid]), fmaxf(wm[2 * NC + tid], wm[3 * NC + tid]));
                col[par * NC + tid].y += kSet - t;
              }
              named_sync(1, 128);
            }
            if (m > 0) {
              // O is rescaled once the product before has completed
              wait(C::B_PE + (ns - 1) % C::PB, (ns - 1) / C::PB);
              if (any_of_128(bad)) {
                bad = true;
                break;
              }
              fence_after();
#pragma unroll 1
              for (int i = 0; i < C::NP; i += 16) {
                uint32_t o[16];
                __syncwarp();
                tmem_ld16(t_addr + C::O_COL + i, o);
                tmem_ld_wait();
                pin(o);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (i + e < 3 * NC) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac[(i + e) % NC]);
                tmem_st16(t_addr + C::O_COL + i, o);
              }
              tmem_st_wait();
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) l[c] *= fac[c];
            logits();
          }
          // P in three terms: each the rest's nearest with the high byte of an fp16 alone
          uint32_t w4[C::NP / 4];
#pragma unroll
          for (int i = 3 * NC / 4; i < C::NP / 4; ++i) w4[i] = 0;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = ex2(y[c + i]);
              l[c + i] = fmaf(e[i], over, l[c + i]);
            }
            __half2 a = __floats2half2_rn(e[0], e[1]), d = __floats2half2_rn(e[2], e[3]);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              const uint32_t ra = *reinterpret_cast<uint32_t *>(&a) + 0x00800080u, rd = *reinterpret_cast<uint32_t *>(&d) + 0x00800080u;
              w4[t * NC / 4 + c / 4] = __byte_perm(ra, rd, 0x7531);
              if (t < 2) {
                const uint32_t ka = ra & 0xff00ff00u, kd = rd & 0xff00ff00u;
                a = __hsub2(a, *reinterpret_cast<const __half2 *>(&ka));
                d = __hsub2(d, *reinterpret_cast<const __half2 *>(&kd));
              }
            }
          }
          if (ns >= C::PB) wait(C::B_PE + pb, ns / C::PB - 1);  // (a wait that gave up: the vote on the next tile tells)
          const uint32_t to = sP + pb * C::P_BYTES + tid * 16;
#pragma unroll
          for (int i = 0; i < C::NP / 16; ++i) sts_v4(to + i * 16 * kKeys, w4[4 * i], w4[4 * i + 1], w4[4 * i + 2], w4[4 * i + 3]);
          fence_proxy_async_smem();
          fence_before();  // (a rescaled O)
          mbar_arrive(bar(C::B_PF + pb));
        }
        if (bad) break;
        // sums over the keys
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
          for (int o = 16; o > 0; o /= 2) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
          if (lane == 0) wm[warp * NC + c] = l[c];
        }
        wait(C::B_OF, seg);
        if (any_of_128(bad)) {
          bad = true;
          break;
        }
        fence_after();
        float o[NC];
        {
          uint32_t r[C::NP];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::NP; i += 16) tmem_ld<16>(t_addr + C::O_COL + i, r + i);
          tmem_ld_wait();
          pin(r);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            o[c] = __uint_as_float(r[c]) + (__uint_as_float(r[NC + c]) + __uint_as_float(r[2 * NC + c]));
        }
        fence_before();
        mbar_arrive(bar(C::B_OE));
        float *part = p.part + (2ll * blockIdx.x + (off == 0 ? 1 : 0)) * C::PART;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          int row, head;
          if (!column_of(p, NC, w, c, row, head)) continue;
          const float sum = wm[c] + wm[NC + c] + wm[2 * NC + c] + wm[3 * NC + c], ref = -col[par * NC + c].y;
          if (whole) {
            const long long at = (long long)(w.q0 + row) * b.h_q + head;
            if (tid < D) static_cast<T *>(b.out)[at * D + tid] = from_f32<T>(sum == 0.f ? 0.f : o[c] / sum);
            if (tid == 0 && b.lse)
              b.lse[(long long)head * b.total_q + w.q0 + row] = sum == 0.f ? -INFINITY : (ref + lg2(sum)) * kLn2;
          } else {
            if (tid < D) part[c * D + tid] = o[c];
            if (tid == 0) {
              part[NC * D + c] = ref;
              part[NC * D + NC + c] = sum;
            }
          }
        }
        ++seg;
      }
      left -= n;
      if (left == 0 && tid == 0) {
        // an item that this CTA begins and others end
        if (w.nt > 0 && off == 0 && n < units) open_item(p, run, w, units - n);
        else no_item(p);
      }
      off = 0;
      if (left > 0) w.next();
    }
    if (bad && tid == 0) no_item(p);
  }
  fence_before();
  __syncthreads();
  if (warp == 5) {
    fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// Columns of a tile: the fewest that hold a sequence's rows of a kv head's group (32 at most: many_rows).
int columns(int max_q, int group) {
  const long long n = (long long)max_q * group;
  return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
}
template <typename F> void with(int d, int nc, F f) {
  auto at = [&](auto dd) {
    if (nc == 4) f(dd, std::integral_constant<int, 4>{});
    else if (nc == 8) f(dd, std::integral_constant<int, 8>{});
    else if (nc == 16) f(dd, std::integral_constant<int, 16>{});
    else f(dd, std::integral_constant<int, 32>{});
  };
  if (d == 64) at(std::integral_constant<int, 64>{});
  else at(std::integral_constant<int, 128>{});
}

}  // namespace

bool pages_tc_supported(int d_qk, int d_v, int dtype, unsigned flags) {
  return (dtype == VLF_F16 || dtype == VLF_BF16) && !(flags & VLF_FLAG_FORCE_SIMT) && d_qk == d_v && (d_qk == 64 || d_qk == 128);
}

size_t pages_tc_workspace(int max_q, int group, int d, int num_sms) {
  if (num_sms < 1) return 0;
  size_t n = 0;
  with(d, columns(max_q, group), [&](auto dd, auto nc) {
    using C = Cfg<decltype(dd)::value, decltype(nc)::value>;
    const size_t grid = (size_t)C::CTAS * num_sms;
    n = ((grid * 2 * sizeof(int4) + 255) & ~(size_t)255) + 2 * grid * C::PART * sizeof(float);
  });
  return n;
}

cudaError_t pages_tc_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;
  const int group = a.p.group, nc = columns(a.p.max_q, group);
  CUtensorMap k_map, v_map;
  const uint64_t heads = (uint64_t)a.num_pages * a.p.h_kv;
  if (!make_tmap_pages(&k_map, a.k_pages, heads, a.page, a.p.d_qk, kKeys) || !make_tmap_pages(&v_map, a.v_pages, heads, a.page, a.p.d_v, kKeys))
    return e;
  with(a.p.d_qk, nc, [&](auto dd, auto cc) {
    constexpr int D = decltype(dd)::value, NC = decltype(cc)::value;
    using C = Cfg<D, NC>;
    TcParams p{};
    p.a = a;
    p.splits = 1;  // (the columns hold a whole group)
    p.rows = NC / group;
    p.magic = magic_of(group);
    const size_t grid = (size_t)C::CTAS * num_sms;
    p.rec = static_cast<int4 *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + ((grid * 2 * sizeof(int4) + 255) & ~(size_t)255));
    const bool bf = a.p.dtype == VLF_BF16;
    const void *kern = bf ? (const void *)pages_tc_kernel<D, NC, true> : (const void *)pages_tc_kernel<D, NC, false>;
    const void *join = bf ? (const void *)pages_join_kernel<D, NC, kKeys, true> : (const void *)pages_join_kernel<D, NC, kKeys, false>;
    if ((e = set_smem_once(kern, C::SMEM)) != cudaSuccess) return;
    void *args[3] = {&k_map, &v_map, &p};
    e = launch_dependent(kern, dim3((unsigned)grid), 192, C::SMEM, st, args);
    if (e == cudaSuccess) count_launch();
    void *jargs[1] = {&p};
    if (e == cudaSuccess) e = launch_dependent(join, dim3((unsigned)grid, (NC + kJoinWarps - 1) / kJoinWarps), 32 * min(NC, kJoinWarps), 0, st, jargs);
    if (e == cudaSuccess) count_launch();
  });
  return e;
}

}  // namespace vlf
