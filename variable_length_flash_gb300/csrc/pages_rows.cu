// Attention over pages in e4m3 for many query rows (prompts, extended chats), 16-bit queries, widths 64 and 128:
// rows are the rows of the products, as in the forward (tc_fwd.cu), and a key tile serves 256 of them.
//
// The products are tcgen05 kind::f16 in fp16.  An e4m3 number is an fp16 number, so four warps turn the
// bytes of a tile into fp16 tiles in shared memory, exactly, once for two query tiles; a query is brought to
// [128, 256) by a power of two for its row, where fp16 holds bf16's 8 bits down to 2^-24 of the row's largest
// (fp16 queries are taken as they are).  Scales of pages: a tile has one for its keys and one for its values,
// the largest of its pages' (of 64 and more tokens: the page's own); smaller ones of other pages are multiplied
// into the fp16 numbers, powers of two.  The key scale goes into the softmax's scale, the value scale into the
// exponent, as in pages_tc.cu, whose runs of key tiles, parts and join these are as well.  P is rounded to
// fp16 with the row's largest between 2^7 and 2^15: half a step of 2^-11, nothing above 2^-31 of the largest lost.
//
// Roles of a CTA (one per SM): warp 0 page loads, warp 1 S = Q K^T, warp 2 O += P V, warps 4-7 bytes to fp16,
// warps 8-15 softmax and output, a thread for each row of the two query tiles.  TMEM: O of both tiles, two S of
// 64 keys each, over which P is written.
#include "e4m3.cuh"
#include "pages_tc.cuh"

namespace vlf {
namespace {

using namespace pages;

constexpr int kN = 64;             // keys of a tile
constexpr float kMove = 8.f;       // log2 of what a row's largest may grow by before O is rescaled
constexpr float kLift = 7.f;       // log2 of a row's largest P when its reference is set
constexpr int kScales = 16;        // tiles whose scales are held (more than the rings let loads run ahead)
constexpr int kThreads = 512;

template <int D> struct RowCfg {
  static constexpr int KB = D / 64;                          // blocks of 64 columns
  static constexpr int QBLK = 128 * 128, Q_TILE = KB * QBLK;
  static constexpr int BLK = kN * 128, T_BYTES = KB * BLK;   // an fp16 tile
  static constexpr int B_BYTES = kN * D;                     // a tile as bytes
  static constexpr int NK = 3, NV = 3, NB = 2;
  static constexpr int OFF_Q = 0, OFF_K = OFF_Q + 2 * Q_TILE, OFF_V = OFF_K + NK * T_BYTES, OFF_BK = OFF_V + NV * T_BYTES,
                       OFF_BV = OFF_BK + NB * B_BYTES, OFF_SC = OFF_BV + NB * B_BYTES;  // float2[kScales][4]
  static constexpr int OFF_RED = OFF_SC + kScales * 4 * 8;   // long long[18]
  static constexpr int OFF_BAR = OFF_RED + 18 * 8;
  static constexpr int B_BKF = 0, B_BKE = B_BKF + NB, B_BVF = B_BKE + NB, B_BVE = B_BVF + NB, B_KF = B_BVE + NB,
                       B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + NV, B_Q = B_VE + NV, B_S = B_Q + 2, B_P = B_S + 4,
                       B_O = B_P + 4, B_OE = B_O + 4, B_SC = B_OE + 2, B_DRAIN = B_SC + kScales, BARS = B_DRAIN + 2;
  static constexpr int SMEM = OFF_BAR + BARS * 8 + 16 + 1024;
  static constexpr int S_COL = 2 * D, TMEM = 512;            // S[tile][buffer] behind the two O
  static constexpr int NC = 256, PART = NC * (D + 2);
};

// Lanes of a query tile that have a row: whole query rows of a group, or 128 heads of one.
__host__ __device__ __forceinline__ int lanes_of(int group) { return group > 128 ? 128 : 128 / group * group; }

__device__ __forceinline__ uint32_t fp16_of(uint32_t two_bytes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two_bytes));
  return h;
}
__device__ __forceinline__ uint32_t scaled(uint32_t h, uint32_t by) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&by));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    pages_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ TcParams p) {
  using C = RowCfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t base = (smem_u32(smem_dyn) + 1023u) & ~1023u;
  uint8_t *const smem = smem_dyn + (base - smem_u32(smem_dyn));
  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V, sBK = base + C::OFF_BK, sBV = base + C::OFF_BV;
  float2 *const scales = reinterpret_cast<float2 *>(smem + C::OFF_SC);
  auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
  uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + C::BARS * 8);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Params &b = p.a.p;
  int *const err = b.err;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(bar(C::B_BKF + i), 1); mbar_init(bar(C::B_BKE + i), 128);
      mbar_init(bar(C::B_BVF + i), 1); mbar_init(bar(C::B_BVE + i), 128);
    }
    for (int i = 0; i < C::NK; ++i) { mbar_init(bar(C::B_KF + i), 128); mbar_init(bar(C::B_KE + i), 1); }
    for (int i = 0; i < C::NV; ++i) { mbar_init(bar(C::B_VF + i), 128); mbar_init(bar(C::B_VE + i), 1); }
    for (int i = 0; i < 4; ++i) { mbar_init(bar(C::B_S + i), 1); mbar_init(bar(C::B_P + i), 128); mbar_init(bar(C::B_O + i), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(bar(C::B_Q + i), 128); mbar_init(bar(C::B_OE + i), 128); mbar_init(bar(C::B_DRAIN + i), 1); }
    for (int i = 0; i < kScales; ++i) mbar_init(bar(C::B_SC + i), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  pdl_wait();
  const Run run = run_of<kN, kThreads>(p, reinterpret_cast<long long *>(smem + C::OFF_RED));
  Walk<kN> w(p);
  const int L = lanes_of(b.group);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, abort_flag, err)); };
  // whether an item has rows for the second query tile
  auto tiles_of = [&](const Walk<kN> &x) {
    return p.splits > 1 ? (b.group - x.qt % p.splits * C::NC > L ? 2 : 1) : ((x.r1 - x.r0) * b.group > L ? 2 : 1);
  };

  if (!run.any) {
    if (threadIdx.x == 0) p.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
  } else if (warp == 0) {
    // ------------------------------------------------------------------ pages
    int off = w.seek(run.seq, run.unit);
    const int page = min(p.a.page, kN), npt = kN / page;  // slots and pages of a tile
    const int log2_page = p.a.log2_page, none = p.a.num_pages * b.h_kv;
    bool ok = true;
    long long left = run.f1 - run.f0;
    int nt = 0;
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        const int32_t *row = p.a.table + (long long)w.s * p.a.max_pages;
        // a lane has a page of a tile, and that of the next one
        auto id_of = [&](int m) {
          const int i = ((w.t0 + off + m) * kN >> log2_page) + lane;
          if (m >= n || lane >= npt || i > (w.hi - 1) >> log2_page || i < w.lo >> log2_page) return -2;  // no key in it
          return max(__ldg(row + i), -1);
        };
        auto real = [&](int id) { return id >= 0 && id < p.a.num_pages; };
        auto scale_of = [&](int id) {
          if (!real(id)) return make_float2(0.f, 0.f);
          const long long at = (long long)id * b.h_kv + w.head;
          return make_float2(__ldg(p.a.k_scale + at), __ldg(p.a.v_scale + at));
        };
        int id = id_of(0), next = id_of(1);
        float2 sc = scale_of(id);
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int after = id_of(m + 2);
          const float2 sc_next = scale_of(next);
          const bool have = id != -2;
          if (have && !real(id)) set_error(err, VLF_ERR_BAD_PAGES);
          const int z = real(id) ? id * b.h_kv + w.head : none;  // (outside: zeros)
          const int bytes = __popc(__ballot_sync(0xffffffffu, have)) * page * D;
          const int y = p.a.page > kN ? (w.t0 + off + m) * kN & (p.a.page - 1) : 0;
          const int sb = nt % C::NB;
          if (nt >= C::NB) ok = wait(C::B_BKE + sb, nt / C::NB - 1);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(C::B_BKF + sb), bytes);
          __syncwarp();
          if (have) tma_load_3d(sBK + sb * C::B_BYTES + lane * page * D, &k_map, 0, y, z, bar(C::B_BKF + sb));
          if (lane < npt) scales[nt % kScales * 4 + lane] = sc;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_SC + nt % kScales));
          if (nt >= C::NB) ok = wait(C::B_BVE + sb, nt / C::NB - 1);
          // (a wait that gave up: the keys' copy is waited for below, the values' was not begun)
          if (!ok) { ++nt; break; }
          if (lane == 0) mbar_expect_tx(bar(C::B_BVF + sb), bytes);
          __syncwarp();
          if (have) tma_load_3d(sBV + sb * C::B_BYTES + lane * page * D, &v_map, 0, y, z, bar(C::B_BVF + sb));
          id = next;
          next = after;
          sc = sc_next;
        }
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0)
      for (int i = 0; i < C::NB && i < nt; ++i) {
        drain_wait(bar(C::B_BKF + i), ((nt - 1 - i) / C::NB) & 1);
        drain_wait(bar(C::B_BVF + i), ((nt - 1 - i) / C::NB) & 1);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    int off = w.seek(run.seq, run.unit);
    const uint32_t id = idesc_f16(0, 128, kN, 0, 0);
    const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024);
    bool ok = true;
    long long left = run.f1 - run.f0;
    int nt = 0, ns[2] = {0, 0}, seg[2] = {0, 0};  // tiles; of each query tile the S issued and items begun
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        const int tiles = tiles_of(w);
        for (int t = 0; t < tiles && ok; ++t) ok = wait(C::B_Q + t, seg[t]++);
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int sl = nt % C::NK;
          ok = wait(C::B_KF + sl, nt / C::NK);
          const uint64_t dk = dk0 + (uint64_t)((sl * C::T_BYTES) >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tiles || !ok) continue;
            const int sb = ns[t] & 1;
            if (ns[t] >= 2) ok = wait(C::B_O + 2 * t + sb, ns[t] / 2 - 1);  // (the P there has been multiplied)
            if (!ok) continue;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::S_COL + (2 * t + sb) * kN, dq0 + (uint64_t)((t * C::Q_TILE + (kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                       dk + (uint64_t)(((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4), id, kk > 0);
            mma_commit_w(bar(C::B_S + 2 * t + sb));
            ++ns[t];
          }
          if (ok) mma_commit_w(bar(C::B_KE + sl));
        }
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
    mma_commit_w(bar(C::B_DRAIN));
    drain_wait(bar(C::B_DRAIN), 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ O += P V
    int off = w.seek(run.seq, run.unit);
    const uint32_t id = idesc_f16(0, 128, D, 0, 1);  // V is MN-major
    const uint64_t dv0 = sdesc_sw128(sV, C::BLK, 1024);
    bool ok = true;
    long long left = run.f1 - run.f0;
    int nt = 0, ns[2] = {0, 0}, seg[2] = {0, 0};
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        const int tiles = tiles_of(w);
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int sl = nt % C::NV;
          ok = wait(C::B_VF + sl, nt / C::NV);
          const uint64_t dv = dv0 + (uint64_t)((sl * C::T_BYTES) >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tiles || !ok) continue;
            const int sb = ns[t] & 1;
            ok = wait(C::B_P + 2 * t + sb, ns[t] / 2);
            if (ok && m == 0 && seg[t] > 0) ok = wait(C::B_OE + t, seg[t] - 1);
            if (!ok) continue;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_ts_w(tmem + t * D, tmem + C::S_COL + (2 * t + sb) * kN + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id,
                       (m > 0 || kk > 0) ? 1u : 0u);
            mma_commit_w(bar(C::B_O + 2 * t + sb));
            ++ns[t];
          }
          if (ok) mma_commit_w(bar(C::B_VE + sl));
        }
        for (int t = 0; t < tiles; ++t) ++seg[t];
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
    mma_commit_w(bar(C::B_DRAIN + 1));
    drain_wait(bar(C::B_DRAIN + 1), 0);
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------------ bytes to fp16
    int off = w.seek(run.seq, run.unit);
    const int tid = threadIdx.x - 128;
    constexpr int PER = D / 16, UNITS = kN * PER / 128;  // 16-byte pieces of a row; of a thread
    const int log2_page = min(p.a.log2_page, 6), npt = kN >> log2_page;
    bool ok = true;
    long long left = run.f1 - run.f0;
    int nt = 0;
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left);
      if (w.nt > 0) {
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int j0 = (w.t0 + off + m) * kN, sb = nt % C::NB, sc = nt % kScales;
          const bool inside = j0 >= w.lo && j0 + kN <= w.hi;
          ok = wait(C::B_SC + sc, nt / kScales);
          float kref = 0.f, vref = 0.f;
          for (int i = 0; ok && i < npt; ++i) {
            kref = fmaxf(kref, scales[sc * 4 + i].x);
            vref = fmaxf(vref, scales[sc * 4 + i].y);
          }
          // one operand: its bytes, the slot of the fp16 tile, the scale of a page against the tile's
          auto turn = [&](uint32_t from, uint32_t to, bool values) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
              const int x = tid + 128 * i, r = x / PER, u = x % PER;
              uint32_t q[4];
              // (rows of D bytes, 16-byte pieces swizzled by the row)
              lds_v4(from + r * D + ((D == 128 ? u ^ (r & 7) : u ^ (r >> 1 & 3)) << 4), q[0], q[1], q[2], q[3]);
              const bool in = inside || (j0 + r >= w.lo && j0 + r < w.hi);
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                h[2 * e] = fp16_of(q[e]);
                h[2 * e + 1] = fp16_of(q[e] >> 16);
              }
              if (npt > 1) {
                const float2 s = scales[sc * 4 + (r >> log2_page)];
                const float f = values ? s.y / vref : s.x / kref;
                const __half2 by = __float2half2_rn(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = scaled(h[e], *reinterpret_cast<const uint32_t *>(&by));
              }
              if (!in) {  // (slots that hold no key of the item)
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = 0;
              }
              const uint32_t at = to + (u >> 2) * C::BLK + r * 128;
              const int c = 2 * (u & 3);
              sts_v4(at + (((c) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
              sts_v4(at + (((c + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
            }
          };
          const int ks = nt % C::NK, vs = nt % C::NV;
          if (ok) ok = wait(C::B_BKF + sb, nt / C::NB);
          if (ok && nt >= C::NK) ok = wait(C::B_KE + ks, nt / C::NK - 1);
          if (!ok) break;
          turn(sBK + sb * C::B_BYTES, sK + ks * C::T_BYTES, false);
          fence_proxy_async_smem();
          mbar_arrive(bar(C::B_BKE + sb));
          mbar_arrive(bar(C::B_KF + ks));
          ok = wait(C::B_BVF + sb, nt / C::NB);
          if (ok && nt >= C::NV) ok = wait(C::B_VE + vs, nt / C::NV - 1);
          if (!ok) break;
          turn(sBV + sb * C::B_BYTES, sV + vs * C::T_BYTES, true);
          fence_proxy_async_smem();
          mbar_arrive(bar(C::B_BVE + sb));
          mbar_arrive(bar(C::B_VF + vs));
        }
      }
      left -= n;
      off = 0;
      if (left > 0) w.next();
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ softmax / output
    const int t = (warp - 8) / 4, r = (threadIdx.x - 256) % 128;  // query tile and row of it
    const uint32_t t_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_addr = t_addr + t * D, s_addr = t_addr + C::S_COL + 2 * t * kN;
    const int log2_page = min(p.a.log2_page, 6), npt = kN >> log2_page;
    int off = w.seek(run.seq, run.unit);
    int nt = 0, ns = 0;  // tiles; the ones of this query tile
    bool ok = true;
    long long left = run.f1 - run.f0;
    while (left > 0 && ok) {
      const int n = (int)min((long long)(w.units() - off), left), units = w.units();
      const bool whole = off == 0 && n == units, live = t < tiles_of(w);
      int row = 0, head = 0;
      const int c = t * L + r;
      const bool have = live && r < L && column_of(p, C::NC, w, c, row, head);
      const long long at = (long long)(w.q0 + row) * b.h_q + head;
      if (w.nt == 0) {
        if (have) {  // a row that sees no key
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(b.out) + at * D);
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
          if (b.lse) b.lse[(long long)head * b.total_q + w.q0 + row] = -INFINITY;
        }
      } else if (!live) {
        nt += n;
      } else {
        // the row's query, in fp16 over a power of two, where the product finds it
        float down = 1.f;
        {
          const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const T *>(b.q) + at * D);
          float up = 1.f;
          if constexpr (BF16) {
            uint32_t top = 0;
            if (have) {
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                const uint4 x = __ldg(q + i);
                top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
              }
            }
            top = max(top & 0xffffu, top >> 16);
            const int ex = min(max((int)(top >> 7) - 127, -100), 127);
            up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
            down = __uint_as_float((uint32_t)(127 - 7 + ex) << 23);
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (have) x = __ldg(q + i);
            if constexpr (BF16) {
              uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2(y[e], 1);
                y[e] = pack2(f.x * up, f.y * up, 0);
              }
              x = make_uint4(y[0], y[1], y[2], y[3]);
            }
            sts_v4(sQ + t * C::Q_TILE + (i >> 3) * C::QBLK + r * 128 + (((i & 7) ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(C::B_Q + t));
        }
        int vlo = 0, vhi = 0x7fffffff;  // the row's keys (of a lane without a row, which nobody reads: all)
        if (have) visible_range(row, w.len - w.q_len, w.len, b.causal, b.window, vlo, vhi);
        const float sl2 = b.scale_log2 * down;
        float m_ref = -INFINITY, l = 0.f;
        for (int m = 0; m < n; ++m, ++nt, ++ns) {
          const int kb = (w.t0 + off + m) * kN, sb = ns & 1, sc = nt % kScales;
          ok = wait(C::B_S + 2 * t + sb, ns / 2) && wait(C::B_SC + sc, nt / kScales);
          if (!ok) break;
          fence_after();
          const uint32_t s_at = s_addr + sb * kN;
          const int elo = vlo - kb, ehi = vhi - kb;
          uint32_t v[kN];
          __syncwarp();
          tmem_ld32_at(s_at, v, 0);
          tmem_ld32_at(s_at + 32, v, 32);
          float kref = 0.f, vref = 0.f;
          for (int i = 0; i < npt; ++i) {
            kref = fmaxf(kref, scales[sc * 4 + i].x);
            vref = fmaxf(vref, scales[sc * 4 + i].y);
          }
          vref = fminf(fmaxf(vref, 0x1p-100f), 0x1p120f);  // (a scale of zero or no number: of no weight)
          const float c1 = fmaxf(kref * sl2, 1e-37f), lv = lg2(vref), over = 1.f / vref;
          tmem_ld_wait();
          pin(v);
          if (!__all_sync(0xffffffffu, elo <= 0 && ehi >= kN)) {
#pragma unroll
            for (int e = 0; e < kN; ++e)
              if (e < elo || e >= ehi) v[e] = 0xff800000u;
          }
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t *x = v + 8 * i;
            auto f = [&](int k) { return __uint_as_float(x[k]); };
            m8[i] = fmax3(fmax3(f(0), f(1), f(2)), fmax3(f(3), f(4), f(5)), fmaxf(f(6), f(7)));
          }
          const float mx = fmaf(fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])), c1, lv);
          const bool move = mx > m_ref + kMove;  // (not by a NaN, nor where nothing is seen)
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mx : m_ref, alpha = move ? ex2(m_ref - m_new) : 1.f;
            if (__any_sync(0xffffffffu, move && l != 0.f) && m > 0) {
              // O is rescaled once the product before (so every earlier one) has completed
              ok = wait(C::B_O + 2 * t + ((ns - 1) & 1), (ns - 1) / 2);
              if (!ok) break;
              fence_after();
              const float f = l != 0.f ? alpha : 1.f;
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                uint32_t o[16];
                __syncwarp();
                tmem_ld16(o_addr + i, o);
                tmem_ld_wait();
                pin(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_addr + i, o);
              }
            }
            l *= alpha;
            m_ref = m_new;
          }
          const float add = m_ref == -INFINITY ? 0.f : lv - m_ref + kLift;
          const uint64_t c2 = f2pack(c1, c1), a2 = f2pack(add, add);
          uint64_t s0 = f2pack(0.f, 0.f), s1 = s0;
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = 32 * ch + 2 * e;
              const float2 x = f2unpack(fma2(f2pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2, a2));
              const float pa = ex2(x.x), pb = ex2(x.y);
              pk[e] = pack2(pa, pb, 0);
              if (e & 1) s1 = add2(s1, f2pack(pa, pb));
              else s0 = add2(s0, f2pack(pa, pb));
            }
            __syncwarp();
            tmem_st16(s_at + ch * 16, pk);
          }
          const float2 f0 = f2unpack(s0), f1 = f2unpack(s1);
          l = fmaf((f0.x + f0.y) + (f1.x + f1.y), over, l);
          __syncwarp();
          tmem_st_wait();
          fence_before();
          mbar_arrive(bar(C::B_P + 2 * t + sb));
        }
        if (ok) ok = wait(C::B_O + 2 * t + ((ns - 1) & 1), (ns - 1) / 2);
        if (!ok) break;
        fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float *part = p.part + (2ll * blockIdx.x + (off == 0 ? 1 : 0)) * C::PART;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o_addr + i, o);
          tmem_ld_wait_for(o);
          if (!have) continue;
          if (whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(b.out) + at * D + i);
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = pack2(l == 0.f ? 0.f : __uint_as_float(o[2 * e]) * inv, l == 0.f ? 0.f : __uint_as_float(o[2 * e + 1]) * inv, BF16);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          } else {
            float2 *dst = reinterpret_cast<float2 *>(part + (long long)c * D + i);
#pragma unroll
            for (int e = 0; e < 16; ++e) dst[e] = make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          }
        }
        fence_before();
        mbar_arrive(bar(C::B_OE + t));
        if (have) {
          const float ref = m_ref - kLift;  // (minus infinity where no key was seen: l is 0 then)
          if (!whole) {
            part[C::NC * D + c] = ref;
            part[C::NC * D + C::NC + c] = l;
          } else if (b.lse) {
            b.lse[(long long)head * b.total_q + w.q0 + row] = l == 0.f ? -INFINITY : (ref + lg2(l)) * kLn2;
          }
        }
      }
      left -= n;
      if (left == 0 && threadIdx.x == 256) {
        // an item that this CTA begins and others end
        const bool open = w.nt > 0 && off == 0 && n < units;
        p.rec[blockIdx.x] = open ? open_item(run, w, units - n) : make_int4(-1, 0, 0, 0);
      }
      off = 0;
      if (left > 0) w.next();
    }
    if (!ok && threadIdx.x == 256) p.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

}  // namespace

size_t pages_rows_workspace(int d, int num_sms) {
  const size_t part = d == 64 ? RowCfg<64>::PART : RowCfg<128>::PART;
  return (((size_t)num_sms * sizeof(int4) + 255) & ~(size_t)255) + 2 * (size_t)num_sms * part * sizeof(float);
}

cudaError_t pages_rows_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st) {
  CUtensorMap k_map, v_map;
  const uint64_t heads = (uint64_t)a.num_pages * a.p.h_kv;
  if (!make_tmap_pages(&k_map, a.k_pages, heads, a.page, a.p.d_qk, kN) || !make_tmap_pages(&v_map, a.v_pages, heads, a.page, a.p.d_v, kN))
    return cudaErrorInvalidValue;
  auto go = [&](auto dd) {
    constexpr int D = decltype(dd)::value;
    using C = RowCfg<D>;
    const int group = a.p.group, L = lanes_of(group);
    TcParams p{};
    p.a = a;
    p.splits = group > 128 ? (group + C::NC - 1) / C::NC : 1;
    p.rows = group > 128 ? 1 : 2 * L / group;
    p.rec = static_cast<int4 *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + (((size_t)num_sms * sizeof(int4) + 255) & ~(size_t)255));
    const bool bf = a.p.dtype == VLF_BF16;
    const void *kern = bf ? (const void *)pages_rows_kernel<D, true> : (const void *)pages_rows_kernel<D, false>;
    const void *join = bf ? (const void *)pages_join_kernel<D, C::NC, kN, true> : (const void *)pages_join_kernel<D, C::NC, kN, false>;
    cudaError_t e = set_smem_once(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    void *args[3] = {&k_map, &v_map, &p};
    e = launch_dependent(kern, dim3((unsigned)num_sms), kThreads, C::SMEM, st, args);
    if (e == cudaSuccess) count_launch();
    void *jargs[1] = {&p};
    if (e == cudaSuccess) e = launch_dependent(join, dim3((unsigned)num_sms, C::NC / kJoinWarps), 32 * kJoinWarps, 0, st, jargs);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  return a.p.d_qk == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace vlf
