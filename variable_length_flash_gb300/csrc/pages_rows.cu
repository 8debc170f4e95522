// Attention over pages in e4m3 for many query rows (prompts, extended chats), 16-bit queries, widths 64 and 128:
// rows are the rows of the products, as in the forward (tc_fwd.cu), and a key tile serves 256 of them.
//
// The products are tcgen05 kind::f16 in fp16.  An e4m3 number is an fp16 number, so eight warps turn the
// bytes of a tile into fp16 tiles in shared memory, exactly, once for two query tiles; a query is brought to
// [128, 256) by a power of two for its row, where fp16 holds bf16's 8 bits down to 2^-24 of the row's largest
// (fp16 queries are taken as they are).  Scales of pages stay out of the fp16 numbers: a page's key scale multiplies the
// logits of its keys, its value scale goes into their exponent, as in pages_tc.cu, whose runs of key tiles, parts
// and join these are as well.  (Tiles that held their pages' values over the largest scale of a page lost those of pages
// 2^16 below it, which a row that sees no other page needs.)  A tile of 64 keys has one page, or, SMALL, two or four.
// P is rounded to fp16 with the row's largest between 2^7 and 2^15: half a step of 2^-11, nothing above 2^-31 of the
// largest lost.
//
// Roles of a CTA (one per SM): warp 0 page loads, warp 1 S = Q K^T, warp 2 O += P V, warp 3 the items of the CTA's
// run, which it lays out in shared memory for the others (their registers are full without it), warps 4-11 bytes
// to fp16, warps 12-19 softmax and output, a thread for each row of the two query tiles: these have the registers that
// the others give up (64 and 144 of the 96 that the launch has; a wait or a walk that is not inlined
// takes more than 64).  TMEM: O of both tiles, two S of 64 keys each, over which P is written.
//
// Bound: latency.  No unit is full (4 x 256 rows on 4096 keys: tensor pipe 33%, issue slots 43%, exponentials 17%, 94% of
// instruction fetches hit); a tile of 64 keys goes from the conversion over S, a vote and P to O with a barrier at
// each hand-over, and the order of a role's instructions moves the whole by several percent.  16 chats of 436 to 8192
// keys with 64 to 436 new rows, 32 heads over 8 of 128: 454 us (757 TFLOP/s, 40% of the rate of a large product), 472
// in pages of 16 tokens; prompts of 4 x 4096 tokens 747 us (736 TFLOP/s); width 64 345 us.  Steps: 2607 us on the
// decode kernel's columns; 598 as rows; 557 with a warp that lays the items out; 506 with bodies short enough for the
// instruction cache; 479 with masks as bits, output places found once and scales ahead of S; 458 with numbers that
// hold no scales.  Slower: exponentials before the vote (829, registers spilled), rolled loops that read S again (525 to
// 566), masks kept in TMEM (534), queries brought in by the converting warps (494).
#include "e4m3.cuh"
#include "pages_tc.cuh"

namespace vlf {
namespace {

using namespace pages;

constexpr int kN = 64;             // keys of a tile
constexpr float kMove = 8.f;       // log2 of what a row's largest may grow by before O is rescaled
constexpr float kLift = 7.f;       // log2 of a row's largest P when its reference is set
constexpr int kScales = 16;        // tiles whose scales are held (more than the rings let loads run ahead)
constexpr int kThreads = 640, kTurners = 256;  // of a CTA; that turn bytes to fp16

// A run's part of an item, as the CTA's warps read it.
struct Item {
  int s, head, q0, q_len, len, r0, r1, split;  // sequence, kv head, first row, lengths, rows, first head of the group (splits)
  int tile, n, lo, hi;                         // key tiles [tile, tile + n), the keys that its rows see
  int flags, pad[3];
};
constexpr int kEnd = 1, kTiles = 2, kWhole = 4, kFirst = 8, kTwo = 16;  // behind the last; has key tiles; is all of the item;
                                                                       // begins it; has rows for the second query tile
constexpr int kItems = 4, kReaders = 19;  // items laid out at a time; warps that read them

template <int D> struct RowCfg {
  static constexpr int KB = D / 64;                          // blocks of 64 columns
  static constexpr int QBLK = 128 * 128, Q_TILE = KB * QBLK;
  static constexpr int BLK = kN * 128, T_BYTES = KB * BLK;   // an fp16 tile
  static constexpr int B_BYTES = kN * D;                     // a tile as bytes
  static constexpr int NK = 3, NV = NK, NB = 2;              // (barriers and slots of values lie behind those of keys)
  static constexpr int OFF_Q = 0, OFF_K = OFF_Q + 2 * Q_TILE, OFF_V = OFF_K + NK * T_BYTES, OFF_BK = OFF_V + NV * T_BYTES,
                       OFF_BV = OFF_BK + NB * B_BYTES, OFF_SC = OFF_BV + NB * B_BYTES;  // float2[kScales][4]
  static constexpr int OFF_DOWN = OFF_SC + kScales * 4 * 8;  // float[256]
  static constexpr int OFF_STAGE = OFF_DOWN + 256 * 4;       // [8 warps][32 rows of 64 bytes]
  static constexpr int OFF_ITEM = OFF_STAGE + 8 * 2048;
  static constexpr int OFF_RED = OFF_ITEM + kItems * (int)sizeof(Item);  // long long[22]
  static constexpr int OFF_BAR = OFF_RED + 22 * 8;
  static constexpr int B_BKF = 0, B_BKE = B_BKF + NB, B_BVF = B_BKE + NB, B_BVE = B_BVF + NB, B_KF = B_BVE + NB,
                       B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + NV, B_Q = B_VE + NV, B_S = B_Q + 2, B_P = B_S + 4,
                       B_O = B_P + 4, B_OE = B_O + 4, B_SC = B_OE + 2, B_IF = B_SC + kScales, B_IE = B_IF + kItems, B_DRAIN = B_IE + kItems, BARS = B_DRAIN + 2;
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

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// SMALL: pages of 16 and 32 tokens.
template <int D, bool BF16, bool SMALL>
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
  float *const downs = reinterpret_cast<float *>(smem + C::OFF_DOWN);
  volatile Item *const items = reinterpret_cast<volatile Item *>(smem + C::OFF_ITEM);
  auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
  uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + C::BARS * 8);
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Params &b = p.a.p;
  int *const err = b.err;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(bar(C::B_BKF + i), 1); mbar_init(bar(C::B_BKE + i), kTurners);
      mbar_init(bar(C::B_BVF + i), 1); mbar_init(bar(C::B_BVE + i), kTurners);
    }
    for (int i = 0; i < C::NK; ++i) { mbar_init(bar(C::B_KF + i), kTurners); mbar_init(bar(C::B_KE + i), 1); }
    for (int i = 0; i < C::NV; ++i) { mbar_init(bar(C::B_VF + i), kTurners); mbar_init(bar(C::B_VE + i), 1); }
    for (int i = 0; i < 4; ++i) { mbar_init(bar(C::B_S + i), 1); mbar_init(bar(C::B_P + i), 128); mbar_init(bar(C::B_O + i), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(bar(C::B_Q + i), 128); mbar_init(bar(C::B_OE + i), 128); mbar_init(bar(C::B_DRAIN + i), 1); }
    for (int i = 0; i < kScales; ++i) mbar_init(bar(C::B_SC + i), 1);
    for (int i = 0; i < kItems; ++i) { mbar_init(bar(C::B_IF + i), 1); mbar_init(bar(C::B_IE + i), kReaders); }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM);
    tmem_relinquish();
  }
  const Run run = run_of<kN, kThreads>(p, reinterpret_cast<long long *>(smem + C::OFF_RED));
  // (here, ahead of the roles: a 64-bit division is a call, which code that changes its registers cannot make)
  Walk<kN> w(p);
  const int run_off = warp == 3 && run.any ? w.seek(run.seq, run.unit) : 0;
  const int L = lanes_of(b.group);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](int i, int parity) {
    // (mbar_wait in line, for the same reason)
    bool done = mbar_try_wait(bar(i), parity & 1);
    if (__builtin_expect(!done, 0)) {
      const uint64_t t0 = globaltimer();
      for (uint32_t n = 1; !done; ++n) {
        done = mbar_try_wait(bar(i), parity & 1);
        if ((n & 31u) || done) continue;
        if (*abort_flag) break;
        if (globaltimer() - t0 > kTimeoutNs) {
          *abort_flag = 1;
          set_error(err, VLF_ERR_TIMEOUT);
          break;
        }
      }
    }
    return __all_sync(0xffffffffu, done);
  };
  // the next item (nullptr behind the last, or where a wait gave up), and a warp's word that it is done with it
  int it = 0;
  auto next_item = [&]() -> volatile Item * {
    if (!wait(C::B_IF + it % kItems, it / kItems)) return nullptr;
    volatile Item *x = items + it % kItems;
    return x->flags & kEnd ? nullptr : x;
  };
  auto done_item = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_IE + it % kItems));
    ++it;
  };

  if (!run.any) {
    if (threadIdx.x == 0) no_item(p);
  } else if (warp < 12) {
  // registers: launched with 96 a thread, 61440 in all; then 64 for 384 threads and 144 for the 256 of the softmax, which is as many
  asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  if (warp == 0) {
    // ------------------------------------------------------------------ pages
    const int page = min(p.a.page, kN), npt = kN / page;  // slots and pages of a tile
    const int log2_page = p.a.log2_page, none = p.a.num_pages * b.h_kv;
    bool ok = true;
    int nt = 0;
    while (volatile Item *const x = ok ? next_item() : nullptr) {
      if (x->flags & kTiles) {
        const int n = x->n, tile = x->tile, lo = x->lo, hi = x->hi, kv_head = x->head;
        const int32_t *row = p.a.table + (long long)x->s * p.a.max_pages;
        // a lane has a page of a tile, and that of the next one
        auto id_of = [&](int m) {
          const int i = ((tile + m) * kN >> log2_page) + lane;
          if (m >= n || lane >= npt || i > (hi - 1) >> log2_page || i < lo >> log2_page) return -2;  // no key in it
          return max(ld(row + i), -1);
        };
        auto real = [&](int id) { return id >= 0 && id < p.a.num_pages; };
        auto scale_of = [&](int id) {
          if (!real(id)) return make_float2(0.f, -1.f);  // (keys of no weight, below)
          const long long at = (long long)id * b.h_kv + kv_head;
          return make_float2(ld(p.a.k_scale + at), ld(p.a.v_scale + at));
        };
        int id = id_of(0), next = id_of(1);
        float2 sc = scale_of(id);
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int after = id_of(m + 2);
          const float2 sc_next = scale_of(next);
          const bool have = id != -2;
          if (have && !real(id)) set_error(err, VLF_ERR_BAD_PAGES);
          const int z = real(id) ? id * b.h_kv + kv_head : none;  // (outside: zeros, so that nothing is a NaN)
          const int bytes = __popc(__ballot_sync(0xffffffffu, have)) * page * D;
          const int y = p.a.page > kN ? (tile + m) * kN & (p.a.page - 1) : 0;
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
      done_item();
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0)
      for (int i = 0; i < C::NB && i < nt; ++i) {
        drain_wait(bar(C::B_BKF + i), ((nt - 1 - i) / C::NB) & 1);
        drain_wait(bar(C::B_BVF + i), ((nt - 1 - i) / C::NB) & 1);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    const uint32_t id = idesc_f16(0, 128, kN, 0, 0);
    const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024);
    bool ok = true;
    int nt = 0, ns0 = 0, ns1 = 0, seg0 = 0, seg1 = 0;  // tiles; of each query tile the S issued and items begun
    while (volatile Item *const x = ok ? next_item() : nullptr) {
      const int flags = x->flags, n = x->n, tiles = flags & kTwo ? 2 : 1;
      done_item();
      if (flags & kTiles) {
        ok = wait(C::B_Q, seg0++);
        if (ok && tiles > 1) ok = wait(C::B_Q + 1, seg1++);
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int sl = nt % C::NK;
          ok = wait(C::B_KF + sl, nt / C::NK);
          const uint64_t dk = dk0 + (uint64_t)((sl * C::T_BYTES) >> 4);
#pragma unroll 1
          for (int t = 0; t < tiles && ok; ++t) {
            const int ns = t ? ns1 : ns0, sb = ns & 1;
            if (ns >= 2) ok = wait(C::B_O + 2 * t + sb, ns / 2 - 1);  // (the P there has been multiplied)
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::S_COL + (2 * t + sb) * kN, dq0 + (uint64_t)((t * C::Q_TILE + (kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                       dk + (uint64_t)(((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4), id, kk > 0);
            mma_commit_w(bar(C::B_S + 2 * t + sb));
            if (t) ++ns1;
            else ++ns0;
          }
          if (ok) mma_commit_w(bar(C::B_KE + sl));
        }
      }
    }
    mma_commit_w(bar(C::B_DRAIN));
    drain_wait(bar(C::B_DRAIN), 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ O += P V
    const uint32_t id = idesc_f16(0, 128, D, 0, 1);  // V is MN-major
    const uint64_t dv0 = sdesc_sw128(sV, C::BLK, 1024);
    bool ok = true;
    int nt = 0, ns0 = 0, ns1 = 0, seg0 = 0, seg1 = 0;
    while (volatile Item *const x = ok ? next_item() : nullptr) {
      const int flags = x->flags, n = x->n, tiles = flags & kTwo ? 2 : 1;
      done_item();
      if (flags & kTiles) {
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int sl = nt % C::NV;
          ok = wait(C::B_VF + sl, nt / C::NV);
          const uint64_t dv = dv0 + (uint64_t)((sl * C::T_BYTES) >> 4);
#pragma unroll 1
          for (int t = 0; t < tiles && ok; ++t) {
            const int ns = t ? ns1 : ns0, sb = ns & 1;
            ok = wait(C::B_P + 2 * t + sb, ns / 2);
            if (ok && m == 0 && (t ? seg1 : seg0) > 0) ok = wait(C::B_OE + t, (t ? seg1 : seg0) - 1);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_ts_w(tmem + t * D, tmem + C::S_COL + (2 * t + sb) * kN + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id,
                       (m > 0 || kk > 0) ? 1u : 0u);
            mma_commit_w(bar(C::B_O + 2 * t + sb));
            if (t) ++ns1;
            else ++ns0;
          }
          if (ok) mma_commit_w(bar(C::B_VE + sl));
        }
        ++seg0;
        if (tiles > 1) ++seg1;
      }
    }
    mma_commit_w(bar(C::B_DRAIN + 1));
    drain_wait(bar(C::B_DRAIN + 1), 0);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ items
    int off = run_off;
    long long left = run.f1 - run.f0;
    for (bool ok = true; ok; ++it) {
      ok = it < kItems || wait(C::B_IE + it % kItems, it / kItems - 1);
      if (!ok) break;
      volatile Item *const x = items + it % kItems;
      const int units = w.units(), n = (int)min((long long)(units - off), left);
      if (lane == 0) {
        if (left > 0) {
          x->s = w.s; x->head = w.head; x->q0 = w.q0; x->q_len = w.q_len; x->len = w.len; x->r0 = w.r0; x->r1 = w.r1;
          x->split = p.splits > 1 ? w.qt % p.splits * C::NC : 0;
          x->tile = w.t0 + off; x->n = n; x->lo = w.lo; x->hi = w.hi;
          const int columns = p.splits > 1 ? b.group - w.qt % p.splits * C::NC : (w.r1 - w.r0) * b.group;
          x->flags = (w.nt > 0 ? kTiles : 0) | (off == 0 && n == units ? kWhole : 0) | (off == 0 ? kFirst : 0) | (columns > L ? kTwo : 0);
        } else {
          x->flags = kEnd;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_IF + it % kItems));
      if (left <= 0) break;
      left -= n;
      if (left == 0 && lane == 0) {
        // an item that this CTA begins and others end
        if (w.nt > 0 && off == 0 && n < units) open_item(p, run, w, units - n);
        else no_item(p);
      }
      off = 0;
      if (left > 0) w.next();
    }
    if (left > 0 && lane == 0) no_item(p);  // (a wait gave up)
  } else {
    // ------------------------------------------------------------------ bytes to fp16
    const int tid = threadIdx.x - 128;
    constexpr int PER = D / 16, UNITS = kN * PER / kTurners;  // 16-byte pieces of a row; of a thread
    bool ok = true;
    int nt = 0;
    while (volatile Item *const x = ok ? next_item() : nullptr) {
      const int flags = x->flags, n = x->n, tile = x->tile, lo = x->lo, hi = x->hi;
      done_item();
      if (flags & kTiles) {
        for (int m = 0; m < n && ok; ++m, ++nt) {
          const int j0 = (tile + m) * kN, sb = nt % C::NB;
          const bool inside = j0 >= lo && j0 + kN <= hi;
          // keys, then values (a body for each: extends of width 128 take 458 us, 475 with one body for both)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (!ok) break;
            const int to_slot = nt % C::NK, full = C::B_BKF + 2 * C::NB * v + sb, turned = C::B_KF + 2 * C::NK * v + to_slot;
            ok = wait(full, nt / C::NB);
            if (ok && nt >= C::NK) ok = wait(turned + C::NK, nt / C::NK - 1);
            if (!ok) break;
            const uint32_t from = sBK + (C::NB * v + sb) * C::B_BYTES, to = sK + (C::NK * v + to_slot) * C::T_BYTES;
            // (rows of D bytes, 16-byte pieces swizzled by the row; eight lanes have four pieces of each of two
            // rows, at width 128 the other half of the second one: no two of them then share a bank, neither
            // here nor where they write)
            const int r = 2 * (tid >> 3) + (tid >> 2 & 1);
            auto piece = [&](int i) { return (tid & 3) + (D == 128 ? ((tid >> 2 & 1) ^ (i & 1)) * 4 : 0); };
            uint32_t q[UNITS][4];
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
              lds_v4(from + r * D + ((D == 128 ? piece(i) ^ (r & 7) : piece(i) ^ (r >> 1 & 3)) << 4), q[i][0], q[i][1], q[i][2], q[i][3]);
            // (slots that hold no key of the item; as bytes, in a branch that most tiles pass by: 491 us as numbers)
            if (!inside && !(j0 + r >= lo && j0 + r < hi)) {
#pragma unroll
              for (int i = 0; i < UNITS; ++i) q[i][0] = q[i][1] = q[i][2] = q[i][3] = 0;
            }
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                h[2 * e] = fp16_of(q[i][e]);
                h[2 * e + 1] = fp16_of(q[i][e] >> 16);
              }
              const uint32_t at = to + (piece(i) >> 2) * C::BLK + r * 128;
              const int c = 2 * (piece(i) & 3);
              sts_v4(at + (((c) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
              sts_v4(at + (((c + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(full + C::NB));
            mbar_arrive(bar(turned));
          }
        }
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // ------------------------------------------------------------------ softmax / output
    const int t = (warp - 12) / 4, r = (threadIdx.x - 384) % 128;  // query tile and row of it
    const uint32_t t_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t o_addr = t_addr + t * D, s_addr = t_addr + C::S_COL + 2 * t * kN;
    constexpr int G = SMALL ? kN / 16 : 1;  // groups of a tile's keys that have a page of their own (one of 32: two groups)
    const int log2_page = p.a.log2_page;
    int nt = 0, ns = 0;  // tiles; the ones of this query tile
    bool ok = true;
    const int wr = 32 * (warp & 3);  // first row of the warp
    // the query row and head of column c of an item; false where there is none
    auto place = [&](volatile Item *x, int c, int &row, int &head) {
      if (p.splits > 1) {
        const int h = x->split + c;
        row = x->r0;
        head = x->head * b.group + h;
        return h < b.group;
      }
      const int i = c * p.magic >> 16;
      row = x->r0 + i;
      head = x->head * b.group + c - i * b.group;
      return row < x->r1;
    };
    while (volatile Item *const x = next_item()) {
      const bool live = t == 0 || (x->flags & kTwo) != 0;
      const int c = t * L + r, n = x->n;
      if (!(x->flags & kTiles)) {
        int row, head;
        if (live && r < L && place(x, c, row, head)) {  // a row that sees no key
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(b.out) + ((long long)(x->q0 + row) * b.h_q + head) * D);
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
          if (b.lse) b.lse[(long long)head * b.total_q + x->q0 + row] = -INFINITY;
        }
      } else if (!live) {
        nt += n;
      } else {
        // The queries of this warp's rows, in fp16 over a power of two, where the product finds them: PL lanes
        // have a row, so that a load takes whole rows.
        {
          constexpr int PL = D / 8, AT_ONCE = 32 / PL, STEPS = 32 / AT_ONCE, FLY = 4;
          const int sub = lane / PL, piece = lane % PL;
    #pragma unroll 1
          for (int i0 = 0; i0 < STEPS; i0 += FLY) {
            uint4 y4[FLY];
    #pragma unroll
            for (int k = 0; k < FLY; ++k) {
              const int r2 = wr + (i0 + k) * AT_ONCE + sub;
              int row2 = 0, head2 = 0;
              y4[k] = make_uint4(0, 0, 0, 0);
              if (r2 < L && place(x, t * L + r2, row2, head2))
                y4[k] = ld(reinterpret_cast<const uint4 *>(static_cast<const T *>(b.q) + ((long long)(x->q0 + row2) * b.h_q + head2) * D) + piece);
            }
    #pragma unroll
            for (int k = 0; k < FLY; ++k) {
              const int r2 = wr + (i0 + k) * AT_ONCE + sub;
              if constexpr (BF16) {
                uint32_t y[4] = {y4[k].x, y4[k].y, y4[k].z, y4[k].w};
                uint32_t top = __vmaxu2(__vmaxu2(y[0] & 0x7fff7fffu, y[1] & 0x7fff7fffu), __vmaxu2(y[2] & 0x7fff7fffu, y[3] & 0x7fff7fffu));
    #pragma unroll
                for (int o = PL / 2; o > 0; o /= 2) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = max(top & 0xffffu, top >> 16);
                const int ex = min(max((int)(top >> 7) - 127, -100), 127);
                // (a query that is not finite: every logit of the row is NaN)
                const float up = __uint_as_float(top >= 0x7f80u ? 0x7fffffffu : (uint32_t)(127 + 7 - ex) << 23);
                if (piece == 0) downs[t * 128 + r2] = __uint_as_float((uint32_t)(127 - 7 + ex) << 23);
    #pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 f = unpack2(y[e], 1);
                  y[e] = pack2(f.x * up, f.y * up, 0);
                }
                y4[k] = make_uint4(y[0], y[1], y[2], y[3]);
              } else {
                uint32_t y[4] = {y4[k].x, y4[k].y, y4[k].z, y4[k].w};
    #pragma unroll
                for (int e = 0; e < 4; ++e) {  // (so here: x + 0 x is x, and NaN for an infinity)
                  const __half2 h = *reinterpret_cast<const __half2 *>(&y[e]), r = __hfma2(h, __half2half2(__ushort_as_half(0)), h);
                  y[e] = *reinterpret_cast<const uint32_t *>(&r);
                }
                y4[k] = make_uint4(y[0], y[1], y[2], y[3]);
              }
              sts_v4(sQ + t * C::Q_TILE + (piece >> 3) * C::QBLK + r2 * 128 + (((piece & 7) ^ (r2 & 7)) << 4), y4[k].x, y4[k].y, y4[k].z, y4[k].w);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(C::B_Q + t));
          __syncwarp();
        }
        const float down = BF16 ? downs[t * 128 + r] : 1.f;
        int vlo = 0, vhi = 0x7fffffff;  // the row's keys (of a lane without a row, which nobody reads: all)
        {
          int row, head;
          if (r < L && place(x, c, row, head))
            visible_range(row, x->len - x->q_len, x->len, b.causal, b.window, vlo, vhi);
        }
        const int tile = x->tile;
        const float sl2 = b.scale_log2 * down;
        float m_ref = -INFINITY, l = 0.f;
        for (int m = 0; m < n; ++m, ++nt, ++ns) {
          const int kb = (tile + m) * kN, sb = ns & 1, sc = nt % kScales;
          // (the scales are there long before S.  Not so for an item's first tile, behind others without rows for this
          // query tile: S tells then that the barrier is in this tile's phase)
          ok = m > 0 || wait(C::B_S + 2 * t + sb, ns / 2);
          ok = ok && wait(C::B_SC + sc, nt / kScales);
          float c1[G], lv[G], over[G];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float2 s2 = scales[sc * 4 + (SMALL ? 16 * g >> log2_page : 0)];
            const float vs = fminf(fmaxf(s2.y, 0x1p-100f), 0x1p120f);  // (a scale of zero or no number: of no weight)
            c1[g] = fmaxf(s2.x * sl2, 1e-37f);
            lv[g] = s2.y < 0.f ? -INFINITY : lg2(vs);  // (a page outside the pool: passed over)
            over[g] = rcp(vs);
          }
          ok = ok && wait(C::B_S + 2 * t + sb, ns / 2);
          if (!ok) break;
          fence_after();
          const uint32_t s_at = s_addr + sb * kN;
          const int elo = vlo - kb, ehi = vhi - kb;
          uint32_t v[kN];
          __syncwarp();
          tmem_ld32_at(s_at, v, 0);
          tmem_ld32_at(s_at + 32, v, 32);
          tmem_ld_wait();
          pin(v);
          if (!__all_sync(0xffffffffu, elo <= 0 && ehi >= kN)) {
            // (a bit for each key that is seen)
            const int first = max(0, min(elo, kN)), end = max(first, min(ehi, kN));
            const uint64_t upto = end >= 64 ? ~0ull : (1ull << end) - 1, from = first >= 64 ? ~0ull : (1ull << first) - 1;
            const uint32_t see0 = (uint32_t)(upto & ~from), see1 = (uint32_t)((upto & ~from) >> 32);
#pragma unroll
            for (int e = 0; e < kN; ++e)
              if (!((e < 32 ? see0 : see1) >> (e & 31) & 1)) v[e] = 0xff800000u;
          }
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t *x = v + 8 * i;
            auto f = [&](int k) { return __uint_as_float(x[k]); };
            m8[i] = fmax3(fmax3(f(0), f(1), f(2)), fmax3(f(3), f(4), f(5)), fmaxf(f(6), f(7)));
          }
          float mx;
          if constexpr (SMALL) {
            float y[G];
#pragma unroll
            for (int g = 0; g < G; ++g) y[g] = fmaf(fmaxf(m8[2 * g], m8[2 * g + 1]), c1[g], lv[g]);
            mx = fmaxf(fmax3(y[0], y[1], y[2]), y[3]);
          } else {
            mx = fmaf(fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])), c1[0], lv[0]);
          }
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
          uint64_t c2[G], a2[G], s0[G], s1[G];
          const float lift = m_ref == -INFINITY ? 0.f : kLift - m_ref;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float add = lv[g] + lift;
            c2[g] = f2pack(c1[g], c1[g]);
            a2[g] = f2pack(add, add);
            s0[g] = s1[g] = f2pack(0.f, 0.f);
          }
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = 32 * ch + 2 * e, g = SMALL ? i / 16 : 0;
              const float2 x = f2unpack(fma2(f2pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2[g], a2[g]));
              const float pa = ex2(x.x), pb = ex2(x.y);
              pk[e] = pack2(pa, pb, 0);
              if (e & 1) s1[g] = add2(s1[g], f2pack(pa, pb));
              else s0[g] = add2(s0[g], f2pack(pa, pb));
            }
            __syncwarp();
            tmem_st16(s_at + ch * 16, pk);
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float2 f0 = f2unpack(s0[g]), f1 = f2unpack(s1[g]);
            l = fmaf((f0.x + f0.y) + (f1.x + f1.y), over[g], l);
          }
          __syncwarp();
          tmem_st_wait();
          fence_before();
          mbar_arrive(bar(C::B_P + 2 * t + sb));
        }
        if (ok) ok = wait(C::B_O + 2 * t + ((ns - 1) & 1), (ns - 1) / 2);
        if (!ok) break;
        fence_after();
        // O through shared memory, 64 bytes of a row at a time, so that stores take whole rows: a lane writes its
        // row's in 16-byte pieces, swizzled by the row, and reads pieces of neighbouring lanes' rows
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float *part = p.part + (2ll * blockIdx.x + (x->flags & kFirst ? 1 : 0)) * C::PART;
        const uint32_t stage = base + C::OFF_STAGE + (warp - 12) * 2048;
        const bool all = (x->flags & kWhole) != 0;
        // four lanes have a row's 64 bytes, eight rows at a time: where this lane's four rows go (-1: nowhere)
        long long to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r2 = 8 * k + lane / 4, c2 = t * L + wr + r2;
          int row2, head2;
          to[k] = -1;
          if (wr + r2 < L && place(x, c2, row2, head2))
            to[k] = (all ? ((long long)(x->q0 + row2) * b.h_q + head2) * (2 * D) : (long long)c2 * (4 * D)) + 16 * (lane % 4);
        }
        uint8_t *const out = all ? static_cast<uint8_t *>(b.out) : reinterpret_cast<uint8_t *>(part);
        auto spread = [&](int at_col) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r2 = 8 * k + lane / 4;
            uint32_t y[4];
            lds_v4(stage + r2 * 64 + ((lane % 4 ^ (r2 >> 1 & 3)) << 4), y[0], y[1], y[2], y[3]);
            if (to[k] >= 0) *reinterpret_cast<uint4 *>(out + to[k] + at_col) = make_uint4(y[0], y[1], y[2], y[3]);
          }
          __syncwarp();
        };
        auto put = [&](int e, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
          sts_v4(stage + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4), x0, x1, x2, x3);
        };
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o_addr + i, o);
          tmem_ld_wait_for(o);
          if (all) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = pack2(l == 0.f ? 0.f : __uint_as_float(o[2 * e]) * inv, l == 0.f ? 0.f : __uint_as_float(o[2 * e + 1]) * inv, BF16);
#pragma unroll
            for (int e = 0; e < 4; ++e) put(e, pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            spread(2 * i);
          } else {
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2) {
#pragma unroll
              for (int e = 0; e < 4; ++e) put(e, o[16 * x2 + 4 * e], o[16 * x2 + 4 * e + 1], o[16 * x2 + 4 * e + 2], o[16 * x2 + 4 * e + 3]);
              spread(4 * (i + 16 * x2));
            }
          }
        }
        fence_before();
        mbar_arrive(bar(C::B_OE + t));
        int row, head;
        if (r < L && place(x, c, row, head)) {
          const float ref = m_ref - kLift;  // (minus infinity where no key was seen: l is 0 then)
          if (!all) {
            part[C::NC * D + c] = ref;
            part[C::NC * D + C::NC + c] = l;
          } else if (b.lse) {
            b.lse[(long long)head * b.total_q + x->q0 + row] = l == 0.f ? -INFINITY : (ref + lg2(l)) * kLn2;
          }
        }
      }
      done_item();
    }
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
  return (((size_t)num_sms * 2 * sizeof(int4) + 255) & ~(size_t)255) + 2 * (size_t)num_sms * part * sizeof(float);
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
    p.magic = magic_of(group);
    p.rec = static_cast<int4 *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + (((size_t)num_sms * 2 * sizeof(int4) + 255) & ~(size_t)255));
    const bool bf = a.p.dtype == VLF_BF16;
    const bool small = a.page < kN;
    const void *kern = bf ? (small ? (const void *)pages_rows_kernel<D, true, true> : (const void *)pages_rows_kernel<D, true, false>)
                          : (small ? (const void *)pages_rows_kernel<D, false, true> : (const void *)pages_rows_kernel<D, false, false>);
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
