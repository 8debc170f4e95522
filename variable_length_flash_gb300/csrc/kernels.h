// Host-side entry points of the kernel translation units (internal to libvlf.so).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace vlf {

// SIMT fp32-FMA kernels (simt.cu): every dtype and head width up to 256.
cudaError_t simt_forward(const Params &p, cudaStream_t st);
// Backward pre-pass: rowdot[h, row] = sum_c dO[row, h, c] * O[row, h, c] (simt.cu).
cudaError_t rowdot_forward(const Params &p, cudaStream_t st);
// ev: NULL or VLF_BWD_STAGES + 1 events recorded before the first and after each stage.
cudaError_t simt_backward(const Params &p, cudaStream_t st, const cudaEvent_t *ev);

// Tensor-core kernels (tc_fwd.cu / tc_bwd.cu).  `supported` says whether the shape has one.
bool tc_forward_supported(const Params &p);
cudaError_t tc_forward(const Params &p, cudaStream_t st);
// Split-KV forward (p.kv_splits > 1, p.o_part / p.lse_part set): the parts, then their combine.
// Only shapes with one query tile per CTA split (tc_forward_splittable).
bool tc_forward_splittable(const Params &p);
cudaError_t tc_forward_split(const Params &p, cudaStream_t st);
// The number of parts the library would cut each CTA's KV band into (1: no split), from the
// problem's launch shape and the device's SM count.
int fwd_num_splits(int num_seqs, int max_q, int max_kv, int h_q, int h_kv, int d_qk, int d_v,
                   int dtype, unsigned flags, int num_sms);
// fp32 inputs on the tensor cores, products in three tf32 passes (tc_fwd32.cu): head widths 32
// and 64.
bool tc_forward32_supported(const Params &p);
cudaError_t tc_forward32(const Params &p, cudaStream_t st);
bool tc_backward_supported(const Params &p);
// fp32 backward on the tensor cores, three tf32 passes (tc_bwd32.cu): head widths 32 and 64.
bool tc_backward32_supported(const Params &p);
cudaError_t tc_backward32(const Params &p, cudaStream_t st, const cudaEvent_t *ev);
cudaError_t tc_backward(const Params &p, cudaStream_t st, const cudaEvent_t *ev);
size_t tc_backward_workspace(int total_q, int h_q, int d_qk);

// Bias bands (bias_bands.cu): the buffer size, and the pass that fills it from p.bias.
size_t bias_bands_bytes(int total_q, int bias_heads);
cudaError_t bias_bands(const Params &p, void *bands, cudaStream_t st);

// ---------------------------------------------------------------- decoding on a bounded cache
// Rotary positions (rope.cu).  Strides in elements between tokens; heads and columns are dense.
struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  const int32_t *positions;  // [axes][total]
  const float *inv_freq;     // [rot / 2]
  int first[4];              // first pair of each axis (half for the axes that are not there)
  int total, h_q, h_k, d, rot, dtype, interleaved, inverse;
  int copy_tail;  // the columns behind rot have to be copied (not in place)
  int hpt;        // set by the launcher: heads per thread
};
cudaError_t rope(const RopeParams &p, cudaStream_t st);

// Norm of each head with the rotary positions in the same pass, and its gradients (norm_rope.cu).
struct Rows {  // of q or k; strides as above
  const void *x, *dy, *w;  // dy: backward; w: NULL (ones) or [d] of type w_dtype
  void *out, *dw;          // y, or dx; dw: backward, NULL or [d]
  long long x_stride, dy_stride, out_stride;
};
struct NormRopeParams {
  Rows q, k;
  const int32_t *positions;
  const float *inv_freq;
  float *part;  // backward: norm_rope_workspace(d) bytes where a dw is wanted, else NULL
  int first[4];
  int total, h_q, h_k, d, rot, dtype, w_dtype, interleaved;
  float eps;
  int lanes, hpt;  // set by the launcher: lanes of a token, heads of a lane
};
size_t norm_rope_workspace(int d);
cudaError_t norm_rope(const NormRopeParams &p, bool backward, cudaStream_t st);

// Attention over a shared prefix and each sequence's own keys (prefix.cu): p.k / p.v / p.cu_kv /
// p.total_kv / p.max_kv describe the own keys; the prefix is [prefix_len, h_kv, d].
struct PrefixParams {
  Params p;
  const void *k_pre, *v_pre;
  int prefix_len;
};
size_t prefix_workspace(int num_seqs, int total_q, int max_q, int max_kv, int prefix, int h_q, int h_kv, int d_qk,
                        int d_v, int dtype, unsigned flags, int num_sms);
cudaError_t prefix_forward(const PrefixParams &pp, void *workspace, int num_sms, cudaStream_t st);

// Attention weight received by each key (key_weights.cu).
struct KeyWeightParams {
  Params p;           // q, k, sequences, mask and scale
  const float *lse;   // [h_q, total_q]
  const float *prev;  // NULL or [h_kv, total_kv]
  float *weights;     // [h_kv, total_kv]
};
size_t key_weights_workspace(int num_seqs, int total_kv, int max_q, int max_kv, int h_q, int h_kv, int d,
                             int dtype, unsigned flags, int num_sms);
cudaError_t key_weights(const KeyWeightParams &kp, void *workspace, int num_sms, cudaStream_t st);

// Cache eviction (cache_evict.cu).
struct EvictParams {
  const void *k, *v;
  const float *weights;  // [h_kv, total_kv]
  const int32_t *cu_kv;
  int num_seqs, total_kv, max_kv, h_kv, d_qk, d_v, dtype, budget, sink, recent, total_out;
  void *k_out, *v_out;
  float *weights_out;  // [h_kv, total_out]
  int *index;          // [h_kv, total_out]
  int *cu_out;         // [num_seqs + 1]
  int *err;
};
cudaError_t cache_evict(const EvictParams &p, cudaStream_t st);

// A cache of pages in e4m3 (pages.cu): k_pages [num_pages][h_kv][page][d_qk], scales [num_pages][h_kv].
struct PagesWriteParams {
  const void *k, *v;              // [total][h_kv][d]
  long long k_stride, v_stride;   // elements between tokens
  void *k_pages, *v_pages;
  float *k_scale, *v_scale;
  const int32_t *table;           // [num_seqs][max_pages]
  const int32_t *cu, *kv_lens;    // new tokens [num_seqs + 1], lengths with them [num_seqs]
  int num_seqs, total, max_pages, num_pages, page, log2_page, h_kv, d_qk, d_v, dtype;
  int *err;
};
cudaError_t pages_write(const PagesWriteParams &p, cudaStream_t st);

struct PagesCopyParams {
  void *k_pages, *v_pages;
  float *k_scale, *v_scale;
  const int32_t *src, *dst;  // [n]; src < 0: no copy
  int n, num_pages, page, h_kv, d_qk, d_v;
  int *err;
  int chunk;  // set by the launcher: pairs per block
};
cudaError_t pages_copy(PagesCopyParams p, cudaStream_t st);

struct PagesForkParams {
  const int32_t *table, *lens, *refs, *parents, *grow;
  int num_in, num_out, max_pages, num_pages, log2_page;
  int *table_out, *lens_out, *refs_out, *src, *dst, *left;
  int *err;
  // workspace
  int *outside, *whole, *owner, *list, *counts, *need, *group, *state, chunks;
};
size_t pages_fork_workspace(int num_pages, int num_out);
cudaError_t pages_fork(PagesForkParams p, void *workspace, cudaStream_t st);

struct PagesCompactParams {
  const int32_t *table, *refs;
  long long entries;  // of the table
  int num_pages;
  int *table_out, *refs_out, *to, *src, *dst, *used;
  // workspace
  int *counts, *order, chunks;
};
size_t pages_compact_workspace(int num_pages);
cudaError_t pages_compact(PagesCompactParams p, void *workspace, cudaStream_t st);

// Attention over it (pages_attn.cu): p.q, p.cu_q, sizes, mask, scale, out and lse as in the forward.
struct PagesAttnParams {
  Params p;
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *table, *kv_lens;
  int max_pages, num_pages, page, log2_page;
};
size_t pages_attn_workspace(int num_seqs, int max_q, int h_q, int h_kv, int d_qk, int d_v, int dtype, unsigned flags,
                            int num_sms);
cudaError_t pages_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st);
// Its tensor-core kernels (pages_tc.cu).
bool pages_tc_supported(int d_qk, int d_v, int dtype, unsigned flags);
size_t pages_tc_workspace(int max_q, int group, int d, int num_sms);
cudaError_t pages_tc_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st);
// The ones for many rows (pages_rows.cu).
size_t pages_rows_workspace(int d, int num_sms);
cudaError_t pages_rows_forward(const PagesAttnParams &a, void *workspace, int num_sms, cudaStream_t st);

// Host-side count of successful kernel launches (api.cu).
void count_launch(int n = 1);
// cudaFuncSetAttribute(kern, MaxDynamicSharedMemorySize, bytes), made once per (kernel, device)
// and raised only when a launch needs more: the runtime call costs microseconds of host time,
// which small problems would pay on every launch.
cudaError_t set_smem_once(const void *kern, int bytes);

// A launch that reports its own error and leaves none behind for a later check.
inline cudaError_t launch_plain(const void *kern, dim3 grid, int threads, int smem, cudaStream_t st, void **args) {
  const cudaError_t e = cudaLaunchKernel(kern, grid, dim3(threads), args, (size_t)smem, st);
  if (e != cudaSuccess) cudaGetLastError();
  else count_launch();
  return e;
}

// Records ev[i] on st when ev is not NULL.
inline cudaError_t mark(const cudaEvent_t *ev, int i, cudaStream_t st) {
  return ev ? cudaEventRecord(ev[i], st) : cudaSuccess;
}

}  // namespace vlf
