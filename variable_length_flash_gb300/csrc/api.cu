// C ABI of libvlf.so (declared in include/vlf.h): argument checks, dispatch to the kernels,
// and the per-device error word that the kernels write instead of trapping.
#include <math.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

// One error word per device (module-scope __device__ variable; each device that loads the
// library holds its own copy).  Kernels get its address through Params::err.  The address is
// looked up once per device and kept for the life of the process; it is not valid after a
// cudaDeviceReset of that device.
__device__ int g_vlf_error_word = 0;

namespace vlf {
static std::atomic<uint64_t> g_launches{0};
void count_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

cudaError_t set_smem_once(const void *kern, int bytes) {
  struct Entry {
    const void *kern;
    int dev, bytes;
  };
  // per host thread (no lock on the launch path): a thread that has not set a kernel's limit
  // itself sets it once more, which is harmless
  thread_local Entry table[256];
  thread_local int n_entries = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n_entries; ++i)
    if (table[i].kern == kern && table[i].dev == dev) {
      if (bytes <= table[i].bytes) return cudaSuccess;
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e == cudaSuccess) table[i].bytes = bytes;
      return e;
    }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && n_entries < 256) table[n_entries++] = Entry{kern, dev, bytes};
  return e;
}
}  // namespace vlf

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int *g_err_ptr[kMaxDevices] = {nullptr};

int *error_word_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  // the last device's address, per host thread, skips the lock on repeated calls
  thread_local int t_dev = -1;
  thread_local int *t_ptr = nullptr;
  if (dev == t_dev) return t_ptr;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_err_ptr[dev]) {
    void *ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_vlf_error_word) != cudaSuccess) return nullptr;
    g_err_ptr[dev] = static_cast<int *>(ptr);
  }
  t_dev = dev;
  t_ptr = g_err_ptr[dev];
  return t_ptr;
}

// The current device's SM count (looked up once per device and host thread); 0 if that fails.
int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  thread_local int count[kMaxDevices] = {0};
  if (!count[dev] && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    count[dev] = 0;
  return count[dev];
}

// The decoding entry points' kernels step over rows and keys with ints, a few tiles past the end at
// most: they take fewer than 2^31 - 2^16 of them.
constexpr long long kMostTokens = 0x7fff0000ll;

// The first pair of each position axis (half for the axes that are not there); false where the sections
// are not `half` pairs in all.
bool first_pairs(int (&first)[4], int n_axes, const int *sections, int half) {
  long long sum = 0;
  for (int a = 0; a < 4; ++a) {
    first[a] = a < n_axes ? (int)sum : half;
    if (a >= n_axes) continue;
    const int n = sections ? sections[a] : half;
    if (n < 0 || (sum += n) > half) return false;
  }
  return sum == half;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether one of the first `outs` of n spans shares a byte with any other.
struct Span {
  const void *p;
  size_t n;
};
bool overlap(const Span *all, int outs, int n) {
  for (int a = 0; a < outs; ++a)
    for (int b = a + 1; b < n; ++b) {
      const uintptr_t x = (uintptr_t)all[a].p, y = (uintptr_t)all[b].p;
      if (all[a].n && all[b].n && x < y + all[b].n && y < x + all[a].n) return true;
    }
  return false;
}

// Shared argument checks of the forward and backward.  Returns VLF_OK or a negative status.
int check_common(const void *q, const void *k, const void *v, const int32_t *cu_q,
                 const int32_t *cu_kv, int num_seqs, int total_q, int total_kv, int max_q,
                 int max_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype, const float *bias,
                 int bias_heads) {
  if (num_seqs < 0 || total_q < 0 || total_kv < 0 || max_q < 0 || max_kv < 0) return VLF_ERR_INVALID;
  if (h_q < 1 || h_kv < 1 || h_q % h_kv != 0) return VLF_ERR_INVALID;
  if (d_qk < 1 || d_v < 1) return VLF_ERR_INVALID;
  if (dtype != VLF_F16 && dtype != VLF_BF16 && dtype != VLF_F32) return VLF_ERR_INVALID;
  if (num_seqs == 0 && (total_q != 0 || total_kv != 0)) return VLF_ERR_INVALID;
  if (num_seqs > 0 && (!cu_q || !cu_kv)) return VLF_ERR_INVALID;
  if ((total_q > 0 && !q) || (total_kv > 0 && (!k || !v))) return VLF_ERR_INVALID;
  if (bias && bias_heads != 1 && bias_heads != h_q) return VLF_ERR_INVALID;
  if (d_qk > 256 || d_v > 256) return VLF_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || h_q > 65535) return VLF_ERR_UNSUPPORTED;
  // row strides of 16-bit data must keep 16-byte alignment for vector / TMA access
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cu_q) || !aligned16(cu_kv) ||
      !aligned16(bias))
    return VLF_ERR_ALIGN;
  return VLF_OK;
}

void fill_common(vlf::Params &p, const void *q, const void *k, const void *v, const int32_t *cu_q,
                 const int32_t *cu_kv, int num_seqs, int total_q, int total_kv, int max_q,
                 int max_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype, float scale,
                 int causal, int window, const float *bias, int bias_heads, unsigned flags) {
  p = vlf::Params{};
  p.q = q; p.k = k; p.v = v; p.cu_q = cu_q; p.cu_kv = cu_kv;
  p.num_seqs = num_seqs; p.total_q = total_q; p.total_kv = total_kv;
  p.max_q = max_q; p.max_kv = max_kv;
  p.h_q = h_q; p.h_kv = h_kv; p.d_qk = d_qk; p.d_v = d_v; p.group = h_q / h_kv;
  p.dtype = dtype;
  p.scale = scale > 0.f ? scale : (float)(1.0 / sqrt((double)d_qk));
  p.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
  p.causal = causal ? 1 : 0;
  p.window = window > 0 ? window : 0;
  p.bias = bias; p.bias_heads = bias ? bias_heads : 0;
  p.flags = flags;
}

// The bias bands' two tables in the caller's buffer (vlf_bias_bands): rows, then blocks.
void attach_bands(vlf::Params &p, const void *bands) {
  if (!bands || !p.bias || p.total_q <= 0) return;
  p.bias_rows = static_cast<const int4 *>(bands);
  p.bias_blocks = p.bias_rows + (size_t)p.total_q * (size_t)p.bias_heads;
}

size_t workspace_bytes_for(int total_q, int h_q, int d_qk, int dtype) {
  if (total_q < 0 || h_q < 1 || d_qk < 1) return 0;
  size_t rowdot = (size_t)h_q * (size_t)total_q * sizeof(float);
  rowdot = (rowdot + 255) & ~(size_t)255;
  if (dtype == VLF_F32) return rowdot;
  return rowdot + vlf::tc_backward_workspace(total_q, h_q, d_qk);
}

// Checks shared by the split-operand latent entry points (beyond check_common on the nope
// tensors): the rope tensors, rope_heads, and the one head shape with a kernel.
int check_latent(const void *q_rope, const void *k_rope, int total_q, int total_kv, int h_kv,
                 int rope_heads, int d_nope, int d_rope, int d_v, int dtype, unsigned flags) {
  if ((total_q > 0 && !q_rope) || (total_kv > 0 && !k_rope)) return VLF_ERR_INVALID;
  if (rope_heads != 1 && rope_heads != h_kv) return VLF_ERR_INVALID;
  if (!aligned16(q_rope) || !aligned16(k_rope)) return VLF_ERR_ALIGN;
  if (d_nope != 128 || d_rope != 64 || d_v != 128) return VLF_ERR_UNSUPPORTED;
  if ((dtype != VLF_F16 && dtype != VLF_BF16) || (flags & VLF_FLAG_FORCE_SIMT)) return VLF_ERR_UNSUPPORTED;
  return VLF_OK;
}

size_t latent_rope_part_bytes(int total_kv, int h_kv, int rope_heads) {
  if (rope_heads != 1 || h_kv <= 1 || total_kv <= 0) return 0;
  return ((size_t)h_kv * (size_t)total_kv * 64 * sizeof(float) + 255) & ~(size_t)255;
}

__global__ void fill_f32_kernel(float *p, size_t n, float v) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = v;
}

// The unsplit forward: the 16-bit tensor-core kernels, the fp32 three-pass tf32 kernel, or the
// SIMT fp32-FMA kernels (forced by VLF_FLAG_FORCE_SIMT, and for shapes without a tensor-core one).
cudaError_t forward_dispatch(const vlf::Params &p, cudaStream_t cs) {
  if (!(p.flags & VLF_FLAG_FORCE_SIMT)) {
    if (vlf::tc_forward_supported(p)) return vlf::tc_forward(p, cs);
    if (vlf::tc_forward32_supported(p)) return vlf::tc_forward32(p, cs);
  }
  return vlf::simt_forward(p, cs);
}

cudaError_t zero16(void *p, size_t elems, cudaStream_t st) {
  return elems && p ? cudaMemsetAsync(p, 0, elems * 2, st) : cudaSuccess;
}

}  // namespace

extern "C" {

int vlf_version(void) { return 100; }

uint64_t vlf_launch_count(void) { return vlf::g_launches.load(std::memory_order_relaxed); }

static vlf::Params shape_params(int h_q, int h_kv, int d_qk, int d_v, int dtype, int bias_heads,
                                unsigned flags) {
  vlf::Params p{};
  p.h_q = h_q; p.h_kv = h_kv; p.d_qk = d_qk; p.d_v = d_v; p.dtype = dtype;
  p.group = h_kv > 0 ? h_q / h_kv : 0;
  p.bias_heads = bias_heads;
  p.flags = flags;
  return p;
}

int vlf_fwd_path(int h_q, int h_kv, int d_qk, int d_v, int dtype, int bias_heads, unsigned flags) {
  if (h_q < 1 || h_kv < 1 || h_q % h_kv || d_qk < 1 || d_v < 1 || dtype < 0 || dtype > 2)
    return VLF_ERR_INVALID;
  if (d_qk > 256 || d_v > 256) return VLF_ERR_UNSUPPORTED;
  vlf::Params p = shape_params(h_q, h_kv, d_qk, d_v, dtype, bias_heads, flags);
  return (!(flags & VLF_FLAG_FORCE_SIMT) &&
          (vlf::tc_forward_supported(p) || vlf::tc_forward32_supported(p))) ? 1 : 0;
}

int vlf_bwd_path(int h_q, int h_kv, int d_qk, int d_v, int dtype, int bias_heads, unsigned flags) {
  if (h_q < 1 || h_kv < 1 || h_q % h_kv || d_qk < 1 || d_v < 1 || dtype < 0 || dtype > 2)
    return VLF_ERR_INVALID;
  if (d_qk > 256 || d_v > 256) return VLF_ERR_UNSUPPORTED;
  vlf::Params p = shape_params(h_q, h_kv, d_qk, d_v, dtype, bias_heads, flags);
  return (!(flags & VLF_FLAG_FORCE_SIMT) &&
          (vlf::tc_backward_supported(p) || vlf::tc_backward32_supported(p))) ? 1 : 0;
}

const char *vlf_status_string(int status) {
  switch (status) {
    case VLF_OK: return "ok";
    case VLF_ERR_INVALID: return "invalid argument";
    case VLF_ERR_UNSUPPORTED: return "unsupported problem (dtype / head width / size)";
    case VLF_ERR_ALIGN: return "pointer not 16-byte aligned";
    case VLF_ERR_LAUNCH: return "CUDA launch or runtime error";
    case VLF_ERR_TIMEOUT: return "device pipeline wait timed out";
    case VLF_ERR_BAD_SEQLENS: return "bad cu_seqlens (out of range, decreasing, or longer than max_seqlen)";
    case VLF_ERR_WORKSPACE: return "backward workspace missing or too small";
    case VLF_ERR_BAD_PAGES: return "bad pages (outside the pool, or tables and counts that disagree)";
    default: return "unknown status";
  }
}

int vlf_sched_kv_band(int r0, int r1, int q_len, int kv_len, int causal, int window, int *lo,
                      int *hi) {
  if (!lo || !hi || q_len < 0 || kv_len < 0 || r0 < 0 || r1 <= r0 || r1 > q_len) return VLF_ERR_INVALID;
  vlf::kv_band(r0, r1, q_len, kv_len, causal, window, *lo, *hi);
  return VLF_OK;
}

int vlf_sched_q_band(int j0, int j1, int q_len, int kv_len, int causal, int window, int *lo,
                     int *hi) {
  if (!lo || !hi || q_len < 0 || kv_len < 0 || j0 < 0 || j1 <= j0 || j1 > kv_len) return VLF_ERR_INVALID;
  vlf::q_band(j0, j1, q_len, kv_len, causal, window, *lo, *hi);
  return VLF_OK;
}

int vlf_attn_varlen_fwd_ex(const void *q, const void *k, const void *v,
                           const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                           int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv,
                           int h_q, int h_kv, int d_qk, int d_v, int dtype, float scale,
                           int causal, int window, const float *bias, int bias_heads, void *out,
                           float *lse, vlf_stream_t stream, unsigned flags,
                           const void *bias_bands) {
  int st = check_common(q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                        max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, bias, bias_heads);
  if (st != VLF_OK) return st;
  if (total_q > 0 && !out) return VLF_ERR_INVALID;
  if (!aligned16(out) || !aligned16(lse)) return VLF_ERR_ALIGN;
  if (num_seqs == 0 || max_seqlen_q == 0) return VLF_OK;
  vlf::Params p;
  fill_common(p, q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv, max_seqlen_q,
              max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, scale, causal, window, bias, bias_heads,
              flags);
  p.out = out;
  p.lse = lse;
  if (!aligned16(bias_bands)) return VLF_ERR_ALIGN;
  attach_bands(p, bias_bands);
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = forward_dispatch(p, cs);
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

int vlf_attn_varlen_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens_q,
                        const int32_t *cu_seqlens_kv, int num_seqs, int total_q, int total_kv,
                        int max_seqlen_q, int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v,
                        int dtype, float scale, int causal, int window, const float *bias,
                        int bias_heads, void *out, float *lse, vlf_stream_t stream) {
  return vlf_attn_varlen_fwd_ex(q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                                max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, scale,
                                causal, window, bias, bias_heads, out, lse, stream, 0u, nullptr);
}

int vlf_fwd_num_splits(int num_seqs, int max_seqlen_q, int max_seqlen_kv, int h_q, int h_kv,
                       int d_qk, int d_v, int dtype, unsigned flags, int num_sms) {
  if (num_sms <= 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 1;
  }
  return vlf::fwd_num_splits(num_seqs, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype,
                             flags, num_sms);
}

size_t vlf_attn_varlen_fwd_split_workspace_size(int total_q, int h_q, int d_v, int num_splits) {
  if (total_q < 0 || h_q < 1 || d_v < 1 || num_splits < 2) return 0;
  const size_t rows = (size_t)num_splits * (size_t)total_q * (size_t)h_q;
  const size_t o = (rows * (size_t)d_v * sizeof(float) + 255) & ~(size_t)255;
  return o + ((rows * sizeof(float) + 255) & ~(size_t)255);
}

int vlf_attn_varlen_fwd_split(const void *q, const void *k, const void *v,
                              const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                              int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                              int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype,
                              float scale, int causal, int window, const float *bias,
                              int bias_heads, void *out, float *lse, int num_splits,
                              void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                              unsigned flags, const void *bias_bands) {
  int st = check_common(q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                        max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, bias, bias_heads);
  if (st != VLF_OK) return st;
  if (num_splits < 0) return VLF_ERR_INVALID;
  if (total_q > 0 && !out) return VLF_ERR_INVALID;
  if (!aligned16(out) || !aligned16(lse) || !aligned16(workspace) || !aligned16(bias_bands))
    return VLF_ERR_ALIGN;
  if (num_seqs == 0 || max_seqlen_q == 0) return VLF_OK;
  vlf::Params p;
  fill_common(p, q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv, max_seqlen_q,
              max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, scale, causal, window, bias, bias_heads,
              flags);
  p.out = out;
  p.lse = lse;
  attach_bands(p, bias_bands);
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  if (num_splits == 0)
    num_splits = vlf_fwd_num_splits(num_seqs, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v,
                                    dtype, flags, 0);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (num_splits >= 2 && !(flags & VLF_FLAG_FORCE_SIMT) && vlf::tc_forward_splittable(p)) {
    if (num_splits > 64 || (long long)num_splits * num_seqs > 65535) return VLF_ERR_UNSUPPORTED;
    const size_t need = vlf_attn_varlen_fwd_split_workspace_size(total_q, h_q, d_v, num_splits);
    if (!workspace || workspace_bytes < need) return VLF_ERR_WORKSPACE;
    const size_t rows = (size_t)num_splits * (size_t)total_q * (size_t)h_q;
    p.kv_splits = num_splits;
    p.o_part = static_cast<float *>(workspace);
    p.lse_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                           ((rows * (size_t)d_v * sizeof(float) + 255) & ~(size_t)255));
    e = vlf::tc_forward_split(p, cs);
  } else {
    e = forward_dispatch(p, cs);
  }
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_attn_varlen_bwd_workspace_size(int total_q, int total_kv, int h_q, int h_kv, int d_qk,
                                          int d_v, int dtype) {
  (void)total_kv; (void)h_kv; (void)d_v;
  return workspace_bytes_for(total_q, h_q, d_qk, dtype);
}

int vlf_attn_varlen_bwd_ex(const void *q, const void *k, const void *v, const void *out,
                           const float *lse, const void *dout, const int32_t *cu_seqlens_q,
                           const int32_t *cu_seqlens_kv, int num_seqs, int total_q, int total_kv,
                           int max_seqlen_q, int max_seqlen_kv, int h_q, int h_kv, int d_qk,
                           int d_v, int dtype, float scale, int causal, int window,
                           const float *bias, int bias_heads, void *dq, void *dk, void *dv,
                           void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                           unsigned flags, void *const *stage_events, int n_stage_events,
                           const void *bias_bands) {
  if (stage_events && n_stage_events < VLF_BWD_STAGES + 1) return VLF_ERR_INVALID;
  int st = check_common(q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                        max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, bias, bias_heads);
  if (st != VLF_OK) return st;
  if (total_q > 0 && (!out || !lse || !dout || !dq)) return VLF_ERR_INVALID;
  if (total_kv > 0 && (!dk || !dv)) return VLF_ERR_INVALID;
  if (!aligned16(out) || !aligned16(lse) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) ||
      !aligned16(dv) || !aligned16(workspace) || !aligned16(bias_bands))
    return VLF_ERR_ALIGN;
  const size_t need = workspace_bytes_for(total_q, h_q, d_qk, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return VLF_ERR_WORKSPACE;
  if (num_seqs == 0) return VLF_OK;
  vlf::Params p;
  fill_common(p, q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv, max_seqlen_q,
              max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, scale, causal, window, bias, bias_heads,
              flags);
  const cudaEvent_t *ev = reinterpret_cast<const cudaEvent_t *>(stage_events);
  p.out = const_cast<void *>(out);
  p.lse = const_cast<float *>(lse);
  p.dout = dout;
  p.dq = dq; p.dk = dk; p.dv = dv;
  p.rowdot = static_cast<float *>(workspace);
  p.dq_acc = nullptr;
  attach_bands(p, bias_bands);
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!(flags & VLF_FLAG_FORCE_SIMT) && vlf::tc_backward_supported(p))
    e = vlf::tc_backward(p, cs, ev);
  else if (!(flags & VLF_FLAG_FORCE_SIMT) && vlf::tc_backward32_supported(p))
    e = vlf::tc_backward32(p, cs, ev);
  else
    e = vlf::simt_backward(p, cs, ev);
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

int vlf_attn_varlen_bwd(const void *q, const void *k, const void *v, const void *out,
                        const float *lse, const void *dout, const int32_t *cu_seqlens_q,
                        const int32_t *cu_seqlens_kv, int num_seqs, int total_q, int total_kv,
                        int max_seqlen_q, int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v,
                        int dtype, float scale, int causal, int window, const float *bias,
                        int bias_heads, void *dq, void *dk, void *dv, void *workspace,
                        size_t workspace_bytes, vlf_stream_t stream) {
  return vlf_attn_varlen_bwd_ex(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_kv, num_seqs,
                                total_q, total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk,
                                d_v, dtype, scale, causal, window, bias, bias_heads, dq, dk, dv,
                                workspace, workspace_bytes, stream, 0u, nullptr, 0, nullptr);
}

int vlf_attn_varlen_fwd_latent(const void *q_nope, const void *q_rope, const void *k_nope,
                               const void *k_rope, const void *v, const int32_t *cu_seqlens_q,
                               const int32_t *cu_seqlens_kv, int num_seqs, int total_q,
                               int total_kv, int max_seqlen_q, int max_seqlen_kv, int h_q,
                               int h_kv, int rope_heads, int d_nope, int d_rope, int d_v,
                               int dtype, float scale, int causal, int window, const float *bias,
                               int bias_heads, void *out, float *lse, vlf_stream_t stream,
                               unsigned flags) {
  int st = check_common(q_nope, k_nope, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q,
                        total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_nope + d_rope, d_v,
                        dtype, bias, bias_heads);
  if (st != VLF_OK) return st;
  st = check_latent(q_rope, k_rope, total_q, total_kv, h_kv, rope_heads, d_nope, d_rope, d_v, dtype, flags);
  if (st != VLF_OK) return st;
  if (total_q > 0 && !out) return VLF_ERR_INVALID;
  if (!aligned16(out) || !aligned16(lse)) return VLF_ERR_ALIGN;
  if (num_seqs == 0 || max_seqlen_q == 0 || total_q == 0) return VLF_OK;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (total_kv == 0) {  // no keys anywhere: O = 0, LSE = -inf
    e = zero16(out, (size_t)total_q * h_q * d_v, cs);
    if (e == cudaSuccess && lse) {
      const size_t n = (size_t)total_q * h_q;
      fill_f32_kernel<<<(unsigned)((n + 255) / 256), 256, 0, cs>>>(lse, n, -INFINITY);
      e = cudaGetLastError();
      if (e == cudaSuccess) vlf::count_launch();
    }
    return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
  }
  vlf::Params p;
  fill_common(p, q_nope, k_nope, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
              max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_nope + d_rope, d_v, dtype, scale, causal,
              window, bias, bias_heads, flags);
  p.latent = 1;
  p.q_rope = q_rope;
  p.k_rope = k_rope;
  p.rope_heads = rope_heads;
  p.out = out;
  p.lse = lse;
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  e = vlf::tc_forward(p, cs);
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_attn_varlen_bwd_latent_workspace_size(int total_q, int total_kv, int h_q, int h_kv,
                                                 int rope_heads, int dtype) {
  if (total_q < 0 || total_kv < 0 || h_q < 1 || h_kv < 1) return 0;
  return workspace_bytes_for(total_q, h_q, 192, dtype) +
         latent_rope_part_bytes(total_kv, h_kv, rope_heads);
}

int vlf_attn_varlen_bwd_latent(const void *q_nope, const void *q_rope, const void *k_nope,
                               const void *k_rope, const void *v, const void *out,
                               const float *lse, const void *dout, const int32_t *cu_seqlens_q,
                               const int32_t *cu_seqlens_kv, int num_seqs, int total_q,
                               int total_kv, int max_seqlen_q, int max_seqlen_kv, int h_q,
                               int h_kv, int rope_heads, int d_nope, int d_rope, int d_v,
                               int dtype, float scale, int causal, int window, const float *bias,
                               int bias_heads, void *dq_nope, void *dq_rope, void *dk_nope,
                               void *dk_rope, void *dv, void *workspace, size_t workspace_bytes,
                               vlf_stream_t stream, unsigned flags, void *const *stage_events,
                               int n_stage_events) {
  if (stage_events && n_stage_events < VLF_BWD_STAGES + 1) return VLF_ERR_INVALID;
  int st = check_common(q_nope, k_nope, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q,
                        total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_nope + d_rope, d_v,
                        dtype, bias, bias_heads);
  if (st != VLF_OK) return st;
  st = check_latent(q_rope, k_rope, total_q, total_kv, h_kv, rope_heads, d_nope, d_rope, d_v, dtype, flags);
  if (st != VLF_OK) return st;
  if (total_q > 0 && (!out || !lse || !dout || !dq_nope || !dq_rope)) return VLF_ERR_INVALID;
  if (total_kv > 0 && (!dk_nope || !dk_rope || !dv)) return VLF_ERR_INVALID;
  if (!aligned16(out) || !aligned16(lse) || !aligned16(dout) || !aligned16(dq_nope) ||
      !aligned16(dq_rope) || !aligned16(dk_nope) || !aligned16(dk_rope) || !aligned16(dv) ||
      !aligned16(workspace))
    return VLF_ERR_ALIGN;
  const size_t rowdot_bytes = workspace_bytes_for(total_q, h_q, 192, dtype);
  const size_t need = rowdot_bytes + latent_rope_part_bytes(total_kv, h_kv, rope_heads);
  if (need > 0 && (!workspace || workspace_bytes < need)) return VLF_ERR_WORKSPACE;
  if (num_seqs == 0) return VLF_OK;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (total_q == 0 || total_kv == 0) {  // nothing attends: every gradient is zero
    cudaError_t e = zero16(dq_nope, (size_t)total_q * h_q * d_nope, cs);
    if (e == cudaSuccess) e = zero16(dq_rope, (size_t)total_q * h_q * d_rope, cs);
    if (e == cudaSuccess) e = zero16(dk_nope, (size_t)total_kv * h_kv * d_nope, cs);
    if (e == cudaSuccess) e = zero16(dk_rope, (size_t)total_kv * rope_heads * d_rope, cs);
    if (e == cudaSuccess) e = zero16(dv, (size_t)total_kv * h_kv * d_v, cs);
    return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
  }
  vlf::Params p;
  fill_common(p, q_nope, k_nope, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
              max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_nope + d_rope, d_v, dtype, scale, causal,
              window, bias, bias_heads, flags);
  p.latent = 1;
  p.q_rope = q_rope;
  p.k_rope = k_rope;
  p.rope_heads = rope_heads;
  p.out = const_cast<void *>(out);
  p.lse = const_cast<float *>(lse);
  p.dout = dout;
  p.dq = dq_nope; p.dk = dk_nope; p.dv = dv;
  p.dq_rope = dq_rope; p.dk_rope = dk_rope;
  p.rowdot = static_cast<float *>(workspace);
  if (latent_rope_part_bytes(total_kv, h_kv, rope_heads) > 0)
    p.dk_rope_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + rowdot_bytes);
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  cudaError_t e = vlf::tc_backward(p, cs, reinterpret_cast<const cudaEvent_t *>(stage_events));
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_bias_bands_size(int total_q, int bias_heads) {
  return vlf::bias_bands_bytes(total_q, bias_heads);
}

int vlf_bias_bands(const float *bias, int bias_heads, const int32_t *cu_seqlens_q,
                   const int32_t *cu_seqlens_kv, int num_seqs, int total_q, int max_seqlen_kv,
                   void *bands, size_t bands_bytes, vlf_stream_t stream) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_kv < 0 || bias_heads < 1) return VLF_ERR_INVALID;
  if (num_seqs > 65535) return VLF_ERR_UNSUPPORTED;
  if (total_q == 0) return VLF_OK;
  if (!bias || num_seqs == 0 || !cu_seqlens_q || !cu_seqlens_kv) return VLF_ERR_INVALID;
  if (!aligned16(bias) || !aligned16(bands) || !aligned16(cu_seqlens_q) || !aligned16(cu_seqlens_kv))
    return VLF_ERR_ALIGN;
  if (!bands || bands_bytes < vlf::bias_bands_bytes(total_q, bias_heads)) return VLF_ERR_WORKSPACE;
  vlf::Params p{};
  p.bias = bias;
  p.bias_heads = bias_heads;
  p.cu_q = cu_seqlens_q;
  p.cu_kv = cu_seqlens_kv;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_kv = max_seqlen_kv;
  const cudaError_t e = vlf::bias_bands(p, bands, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

int vlf_check_error(vlf_stream_t stream) {
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(cs) != cudaSuccess) return VLF_ERR_LAUNCH;
  int *ptr = error_word_ptr();
  if (!ptr) return VLF_ERR_LAUNCH;
  int word = 0;
  if (cudaMemcpy(&word, ptr, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return VLF_ERR_LAUNCH;
  if (word != 0) {
    const int zero = 0;
    if (cudaMemcpy(ptr, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return VLF_ERR_LAUNCH;
  }
  if (cudaGetLastError() != cudaSuccess) return VLF_ERR_LAUNCH;
  return word;
}

int vlf_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
             const int32_t *positions, int n_axes, const int *sections, const float *inv_freq,
             int total, int h_q, int h_k, int d, int rot, int dtype, int interleaved, int inverse,
             void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
             vlf_stream_t stream) {
  if (total < 0 || h_q < 1 || h_k < 0 || d < 1 || rot < 0 || rot > d || rot % 2) return VLF_ERR_INVALID;
  if (dtype != VLF_F16 && dtype != VLF_BF16 && dtype != VLF_F32) return VLF_ERR_INVALID;
  if (n_axes < 1 || n_axes > 4 || (!sections && n_axes != 1)) return VLF_ERR_INVALID;
  vlf::RopeParams p{};
  const int half = rot / 2;
  if (!first_pairs(p.first, n_axes, sections, half)) return VLF_ERR_INVALID;
  if (d > 256 || h_q > 65535 || h_k > 65535) return VLF_ERR_UNSUPPORTED;
  if (total == 0) return VLF_OK;
  if (!q || !q_out || (h_k > 0 && (!k || !k_out)) || (half > 0 && (!positions || !inv_freq))) return VLF_ERR_INVALID;
  const int64_t nq = (int64_t)h_q * d, nk = (int64_t)h_k * d;
  if (q_stride < 0 || k_stride < 0 || (total > 1 && (q_out_stride < nq || (h_k > 0 && k_out_stride < nk))))
    return VLF_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(positions) ||
      !aligned16(inv_freq))
    return VLF_ERR_ALIGN;
  // in place: the same elements, or none
  if ((q == q_out && total > 1 && q_stride != q_out_stride) ||
      (h_k > 0 && k == k_out && total > 1 && k_stride != k_out_stride))
    return VLF_ERR_INVALID;
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.q_stride = q_stride; p.k_stride = k_stride; p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
  p.positions = positions; p.inv_freq = inv_freq;
  p.total = total; p.h_q = h_q; p.h_k = h_k; p.d = d; p.rot = rot; p.dtype = dtype;
  p.interleaved = interleaved ? 1 : 0; p.inverse = inverse ? 1 : 0;
  p.copy_tail = rot < d && (q != q_out || (h_k > 0 && k != k_out));
  return vlf::rope(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_attn_varlen_fwd_prefix_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                                 int max_seqlen_kv, int prefix_len, int h_q,
                                                 int h_kv, int d_qk, int d_v, int dtype,
                                                 unsigned flags, int num_sms) {
  if (num_sms <= 0) num_sms = sm_count();
  if (max_seqlen_q > total_q) max_seqlen_q = total_q;  // (as in the call)
  return vlf::prefix_workspace(num_seqs, total_q, max_seqlen_q, max_seqlen_kv, prefix_len, h_q, h_kv, d_qk,
                               d_v, dtype, flags, num_sms);
}

int vlf_attn_varlen_fwd_prefix(const void *q, const void *k_prefix, const void *v_prefix,
                               int prefix_len, const void *k, const void *v,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                               int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                               int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype,
                               float scale, int causal, int window, void *out, float *lse,
                               void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                               unsigned flags) {
  int st = check_common(q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                        max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, nullptr, 0);
  if (st != VLF_OK) return st;
  if (prefix_len < 0 || (prefix_len > 0 && (!k_prefix || !v_prefix))) return VLF_ERR_INVALID;
  if (total_q > 0 && !out) return VLF_ERR_INVALID;
  const long long own = max_seqlen_kv < total_kv ? max_seqlen_kv : total_kv;  // (no sequence has more keys)
  if (total_q >= kMostTokens || total_kv >= kMostTokens || prefix_len + own >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
    return VLF_ERR_ALIGN;
  if (num_seqs == 0 || max_seqlen_q == 0) return VLF_OK;
  if (total_q > 0 && max_seqlen_q > total_q) max_seqlen_q = total_q;  // (no sequence has more)
  vlf::PrefixParams pp{};
  fill_common(pp.p, q, k, v, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv, max_seqlen_q,
              max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype, scale, causal, window, nullptr, 0, flags);
  pp.p.out = out;
  pp.p.lse = lse;
  pp.p.err = error_word_ptr();
  if (!pp.p.err) return VLF_ERR_LAUNCH;
  pp.k_pre = k_prefix;
  pp.v_pre = v_prefix;
  pp.prefix_len = prefix_len;
  const int sms = sm_count();
  const size_t need = vlf::prefix_workspace(num_seqs, total_q, max_seqlen_q, max_seqlen_kv, prefix_len, h_q, h_kv,
                                            d_qk, d_v, dtype, flags, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return VLF_ERR_WORKSPACE;
  const cudaError_t e = vlf::prefix_forward(pp, workspace, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_attn_key_weights_workspace_size(int num_seqs, int total_kv, int max_seqlen_q,
                                           int max_seqlen_kv, int h_q, int h_kv, int d, int dtype,
                                           unsigned flags, int num_sms) {
  if (num_sms <= 0) num_sms = sm_count();
  if (max_seqlen_kv > total_kv) max_seqlen_kv = total_kv;  // (as in the call)
  return vlf::key_weights_workspace(num_seqs, total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d, dtype,
                                    flags, num_sms);
}

int vlf_attn_key_weights(const void *q, const void *k, const float *lse,
                         const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                         int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv, int h_q,
                         int h_kv, int d, int dtype, float scale, int causal, int window,
                         const float *prev, float *weights, void *workspace,
                         size_t workspace_bytes, vlf_stream_t stream, unsigned flags) {
  int st = check_common(q, k, k, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv,
                        max_seqlen_q, max_seqlen_kv, h_q, h_kv, d, d, dtype, nullptr, 0);
  if (st != VLF_OK) return st;
  if ((total_q > 0 && !lse) || (total_kv > 0 && !weights)) return VLF_ERR_INVALID;
  if (total_q >= kMostTokens || total_kv >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(lse) || !aligned16(prev) || !aligned16(weights) || !aligned16(workspace)) return VLF_ERR_ALIGN;
  if (num_seqs == 0 || max_seqlen_kv == 0) return VLF_OK;
  if (total_kv > 0 && max_seqlen_kv > total_kv) max_seqlen_kv = total_kv;  // (no sequence has more)
  vlf::KeyWeightParams kp{};
  fill_common(kp.p, q, k, nullptr, cu_seqlens_q, cu_seqlens_kv, num_seqs, total_q, total_kv, max_seqlen_q,
              max_seqlen_kv, h_q, h_kv, d, d, dtype, scale, causal, window, nullptr, 0, flags);
  kp.p.err = error_word_ptr();
  if (!kp.p.err) return VLF_ERR_LAUNCH;
  kp.lse = lse;
  kp.prev = prev;
  kp.weights = weights;
  const int sms = sm_count();
  const size_t need = vlf::key_weights_workspace(num_seqs, total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d,
                                                 dtype, flags, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return VLF_ERR_WORKSPACE;
  const cudaError_t e = vlf::key_weights(kp, workspace, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

int vlf_cache_evict(const void *k, const void *v, const float *weights,
                    const int32_t *cu_seqlens_kv, int num_seqs, int total_kv, int max_seqlen_kv,
                    int h_kv, int d_qk, int d_v, int dtype, int budget, int sink, int recent,
                    int total_out, void *k_out, void *v_out, float *weights_out,
                    int32_t *index_out, int32_t *cu_out, vlf_stream_t stream) {
  if (num_seqs < 0 || total_kv < 0 || max_seqlen_kv < 0 || h_kv < 1 || d_qk < 1 || d_v < 1 || total_out < 0)
    return VLF_ERR_INVALID;
  if (dtype != VLF_F16 && dtype != VLF_BF16 && dtype != VLF_F32) return VLF_ERR_INVALID;
  if (budget < 0 || sink < 0 || recent < 0 || (long long)sink + recent > budget) return VLF_ERR_INVALID;
  if (num_seqs == 0 && total_kv != 0) return VLF_ERR_INVALID;
  if (num_seqs > 0 && (!cu_seqlens_kv || !cu_out)) return VLF_ERR_INVALID;
  if (total_kv > 0 && (!k || !v || !weights)) return VLF_ERR_INVALID;
  if (total_out > 0 && (!k_out || !v_out || !weights_out || !index_out)) return VLF_ERR_INVALID;
  if (d_qk > 256 || d_v > 256 || num_seqs > 65535 || h_kv > 65535 || total_kv >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned16(weights) || !aligned16(cu_seqlens_kv) || !aligned16(k_out) ||
      !aligned16(v_out) || !aligned16(weights_out) || !aligned16(index_out) || !aligned16(cu_out))
    return VLF_ERR_ALIGN;
  if (num_seqs == 0) return VLF_OK;
  // kept rows are read while others are written: an output shares no byte with an input or another output
  const size_t es = dtype == VLF_F32 ? 4 : 2, in = (size_t)total_kv * h_kv, to = (size_t)total_out * h_kv;
  const size_t cu = ((size_t)num_seqs + 1) * 4;
  const Span all[9] = {
      {k_out, to * d_qk * es}, {v_out, to * d_v * es}, {weights_out, to * 4}, {index_out, to * 4}, {cu_out, cu},
      {k, in * d_qk * es}, {v, in * d_v * es}, {weights, in * 4}, {cu_seqlens_kv, cu}};
  if (overlap(all, 5, 9)) return VLF_ERR_INVALID;
  vlf::EvictParams p{};
  p.k = k; p.v = v; p.weights = weights; p.cu_kv = cu_seqlens_kv;
  p.num_seqs = num_seqs; p.total_kv = total_kv; p.h_kv = h_kv;
  p.max_kv = max_seqlen_kv < total_kv ? max_seqlen_kv : total_kv;  // (no sequence has more)
  p.d_qk = d_qk; p.d_v = d_v; p.dtype = dtype; p.budget = budget; p.sink = sink; p.recent = recent;
  p.total_out = total_out; p.k_out = k_out; p.v_out = v_out; p.weights_out = weights_out;
  p.index = index_out; p.cu_out = cu_out;
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  return vlf::cache_evict(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

namespace {
// The arguments that vlf_norm_rope and its backward share, into p (strides, weights and positions among
// them; the outputs are the caller's).  VLF_OK with total = 0 as well.
int norm_rope_args(vlf::NormRopeParams &p, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                   const void *q_weight, const void *k_weight, int weight_dtype, float eps,
                   const int32_t *positions, int n_axes, const int *sections, const float *inv_freq, int total,
                   int h_q, int h_k, int d, int rot, int dtype, int interleaved) {
  if (total < 0 || h_q < 1 || h_k < 0 || d < 1 || rot < 0 || rot > d || rot % 2) return VLF_ERR_INVALID;
  if (dtype != VLF_F16 && dtype != VLF_BF16 && dtype != VLF_F32) return VLF_ERR_INVALID;
  if ((q_weight || k_weight) && weight_dtype != dtype && weight_dtype != VLF_F32) return VLF_ERR_INVALID;
  if (!(eps >= 0.f) || isinf(eps)) return VLF_ERR_INVALID;
  if (n_axes < 1 || n_axes > 4 || (!sections && n_axes != 1)) return VLF_ERR_INVALID;
  if (!first_pairs(p.first, n_axes, sections, rot / 2)) return VLF_ERR_INVALID;
  if (d > 256 || h_q > 65535 || h_k > 65535) return VLF_ERR_UNSUPPORTED;
  if (total > 0 && (!q || (h_k > 0 && !k) || (rot > 0 && (!positions || !inv_freq)))) return VLF_ERR_INVALID;
  if (q_stride < 0 || k_stride < 0) return VLF_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(positions) ||
      !aligned16(inv_freq))
    return VLF_ERR_ALIGN;
  p.q.x = q; p.q.x_stride = q_stride; p.q.w = q_weight;
  p.k.x = k; p.k.x_stride = k_stride; p.k.w = k_weight;
  p.positions = positions; p.inv_freq = inv_freq;
  p.total = total; p.h_q = h_q; p.h_k = h_k; p.d = d; p.rot = rot; p.dtype = dtype; p.w_dtype = weight_dtype;
  p.interleaved = interleaved ? 1 : 0;
  p.eps = eps;
  return VLF_OK;
}
// Whether an output is written in place of an input with another stride.
bool other_stride(const void *in, int64_t in_stride, const void *out, int64_t out_stride, int total) {
  return in == out && total > 1 && in_stride != out_stride;
}
}  // namespace

int vlf_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                  const void *k_weight, int weight_dtype, float eps, const int32_t *positions, int n_axes,
                  const int *sections, const float *inv_freq, int total, int h_q, int h_k, int d, int rot,
                  int dtype, int interleaved, void *q_out, int64_t q_out_stride, void *k_out,
                  int64_t k_out_stride, vlf_stream_t stream) {
  vlf::NormRopeParams p{};
  const int st = norm_rope_args(p, q, q_stride, k, k_stride, q_weight, k_weight, weight_dtype, eps, positions, n_axes,
                                sections, inv_freq, total, h_q, h_k, d, rot, dtype, interleaved);
  if (st != VLF_OK) return st;
  if (total == 0) return VLF_OK;
  if (!q_out || (h_k > 0 && !k_out)) return VLF_ERR_INVALID;
  if (total > 1 && (q_out_stride < (int64_t)h_q * d || (h_k > 0 && k_out_stride < (int64_t)h_k * d))) return VLF_ERR_INVALID;
  if (!aligned16(q_out) || !aligned16(k_out)) return VLF_ERR_ALIGN;
  if (other_stride(q, q_stride, q_out, q_out_stride, total) ||
      (h_k > 0 && other_stride(k, k_stride, k_out, k_out_stride, total)))
    return VLF_ERR_INVALID;
  p.q.out = q_out; p.q.out_stride = q_out_stride;
  p.k.out = k_out; p.k.out_stride = k_out_stride;
  return vlf::norm_rope(p, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_norm_rope_bwd_workspace_size(int d) { return d < 1 || d > 256 ? 0 : vlf::norm_rope_workspace(d); }

int vlf_norm_rope_bwd(const void *dq_out, int64_t dq_out_stride, const void *dk_out, int64_t dk_out_stride,
                      const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                      const void *k_weight, int weight_dtype, float eps, const int32_t *positions, int n_axes,
                      const int *sections, const float *inv_freq, int total, int h_q, int h_k, int d, int rot,
                      int dtype, int interleaved, void *dq, int64_t dq_stride, void *dk, int64_t dk_stride,
                      void *dq_weight, void *dk_weight, void *workspace, size_t workspace_bytes,
                      vlf_stream_t stream) {
  vlf::NormRopeParams p{};
  const int st = norm_rope_args(p, q, q_stride, k, k_stride, q_weight, k_weight, weight_dtype, eps, positions, n_axes,
                                sections, inv_freq, total, h_q, h_k, d, rot, dtype, interleaved);
  if (st != VLF_OK) return st;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return VLF_ERR_INVALID;
  if (total > 0 && (!dq_out || !dq || (h_k > 0 && (!dk_out || !dk)))) return VLF_ERR_INVALID;
  if (dq_out_stride < 0 || dk_out_stride < 0 ||
      (total > 1 && (dq_stride < (int64_t)h_q * d || (h_k > 0 && dk_stride < (int64_t)h_k * d))))
    return VLF_ERR_INVALID;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) || !aligned16(dq_weight) ||
      !aligned16(dk_weight) || !aligned16(workspace))
    return VLF_ERR_ALIGN;
  if (total > 0 && (other_stride(q, q_stride, dq, dq_stride, total) || other_stride(dq_out, dq_out_stride, dq, dq_stride, total) ||
                    (h_k > 0 && (other_stride(k, k_stride, dk, dk_stride, total) ||
                                 other_stride(dk_out, dk_out_stride, dk, dk_stride, total)))))
    return VLF_ERR_INVALID;
  if (dq_weight || dk_weight) {
    if (!workspace || workspace_bytes < vlf::norm_rope_workspace(d)) return VLF_ERR_WORKSPACE;
    p.part = static_cast<float *>(workspace);
  }
  p.q.dy = dq_out; p.q.dy_stride = dq_out_stride; p.q.out = dq; p.q.out_stride = dq_stride; p.q.dw = dq_weight;
  p.k.dy = dk_out; p.k.dy_stride = dk_out_stride; p.k.out = dk; p.k.out_stride = dk_stride; p.k.dw = dk_weight;
  return vlf::norm_rope(p, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

namespace {
// log2 of a page's tokens; -1 where a page of that size is not supported.
int log2_of_page(int page) {
  for (int l = 4; l <= 8; ++l)
    if (page == 1 << l) return l;
  return -1;
}
// Sizes that every call on pages shares.
int check_pool(const void *k_pages, const void *v_pages, const void *k_scale, const void *v_scale, int num_pages,
               int page, int h_kv, int d_qk, int d_v) {
  if (num_pages < 0 || h_kv < 1 || d_qk < 1 || d_v < 1) return VLF_ERR_INVALID;
  if (num_pages > 0 && (!k_pages || !v_pages || !k_scale || !v_scale)) return VLF_ERR_INVALID;
  if (log2_of_page(page) < 0 || d_qk > 256 || d_v > 256 || h_kv > 32767) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scale) || !aligned16(v_scale)) return VLF_ERR_ALIGN;
  return VLF_OK;
}
int check_table(const int32_t *table, const int32_t *lens, int num_seqs, int max_pages, int page) {
  if (num_seqs < 0 || max_pages < 0 || page < 1) return VLF_ERR_INVALID;
  if (num_seqs > 0 && ((max_pages > 0 && !table) || !lens)) return VLF_ERR_INVALID;
  if (num_seqs > 65535 || (long long)max_pages * page >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(table) || !aligned16(lens)) return VLF_ERR_ALIGN;
  return VLF_OK;
}
}  // namespace

int vlf_pages_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *k_pages, void *v_pages,
                    float *k_scale, float *v_scale, const int32_t *page_table, const int32_t *cu_seqlens,
                    const int32_t *seqlens_kv, int num_seqs, int total, int max_pages, int num_pages, int page,
                    int h_kv, int d_qk, int d_v, int dtype, vlf_stream_t stream) {
  int st = check_pool(k_pages, v_pages, k_scale, v_scale, num_pages, page, h_kv, d_qk, d_v);
  if (st == VLF_OK) st = check_table(page_table, seqlens_kv, num_seqs, max_pages, page);
  if (st != VLF_OK) return st;
  if (total < 0 || (num_seqs == 0 && total != 0) || (num_seqs > 0 && !cu_seqlens)) return VLF_ERR_INVALID;
  if (dtype != VLF_F16 && dtype != VLF_BF16 && dtype != VLF_F32) return VLF_ERR_INVALID;
  if (total >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (total > 0 && (!k || !v)) return VLF_ERR_INVALID;
  if (total > 1 && (k_stride < 0 || v_stride < 0)) return VLF_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cu_seqlens)) return VLF_ERR_ALIGN;
  if (total == 0) return VLF_OK;
  vlf::PagesWriteParams p{};
  p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
  p.k_pages = k_pages; p.v_pages = v_pages; p.k_scale = k_scale; p.v_scale = v_scale;
  p.table = page_table; p.cu = cu_seqlens; p.kv_lens = seqlens_kv;
  p.num_seqs = num_seqs; p.total = total; p.max_pages = max_pages; p.num_pages = num_pages;
  p.page = page; p.log2_page = log2_of_page(page);
  p.h_kv = h_kv; p.d_qk = d_qk; p.d_v = d_v; p.dtype = dtype;
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  return vlf::pages_write(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_attn_varlen_fwd_pages_workspace_size(int num_seqs, int total_q, int max_seqlen_q, int h_q, int h_kv,
                                                int d_qk, int d_v, int dtype, unsigned flags, int num_sms) {
  if (num_seqs < 1 || total_q < 1 || max_seqlen_q < 1 || h_kv < 1 || h_q < h_kv || h_q % h_kv) return 0;
  if (num_sms <= 0) num_sms = sm_count();
  if (max_seqlen_q > total_q) max_seqlen_q = total_q;  // (as in the call)
  return vlf::pages_attn_workspace(num_seqs, max_seqlen_q, h_q, h_kv, d_qk, d_v, dtype, flags, num_sms);
}

int vlf_attn_varlen_fwd_pages(const void *q, const void *k_pages, const void *v_pages, const float *k_scale,
                              const float *v_scale, const int32_t *page_table, const int32_t *cu_seqlens_q,
                              const int32_t *seqlens_kv, int num_seqs, int total_q, int max_seqlen_q,
                              int max_pages, int num_pages, int page, int h_q, int h_kv, int d_qk, int d_v,
                              int dtype, float scale, int causal, int window, void *out, float *lse,
                              void *workspace, size_t workspace_bytes, vlf_stream_t stream, unsigned flags) {
  int st = check_pool(k_pages, v_pages, k_scale, v_scale, num_pages, page, h_kv, d_qk, d_v);
  if (st == VLF_OK) st = check_table(page_table, seqlens_kv, num_seqs, max_pages, page);
  if (st == VLF_OK)
    st = check_common(q, k_pages, v_pages, cu_seqlens_q, seqlens_kv, num_seqs, total_q, 0, max_seqlen_q, 0, h_q, h_kv,
                      d_qk, d_v, dtype, nullptr, 0);
  if (st != VLF_OK) return st;
  if (total_q > 0 && !out) return VLF_ERR_INVALID;
  if (total_q >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  if (!aligned16(out) || !aligned16(lse) || !aligned16(workspace)) return VLF_ERR_ALIGN;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return VLF_OK;
  if (max_seqlen_q > total_q) max_seqlen_q = total_q;  // (no sequence has more)
  vlf::PagesAttnParams a{};
  fill_common(a.p, q, k_pages, v_pages, cu_seqlens_q, nullptr, num_seqs, total_q, 0, max_seqlen_q, max_pages * page, h_q,
              h_kv, d_qk, d_v, dtype, scale, causal, window, nullptr, 0, flags);
  a.p.out = out;
  a.p.lse = lse;
  a.p.err = error_word_ptr();
  if (!a.p.err) return VLF_ERR_LAUNCH;
  a.k_pages = static_cast<const uint8_t *>(k_pages);
  a.v_pages = static_cast<const uint8_t *>(v_pages);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.table = page_table; a.kv_lens = seqlens_kv;
  a.max_pages = max_pages; a.num_pages = num_pages; a.page = page; a.log2_page = log2_of_page(page);
  const int sms = sm_count();
  const size_t need = vlf::pages_attn_workspace(num_seqs, max_seqlen_q, h_q, h_kv, d_qk, d_v, dtype, flags, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return VLF_ERR_WORKSPACE;
  const cudaError_t e = vlf::pages_forward(a, workspace, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

int vlf_pages_copy(void *k_pages, void *v_pages, float *k_scale, float *v_scale, const int32_t *src,
                   const int32_t *dst, int n, int num_pages, int page, int h_kv, int d_qk, int d_v,
                   vlf_stream_t stream) {
  const int st = check_pool(k_pages, v_pages, k_scale, v_scale, num_pages, page, h_kv, d_qk, d_v);
  if (st != VLF_OK) return st;
  if (n < 0 || (n > 0 && (!src || !dst))) return VLF_ERR_INVALID;
  if (!aligned16(src) || !aligned16(dst)) return VLF_ERR_ALIGN;
  if (n == 0) return VLF_OK;
  vlf::PagesCopyParams p{};
  p.k_pages = k_pages; p.v_pages = v_pages; p.k_scale = k_scale; p.v_scale = v_scale;
  p.src = src; p.dst = dst; p.n = n; p.num_pages = num_pages; p.page = page;
  p.h_kv = h_kv; p.d_qk = d_qk; p.d_v = d_v;
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  return vlf::pages_copy(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_pages_fork_workspace_size(int num_pages, int num_out) {
  return num_pages < 0 || num_out < 0 ? 0 : vlf::pages_fork_workspace(num_pages, num_out);
}

int vlf_pages_fork(const int32_t *page_table, const int32_t *seqlens, const int32_t *refs, const int32_t *parents,
                   const int32_t *grow, int num_in, int num_out, int max_pages, int num_pages, int page,
                   int32_t *table_out, int32_t *seqlens_out, int32_t *refs_out, int32_t *src, int32_t *dst,
                   int32_t *left, void *workspace, size_t workspace_bytes, vlf_stream_t stream) {
  if (num_pages < 0 || num_out < 0 || !left || (num_pages > 0 && (!refs || !refs_out))) return VLF_ERR_INVALID;
  if (log2_of_page(page) < 0) return VLF_ERR_UNSUPPORTED;
  const int st = check_table(page_table, seqlens, num_in, max_pages, page);
  if (st != VLF_OK) return st;
  if (num_out > 0 && (!parents || !grow || (max_pages > 0 && !table_out) || !seqlens_out || !src || !dst)) return VLF_ERR_INVALID;
  if (num_out > 65535 || num_pages >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  const void *all16[] = {refs, parents, grow, table_out, seqlens_out, refs_out, src, dst, left, workspace};
  for (const void *x : all16)
    if (!aligned16(x)) return VLF_ERR_ALIGN;
  if (!workspace || workspace_bytes < vlf::pages_fork_workspace(num_pages, num_out)) return VLF_ERR_WORKSPACE;
  const size_t row = (size_t)max_pages * 4, in = num_in, out = num_out, pool = (size_t)num_pages * 4;
  const Span all[12] = {{table_out, out * row}, {seqlens_out, out * 4}, {refs_out, pool}, {src, out * 4}, {dst, out * 4},
                        {left, 4}, {workspace, workspace_bytes}, {page_table, in * row}, {seqlens, in * 4}, {refs, pool},
                        {parents, out * 4}, {grow, out * 4}};
  if (overlap(all, 7, 12)) return VLF_ERR_INVALID;
  vlf::PagesForkParams p{};
  p.table = page_table; p.lens = seqlens; p.refs = refs; p.parents = parents; p.grow = grow;
  p.num_in = num_in; p.num_out = num_out; p.max_pages = max_pages; p.num_pages = num_pages;
  p.log2_page = log2_of_page(page);
  p.table_out = table_out; p.lens_out = seqlens_out; p.refs_out = refs_out; p.src = src; p.dst = dst; p.left = left;
  p.err = error_word_ptr();
  if (!p.err) return VLF_ERR_LAUNCH;
  return vlf::pages_fork(p, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

size_t vlf_pages_compact_workspace_size(int num_pages) {
  return num_pages < 0 ? 0 : vlf::pages_compact_workspace(num_pages);
}

int vlf_pages_compact(const int32_t *page_table, const int32_t *refs, int num_seqs, int max_pages, int num_pages,
                      int32_t *table_out, int32_t *refs_out, int32_t *to, int32_t *src, int32_t *dst, int32_t *used,
                      void *workspace, size_t workspace_bytes, vlf_stream_t stream) {
  if (num_seqs < 0 || max_pages < 0 || num_pages < 1 || !used || !refs || !refs_out || !to) return VLF_ERR_INVALID;
  const long long entries = (long long)num_seqs * max_pages;
  if ((entries > 0 && (!page_table || !table_out)) || (num_pages > 1 && (!src || !dst))) return VLF_ERR_INVALID;
  if (num_seqs > 65535 || num_pages >= kMostTokens) return VLF_ERR_UNSUPPORTED;
  const void *all16[] = {page_table, refs, table_out, refs_out, to, src, dst, used, workspace};
  for (const void *x : all16)
    if (!aligned16(x)) return VLF_ERR_ALIGN;
  if (!workspace || workspace_bytes < vlf::pages_compact_workspace(num_pages)) return VLF_ERR_WORKSPACE;
  const size_t table = (size_t)entries * 4, pool = (size_t)num_pages * 4, half = (size_t)(num_pages / 2) * 4;
  const Span all[9] = {{table_out, table}, {refs_out, pool}, {to, pool}, {src, half}, {dst, half}, {used, 4},
                       {workspace, workspace_bytes}, {page_table, table}, {refs, pool}};
  if (overlap(all, 7, 9)) return VLF_ERR_INVALID;
  vlf::PagesCompactParams p{};
  p.table = page_table; p.refs = refs; p.entries = entries; p.num_pages = num_pages;
  p.table_out = table_out; p.refs_out = refs_out; p.to = to; p.src = src; p.dst = dst; p.used = used;
  return vlf::pages_compact(p, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? VLF_OK : VLF_ERR_LAUNCH;
}

}  // extern "C"
