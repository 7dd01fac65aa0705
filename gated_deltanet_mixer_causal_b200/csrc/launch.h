// launch.h -- internal launchers behind the C ABI (gdn_api.cu). Each enqueues its kernels
// on `stream` and returns cudaGetLastError(); arguments are validated by the caller.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// A failed launch's error, not left behind for the next call that asks for the last one.
inline cudaError_t launch_result(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Raises a kernel's limit of dynamic shared memory on the current device, once for each device
// (numbers below 64; others every time). `prepared` is the kernel's own.
template <typename K>
inline cudaError_t raise_smem_limit(K kernel, int bytes, std::atomic<uint64_t>& prepared) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (prepared.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) prepared.fetch_or(bit, std::memory_order_relaxed);
  return launch_result(e);
}

// Launches a kernel that begins with wait_for_previous_grid (common.cuh), so that its launch
// overlaps the end of the kernel before it.
template <typename... P, typename... A>
inline cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                     A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid; cfg.blockDim = block; cfg.dynamicSmemBytes = smem; cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr; cfg.numAttrs = 1;
  return launch_result(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

constexpr int kF32 = 0;   // GDN_F32
constexpr int kBF16 = 1;  // GDN_BF16

cudaError_t launch_conv1d_silu(int dtype, const void* x, void* y, const void* w,
                               const int32_t* cu, int32_t n_seq, int64_t T, int32_t Cc,
                               const void* conv_state_in, void* conv_state_out,
                               cudaStream_t stream);

// state_dtype: kF32, or kBF16 for bf16 state storage (fp32 arithmetic)
cudaError_t launch_decode_step(int dtype, const void* x, const void* conv_w, void* conv_state,
                               const float* g, const float* beta, void* state, int state_dtype,
                               void* o, int32_t B, int32_t Hk, int32_t Hv, int32_t d, float scale,
                               cudaStream_t stream);
// n_tok (1..8) tokens per sequence; x [B, n_tok, Cc], g/beta [B, n_tok, Hv], o [B, n_tok, Hv, d]
cudaError_t launch_decode_tokens(int dtype, const void* x, const void* conv_w, void* conv_state,
                                 const float* g, const float* beta, void* state, int state_dtype,
                                 void* o, int32_t B, int32_t n_tok, int32_t Hk, int32_t Hv, int32_t d,
                                 float scale, cudaStream_t stream);

// States at block boundaries (prefix caching): after every block_tokens tokens of a sequence
// (block_tokens a positive multiple of 64; 0 = none), its state goes to row
// block_rows[n] + m - 1 of block_states [n_block_rows, Hv, dv, dk] (the state dtype of the
// call) for the m-th boundary; rows outside [0, n_block_rows) are skipped.
struct BlockStates {
  int32_t block_tokens = 0;
  void* states = nullptr;
  const int32_t* rows = nullptr;
  int64_t n_rows = 0;
};

// Token-by-token fp32 recurrence (SIMT): the fp32-activation prefill path. States (initial,
// final, block) are stored as state_dtype (kF32, or kBF16 storage with fp32 math).
cudaError_t launch_prefill_recurrent(int dtype, const void* q, const void* k, const void* v,
                                     const float* g, const float* beta, void* o, int64_t T,
                                     int32_t Hk, int32_t Hv, int32_t d, int64_t qk_stride,
                                     int64_t v_stride, const int32_t* cu, int32_t n_seq,
                                     const void* init, void* final_state, int state_dtype,
                                     float scale, int32_t l2norm, BlockStates blocks,
                                     cudaStream_t stream);

// Chunked WY/UT prefill on tcgen05 (bf16 activations, dk = dv = 128, at most
// kPrefillTcMaxG value heads per key head). Needs
// prefill_chunk_tc_workspace(...) bytes of workspace.
constexpr int kPrefillTcMaxG = 8;
size_t prefill_chunk_tc_workspace(int64_t T, int32_t n_seq, int32_t Hv);
// The workspace's first int: 0, or the code of a bounded wait that gave up in the last call.
const char* prefill_chunk_tc_error_string(int code);
int prefill_chunk_tc_launches(int64_t T, int32_t n_seq, int32_t Hv, int num_sms);
cudaError_t launch_prefill_chunk_tc(const void* q, const void* k, const void* v, const float* g,
                                    const float* beta, void* o, int64_t T, int32_t Hk, int32_t Hv,
                                    int64_t qk_stride, int64_t v_stride, const int32_t* cu,
                                    int32_t n_seq, const void* init, void* fin, int state_dtype,
                                    float scale, BlockStates blocks, void* workspace,
                                    cudaStream_t stream);

// The paged decode's arguments (validated): pools with page strides in elements.
struct PagedDecode {
  const void* x; int64_t x_stride;          // [B, n_tok, Cc], a token every x_stride elements
  const void* conv_w;
  void* conv_pool; int64_t conv_stride;
  void* state_pool; int64_t state_stride;
  int32_t n_pages;
  const int32_t* read_pages;                // [B]
  const int32_t* write_pages;               // [B, n_tok] or null: the last state to the page read
  const int32_t* n_valid;                   // [B] or null: n_tok
  const float* g; const float* beta;        // [B, n_tok, Hv]
  const void* z; int64_t z_stride;          // output gate [B, n_tok, Hv, dv] or null
  const void* norm_w; float eps;
  void* o;                                  // [B, n_tok, Hv, dv]
  int32_t B, n_tok, Hk, Hv;
  float scale;
};
size_t decode_paged_smem(int n_tok, int64_t G, int d);
cudaError_t launch_decode_paged(int dtype, int state_dtype, int d, const PagedDecode& a, cudaStream_t stream);

// Page copies: strides in bytes; every page a multiple of 16 bytes.
constexpr int kPagesMaxList = 2048;
constexpr int kPagesMaxPools = 4;
struct PagePool {
  const char* src; char* dst;
  int64_t page_bytes, src_page, src_layer, dst_page, dst_layer;
  int32_t layers;
  bool same;                                // src and dst are one pool
};
struct PagesCopy {
  PagePool pool[kPagesMaxPools]; int32_t n_pools;
  int32_t src_pages, dst_pages;
  const int32_t* src; const int32_t* dst; int32_t n;
};
// plain: no destination is named twice and none is another entry's source
bool pages_copy_fits(const PagesCopy& a, bool plain);      // one launch can number its tiles
cudaError_t launch_pages_copy(const PagesCopy& a, bool plain, cudaStream_t stream);
cudaError_t launch_pages_take(int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n, int32_t* out,
                              cudaStream_t stream);
cudaError_t launch_pages_ref(int32_t* refs, int32_t n_pages, const int32_t* pages, int32_t n, int32_t delta,
                             cudaStream_t stream);
cudaError_t launch_pages_plan(int32_t* refs, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* src,
                              int32_t* dst, int32_t* map, int32_t* n_live, cudaStream_t stream);

// Norms. Weight gradients go through at most kNormParts rows of fp32 parts in `part`.
constexpr int kNormParts = 592;
struct GatedNorm {
  const void *o, *z; int64_t z_stride; const void* w; float eps;
  void* y;                                  // forward
  const void* dy; void *dout, *dz; int64_t dz_stride; float *dw, *part;   // backward
  int64_t rows; int32_t H; bool back;
};
struct AddNorm {
  const void *x, *w; float scale, w_add, eps;
  const void* res;                          // forward: the residual; backward: dh or null
  void* h;                                  // forward: written; backward: read
  void* n;                                  // forward: written; backward: dn, read
  void *dres, *dx; float *dw, *part;        // backward
  int64_t rows; int32_t D; bool back;
};
cudaError_t launch_gated_norm(int dtype, int d, const GatedNorm& a, cudaStream_t stream);
cudaError_t launch_add_norm(int dtype, int res_dtype, const AddNorm& a, cudaStream_t stream);

// Workspace bytes the prefill path chosen for these arguments needs (0 for the
// token-recurrent path, which takes no workspace); SIZE_MAX for unsupported shapes.
size_t prefill_workspace_need(gdn_dtype_t dt, int64_t T, int32_t n_seq, int32_t Hk, int32_t Hv,
                              int32_t dk, int32_t dv, int32_t qk_l2norm);

// Records the calling thread's gdn_last_error() text and returns s.
gdn_status_t set_error(gdn_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

}  // namespace gdn
