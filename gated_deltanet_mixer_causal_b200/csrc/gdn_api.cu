// gdn_api.cu -- the extern "C" boundary of libgdn.so (declared in include/gdn.h).
//
// Every entry point validates its arguments on the host before launching anything,
// returns a status code, never prints and never throws. Work is enqueued on the caller's
// stream; the library allocates no device memory.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "gdn.h"
#include "launch.h"

namespace {

thread_local char g_last_error[256] = "";

gdn_status_t fail(gdn_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status_t fail(gdn_status_t s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

gdn_status_t ok() {
  g_last_error[0] = '\0';
  return GDN_OK;
}

gdn_status_t cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Pages of `bytes` at l * layer + p * page keep apart: either a layer's pages lie behind one
// another and the layers behind those, or the other way round.
bool pages_apart(int32_t pages, int64_t page, int32_t layers, int64_t layer, int64_t bytes) {
  if (page % 16 || layer % 16 || page < 0 || layer < 0) return false;
  if (pages > 1 && page < bytes) return false;
  if (layers <= 1 || pages < 1) return true;
  if (layer < bytes) return false;
  return layer >= (pages - 1) * page + bytes || page >= (layers - 1) * layer + bytes || pages == 1;
}

int64_t greatest_common(int64_t a, int64_t b) {
  while (b != 0) { const int64_t r = a % b; a = b; b = r; }
  return a;
}

// [a, a + na) and [b, b + nb) share a byte (null or empty ranges never overlap).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

// The pages of a pool in one layout: `bytes` at `at` + l * layer + p * page.
struct Pages {
  const void* at;
  int64_t bytes, page, layer;
  int32_t pages, layers;
  size_t extent() const {
    return pages > 0 && layers > 0 ? (size_t)((layers - 1) * layer + (pages - 1) * page + bytes) : 0;
  }
};

// No page of one shares a byte with a page of the other: their extents lie apart, or both repeat at
// a common step in which their parts do. The parts are single pages, or all the layers of a page
// (records of a page), or all the pages of a layer.
bool pools_apart(const Pages& a, const Pages& b) {
  if (!overlap(a.at, a.extent(), b.at, b.extent())) return true;
  const int64_t delta = (int64_t)((intptr_t)b.at - (intptr_t)a.at);
  for (int part = 0; part < 3; ++part) {
    int64_t step = 0, size[2];
    const Pages* both[2] = {&a, &b};
    for (int i = 0; i < 2; ++i) {
      const Pages& p = *both[i];
      size[i] = p.bytes;
      if (part == 1) size[i] += (p.layers - 1) * p.layer;
      else if (p.layers > 1) step = greatest_common(step, p.layer);
      if (part == 2) size[i] += (p.pages - 1) * p.page;
      else if (p.pages > 1) step = greatest_common(step, p.page);
    }
    if (step == 0) continue;
    const int64_t from = (delta % step + step) % step;      // of b's part in the step that begins with a's
    if (from >= size[0] && from + size[1] <= step) return true;
  }
  return false;
}

size_t elt_size(gdn_dtype_t dt) { return dt == GDN_F32 ? 4 : 2; }

bool valid_dtype(gdn_dtype_t dt) { return dt == GDN_F32 || dt == GDN_BF16; }

bool supported_head_dim(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// bf16 activations with 128-wide heads (and at most 8 value heads per key head) run the
// chunked tensor-core prefill; everything else runs the token-by-token fp32 kernel.
// TMA coordinates are 32-bit: the tensor-core prefill addresses tokens and workspace rows
// (chunk slot x value head x 128) with int32, which bounds the tokens of one call.
bool tc_rows_fit(int64_t T, int32_t n_seq, int32_t Hv) {
  const int64_t slots = (T + 63) / 64 + (n_seq < 1 ? 1 : n_seq);
  return T <= 0x7fffffffLL && slots * Hv * 128 <= 0x7fffffffLL;
}

// The tensor-core prefill folds the q/k L2 norm into its factors; inputs used as given
// (qk_l2norm = 0) take the token-recurrent path.
bool use_tensor_core_prefill(gdn_dtype_t dt, int32_t d, int32_t Hk, int32_t Hv, int32_t qk_l2norm = 1) {
  return dt == GDN_BF16 && d == 128 && Hv / Hk <= gdn::kPrefillTcMaxG && qk_l2norm != 0;
}

}  // namespace

namespace gdn {

size_t prefill_workspace_need(gdn_dtype_t dt, int64_t T, int32_t n_seq, int32_t Hk, int32_t Hv,
                              int32_t dk, int32_t dv, int32_t qk_l2norm) {
  if (!valid_dtype(dt) || T < 0 || Hk <= 0 || Hv <= 0 || Hv % Hk != 0 || dk != dv ||
      !supported_head_dim(dk))
    return SIZE_MAX;
  if (n_seq < 1) n_seq = 1;
  if (!use_tensor_core_prefill(dt, dk, Hk, Hv, qk_l2norm)) return 0;
  return tc_rows_fit(T, n_seq, Hv) ? prefill_chunk_tc_workspace(T, n_seq, Hv) : SIZE_MAX;
}

gdn_status_t set_error(gdn_status_t s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

}  // namespace gdn

extern "C" {

const char* gdn_status_string(gdn_status_t s) {
  switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
    case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT";
  }
  return "GDN_ERR_UNKNOWN";
}

const char* gdn_last_error(void) { return g_last_error; }

const char* gdn_version(void) { return "0.1.0"; }

gdn_status_t gdn_conv1d_silu(const void* x, void* y, gdn_dtype_t dt, const void* w,
                             const int32_t* cu_seqlens, int32_t n_seq, int64_t T, int32_t Cc,
                             const void* conv_state_in, void* conv_state_out,
                             gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "conv1d_silu: unknown dtype %d", (int)dt);
  if (T < 0) return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: T = %lld < 0", (long long)T);
  if (Cc <= 0 || Cc % 8 != 0)
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: Cc = %d must be a positive multiple of 8", Cc);
  if (cu_seqlens == nullptr) n_seq = 1;
  if (n_seq < 1 || n_seq > 65535)
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: n_seq = %d outside [1, 65535]", n_seq);
  if (T > 0 && (x == nullptr || y == nullptr || w == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: x, y and w must be non-null");
  if (!aligned16(x) || !aligned16(y) || !aligned16(w) || !aligned16(conv_state_in) ||
      !aligned16(conv_state_out))
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: pointers must be 16-byte aligned");
  const size_t es = elt_size(dt);
  const size_t xb = (size_t)T * Cc * es, sb = (size_t)n_seq * 3 * Cc * es;
  if (overlap(x, xb, y, xb)) return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: y overlaps x");
  if (overlap(conv_state_in, sb, conv_state_out, sb))
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: conv_state_out overlaps conv_state_in");
  if (overlap(y, xb, conv_state_out, sb) || overlap(y, xb, conv_state_in, sb) ||
      overlap(x, xb, conv_state_out, sb))
    return fail(GDN_ERR_INVALID_ARG, "conv1d_silu: conv states overlap x or y");
  return cuda_status(gdn::launch_conv1d_silu((int)dt, x, y, w, cu_seqlens, n_seq, T, Cc,
                                             conv_state_in, conv_state_out, (cudaStream_t)stream),
                     "conv1d_silu launch");
}

size_t gdn_chunk_prefill_workspace_size(int64_t T, int32_t n_seq, int32_t Hk, int32_t Hv,
                                        int32_t dk, int32_t dv, gdn_dtype_t dt) {
  return gdn::prefill_workspace_need(dt, T, n_seq, Hk, Hv, dk, dv, 1);
}

int32_t gdn_chunk_prefill_path(gdn_dtype_t dt, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                               int32_t qk_l2norm) {
  if (!valid_dtype(dt) || Hk <= 0 || Hv <= 0 || Hv % Hk != 0 || dk != dv || !supported_head_dim(dk))
    return -1;
  return use_tensor_core_prefill(dt, dk, Hk, Hv, qk_l2norm) ? GDN_PATH_CHUNKED_TC : GDN_PATH_RECURRENT;
}

int32_t gdn_chunk_prefill_launches(int64_t T, int32_t n_seq, int32_t Hk, int32_t Hv, int32_t dk,
                                   int32_t dv, gdn_dtype_t dt, int32_t qk_l2norm, int32_t num_sms) {
  if (gdn_chunk_prefill_path(dt, Hk, Hv, dk, dv, qk_l2norm) < 0 || T < 0 || n_seq < 1 || num_sms < 1) return -1;
  if (!use_tensor_core_prefill(dt, dk, Hk, Hv, qk_l2norm)) return 1;
  if (!tc_rows_fit(T, n_seq, Hv)) return -1;
  return gdn::prefill_chunk_tc_launches(T, n_seq, Hv, num_sms);
}

gdn_status_t gdn_chunk_prefill_ex(const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, void* o, gdn_dtype_t dt, int64_t T,
                                  int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, int64_t qk_stride,
                                  int64_t v_stride, const int32_t* cu_seqlens, int32_t n_seq,
                                  const void* initial_state, void* final_state,
                                  gdn_dtype_t state_dt, float scale, int32_t qk_l2norm,
                                  int32_t block_tokens, void* block_states,
                                  const int32_t* block_rows, int64_t n_block_rows, void* workspace,
                                  size_t workspace_bytes, gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "chunk_prefill: unknown dtype %d", (int)dt);
  if (!valid_dtype(state_dt))
    return fail(GDN_ERR_UNSUPPORTED, "chunk_prefill: unknown state dtype %d", (int)state_dt);
  if (T < 0) return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: T = %lld < 0", (long long)T);
  if (Hk <= 0 || Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: Hk, Hv must be > 0");
  if (Hv % Hk != 0) return fail(GDN_ERR_UNSUPPORTED, "chunk_prefill: Hv %% Hk != 0 (%d, %d)", Hv, Hk);
  if (dk != dv || !supported_head_dim(dk))
    return fail(GDN_ERR_UNSUPPORTED, "chunk_prefill: head dims dk=%d dv=%d (need dk = dv in {16,32,64,128})", dk, dv);
  if (cu_seqlens == nullptr) n_seq = 1;
  if (n_seq < 1) return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: n_seq = %d < 1", n_seq);
  if (qk_stride == 0) qk_stride = (int64_t)Hk * dk;
  if (v_stride == 0) v_stride = (int64_t)Hv * dv;
  if (qk_stride < (int64_t)Hk * dk || v_stride < (int64_t)Hv * dv || qk_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: strides (%lld, %lld) must cover a token row and be multiples of 8",
                (long long)qk_stride, (long long)v_stride);
  if (T > 0 && (!q || !k || !v || !g || !beta || !o))
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: q, k, v, g, beta, o must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
      !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state))
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: pointers must be 16-byte aligned");
  const size_t es = elt_size(dt);
  const size_t ob = (size_t)T * Hv * dv * es;
  const size_t qkb = T > 0 ? ((size_t)(T - 1) * qk_stride + (size_t)Hk * dk) * es : 0;
  const size_t vb = T > 0 ? ((size_t)(T - 1) * v_stride + (size_t)Hv * dv) * es : 0;
  const size_t sts = elt_size(state_dt);
  const size_t gb = (size_t)T * Hv * 4, stb = (size_t)n_seq * Hv * dv * dk * sts;
  if (overlap(o, ob, q, qkb) || overlap(o, ob, k, qkb) || overlap(o, ob, v, vb) ||
      overlap(o, ob, g, gb) || overlap(o, ob, beta, gb) || overlap(o, ob, initial_state, stb) ||
      overlap(o, ob, final_state, stb))
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: o overlaps an input or a state");
  if (final_state != initial_state && overlap(initial_state, stb, final_state, stb))
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: final_state partially overlaps initial_state");
  gdn::BlockStates blocks;
  if (block_tokens < 0 || block_tokens % 64 != 0)
    return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: block_tokens = %d must be 0 or a positive multiple of 64",
                block_tokens);
  if (block_tokens > 0) {
    if (!block_states || !block_rows || n_block_rows < 1)
      return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: block states need block_states, block_rows and n_block_rows >= 1");
    if (!aligned16(block_states))
      return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: block_states must be 16-byte aligned");
    const size_t bsb = (size_t)n_block_rows * Hv * dv * dk * sts;
    if (overlap(block_states, bsb, q, qkb) || overlap(block_states, bsb, k, qkb) ||
        overlap(block_states, bsb, v, vb) || overlap(block_states, bsb, g, gb) ||
        overlap(block_states, bsb, beta, gb) || overlap(block_states, bsb, o, ob) ||
        overlap(block_states, bsb, initial_state, stb) || overlap(block_states, bsb, final_state, stb) ||
        overlap(block_states, bsb, block_rows, (size_t)n_seq * 4))
      return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: block_states overlaps another buffer");
    blocks.block_tokens = block_tokens;
    blocks.states = block_states;
    blocks.rows = block_rows;
    blocks.n_rows = n_block_rows;
  }
  const bool tensor_core = use_tensor_core_prefill(dt, dk, Hk, Hv, qk_l2norm);
  if (tensor_core && !tc_rows_fit(T, n_seq, Hv))
    return fail(GDN_ERR_UNSUPPORTED, "chunk_prefill: %lld tokens of %d value heads exceed the 32-bit "
                "TMA coordinates of one call; split the batch", (long long)T, Hv);
  const size_t need = tensor_core ? gdn::prefill_chunk_tc_workspace(T, n_seq, Hv) : 0;
  if (workspace_bytes < need || (need > 0 && workspace == nullptr))
    return fail(GDN_ERR_WORKSPACE, "chunk_prefill: workspace %zu bytes < %zu needed", workspace_bytes, need);
  if (T == 0 && final_state == nullptr) return ok();
  if (tensor_core) {
    if (!aligned16(workspace) || ((uintptr_t)workspace & 255u) != 0)
      return fail(GDN_ERR_INVALID_ARG, "chunk_prefill: workspace must be 256-byte aligned");
    return cuda_status(gdn::launch_prefill_chunk_tc(q, k, v, g, beta, o, T, Hk, Hv, qk_stride, v_stride,
                                                    cu_seqlens, n_seq, initial_state, final_state,
                                                    (int)state_dt, scale, blocks, workspace,
                                                    (cudaStream_t)stream),
                       "chunk_prefill (tensor-core) launch");
  }
  if (workspace != nullptr && workspace_bytes >= sizeof(int)) {   // no wait can fail here
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_status(e, "chunk_prefill: clearing the status word");
  }
  return cuda_status(gdn::launch_prefill_recurrent((int)dt, q, k, v, g, beta, o, T, Hk, Hv, dk,
                                                   qk_stride, v_stride, cu_seqlens, n_seq,
                                                   initial_state, final_state, (int)state_dt, scale,
                                                   qk_l2norm, blocks, (cudaStream_t)stream),
                     "chunk_prefill launch");
}

gdn_status_t gdn_prefill_status(const void* workspace, gdn_stream_t stream) {
  if (workspace == nullptr) return fail(GDN_ERR_INVALID_ARG, "prefill_status: workspace is NULL");
  int word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, workspace, sizeof(int), cudaMemcpyDeviceToHost,
                                  (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e, "prefill_status");
  if (word == 0) return ok();
  return fail(GDN_ERR_TIMEOUT, "prefill_status: a bounded device-side wait gave up (%s, code %d); "
              "the outputs of that call are invalid", gdn::prefill_chunk_tc_error_string(word), word);
}

gdn_status_t gdn_chunk_prefill(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, void* o, gdn_dtype_t dt, int64_t T,
                               int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, int64_t qk_stride,
                               int64_t v_stride, const int32_t* cu_seqlens, int32_t n_seq,
                               const float* initial_state, float* final_state, float scale,
                               int32_t qk_l2norm, void* workspace, size_t workspace_bytes,
                               gdn_stream_t stream) {
  return gdn_chunk_prefill_ex(q, k, v, g, beta, o, dt, T, Hk, Hv, dk, dv, qk_stride, v_stride,
                              cu_seqlens, n_seq, initial_state, final_state, GDN_F32, scale,
                              qk_l2norm, 0, nullptr, nullptr, 0, workspace, workspace_bytes, stream);
}

gdn_status_t gdn_decode_step_ex(const void* x, const void* conv_w, void* conv_state, const float* g,
                                const float* beta, void* state, gdn_dtype_t state_dt, void* o,
                                gdn_dtype_t dt, int32_t B, int32_t Hk, int32_t Hv, int32_t dk,
                                int32_t dv, float scale, gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_step: unknown dtype %d", (int)dt);
  if (!valid_dtype(state_dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_step: unknown state dtype %d", (int)state_dt);
  if (B < 0) return fail(GDN_ERR_INVALID_ARG, "decode_step: B = %d < 0", B);
  if (Hk <= 0 || Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "decode_step: Hk, Hv must be > 0");
  if (Hv % Hk != 0) return fail(GDN_ERR_UNSUPPORTED, "decode_step: Hv %% Hk != 0 (%d, %d)", Hv, Hk);
  if (dk != dv || !supported_head_dim(dk))
    return fail(GDN_ERR_UNSUPPORTED, "decode_step: head dims dk=%d dv=%d (need dk = dv in {16,32,64,128})", dk, dv);
  if ((int64_t)B * Hk > 0x7fffffffLL) return fail(GDN_ERR_INVALID_ARG, "decode_step: B * Hk too large");
  if (B == 0) return ok();
  if (!x || !conv_w || !conv_state || !g || !beta || !state || !o)
    return fail(GDN_ERR_INVALID_ARG, "decode_step: all pointers must be non-null");
  if (!aligned16(x) || !aligned16(conv_w) || !aligned16(conv_state) || !aligned16(g) ||
      !aligned16(beta) || !aligned16(state) || !aligned16(o))
    return fail(GDN_ERR_INVALID_ARG, "decode_step: pointers must be 16-byte aligned");
  const size_t es = elt_size(dt);
  const int64_t Cc = 2LL * Hk * dk + (int64_t)Hv * dv;
  const size_t xb = (size_t)B * Cc * es, csb = (size_t)B * 3 * Cc * es;
  const size_t stb = (size_t)B * Hv * dv * dk * elt_size(state_dt), ob = (size_t)B * Hv * dv * es;
  const size_t gb = (size_t)B * Hv * 4, wb = (size_t)Cc * 4 * es;
  const void* ro[4] = {x, conv_w, g, beta};
  const size_t rob[4] = {xb, wb, gb, gb};
  for (int i = 0; i < 4; ++i)
    if (overlap(ro[i], rob[i], conv_state, csb) || overlap(ro[i], rob[i], state, stb) ||
        overlap(ro[i], rob[i], o, ob))
      return fail(GDN_ERR_INVALID_ARG, "decode_step: an output overlaps an input");
  if (overlap(conv_state, csb, state, stb) || overlap(conv_state, csb, o, ob) ||
      overlap(state, stb, o, ob))
    return fail(GDN_ERR_INVALID_ARG, "decode_step: conv_state, state and o must not overlap");
  return cuda_status(gdn::launch_decode_step((int)dt, x, conv_w, conv_state, g, beta, state,
                                             (int)state_dt, o, B, Hk, Hv, dk, scale,
                                             (cudaStream_t)stream),
                     "decode_step launch");
}

gdn_status_t gdn_decode_step(const void* x, const void* conv_w, void* conv_state, const float* g,
                             const float* beta, float* state, void* o, gdn_dtype_t dt, int32_t B,
                             int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, float scale,
                             gdn_stream_t stream) {
  return gdn_decode_step_ex(x, conv_w, conv_state, g, beta, state, GDN_F32, o, dt, B, Hk, Hv, dk,
                            dv, scale, stream);
}

gdn_status_t gdn_decode_tokens_ex(const void* x, const void* conv_w, void* conv_state, const float* g,
                                  const float* beta, void* state, gdn_dtype_t state_dt, void* o,
                                  gdn_dtype_t dt, int32_t B, int32_t n_tok, int32_t Hk, int32_t Hv,
                                  int32_t dk, int32_t dv, float scale, gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_tokens: unknown dtype %d", (int)dt);
  if (!valid_dtype(state_dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_tokens: unknown state dtype %d", (int)state_dt);
  if (B < 0) return fail(GDN_ERR_INVALID_ARG, "decode_tokens: B = %d < 0", B);
  if (n_tok < 1 || n_tok > 8) return fail(GDN_ERR_INVALID_ARG, "decode_tokens: n_tok = %d outside [1, 8]", n_tok);
  if (Hk <= 0 || Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "decode_tokens: Hk, Hv must be > 0");
  if (Hv % Hk != 0) return fail(GDN_ERR_UNSUPPORTED, "decode_tokens: Hv %% Hk != 0 (%d, %d)", Hv, Hk);
  if (dk != dv || !supported_head_dim(dk))
    return fail(GDN_ERR_UNSUPPORTED, "decode_tokens: head dims dk=%d dv=%d (need dk = dv in {16,32,64,128})", dk, dv);
  const int64_t G = Hv / Hk;
  if ((int64_t)n_tok * ((2 + G) * dk + G * dk + 1) * 4 > 227 * 1024)
    return fail(GDN_ERR_UNSUPPORTED, "decode_tokens: %d tokens of %lld value heads per key head exceed shared memory",
                n_tok, (long long)G);
  if ((int64_t)B * Hk > 0x7fffffffLL) return fail(GDN_ERR_INVALID_ARG, "decode_tokens: B * Hk too large");
  if (B == 0) return ok();
  if (!x || !conv_w || !conv_state || !g || !beta || !state || !o)
    return fail(GDN_ERR_INVALID_ARG, "decode_tokens: all pointers must be non-null");
  if (!aligned16(x) || !aligned16(conv_w) || !aligned16(conv_state) || !aligned16(g) ||
      !aligned16(beta) || !aligned16(state) || !aligned16(o))
    return fail(GDN_ERR_INVALID_ARG, "decode_tokens: pointers must be 16-byte aligned");
  const size_t es = elt_size(dt);
  const int64_t Cc = 2LL * Hk * dk + (int64_t)Hv * dv;
  const size_t xb = (size_t)B * n_tok * Cc * es, csb = (size_t)B * 3 * Cc * es;
  const size_t stb = (size_t)B * Hv * dv * dk * elt_size(state_dt), ob = (size_t)B * n_tok * Hv * dv * es;
  const size_t gb = (size_t)B * n_tok * Hv * 4, wb = (size_t)Cc * 4 * es;
  const void* ro[4] = {x, conv_w, g, beta};
  const size_t rob[4] = {xb, wb, gb, gb};
  for (int i = 0; i < 4; ++i)
    if (overlap(ro[i], rob[i], conv_state, csb) || overlap(ro[i], rob[i], state, stb) ||
        overlap(ro[i], rob[i], o, ob))
      return fail(GDN_ERR_INVALID_ARG, "decode_tokens: an output overlaps an input");
  if (overlap(conv_state, csb, state, stb) || overlap(conv_state, csb, o, ob) ||
      overlap(state, stb, o, ob))
    return fail(GDN_ERR_INVALID_ARG, "decode_tokens: conv_state, state and o must not overlap");
  return cuda_status(gdn::launch_decode_tokens((int)dt, x, conv_w, conv_state, g, beta, state,
                                               (int)state_dt, o, B, n_tok, Hk, Hv, dk, scale,
                                               (cudaStream_t)stream),
                     "decode_tokens launch");
}

gdn_status_t gdn_decode_tokens(const void* x, const void* conv_w, void* conv_state, const float* g,
                               const float* beta, float* state, void* o, gdn_dtype_t dt, int32_t B,
                               int32_t n_tok, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                               float scale, gdn_stream_t stream) {
  return gdn_decode_tokens_ex(x, conv_w, conv_state, g, beta, state, GDN_F32, o, dt, B, n_tok, Hk,
                              Hv, dk, dv, scale, stream);
}

gdn_status_t gdn_decode_paged(const void* x, int64_t x_stride, const void* conv_w, void* conv_pool,
                              int64_t conv_stride, void* state_pool, int64_t state_stride,
                              gdn_dtype_t state_dt, int32_t n_pages, const int32_t* read_pages,
                              const int32_t* write_pages, const int32_t* n_valid, const float* g,
                              const float* beta, const void* z, int64_t z_stride, const void* norm_w,
                              float eps, void* o, gdn_dtype_t dt, int32_t B, int32_t n_tok, int32_t Hk,
                              int32_t Hv, int32_t dk, int32_t dv, float scale, gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_paged: unknown dtype %d", (int)dt);
  if (!valid_dtype(state_dt)) return fail(GDN_ERR_UNSUPPORTED, "decode_paged: unknown state dtype %d", (int)state_dt);
  if (B < 0) return fail(GDN_ERR_INVALID_ARG, "decode_paged: B = %d < 0", B);
  if (n_tok < 1 || n_tok > 8) return fail(GDN_ERR_INVALID_ARG, "decode_paged: n_tok = %d outside [1, 8]", n_tok);
  if (Hk <= 0 || Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "decode_paged: Hk, Hv must be > 0");
  if (Hv % Hk != 0) return fail(GDN_ERR_UNSUPPORTED, "decode_paged: Hv %% Hk != 0 (%d, %d)", Hv, Hk);
  if (dk != dv || !supported_head_dim(dk))
    return fail(GDN_ERR_UNSUPPORTED, "decode_paged: head dims dk=%d dv=%d (need dk = dv in {16,32,64,128})", dk, dv);
  const int64_t G = Hv / Hk, Cc = 2LL * Hk * dk + (int64_t)Hv * dv;
  if (Cc > 0x7fffffffLL || gdn::decode_paged_smem(n_tok, G, dk) > 224 * 1024)
    return fail(GDN_ERR_UNSUPPORTED, "decode_paged: %d tokens of %lld value heads per key head exceed shared memory",
                n_tok, (long long)G);
  if ((int64_t)B * Hk > 0x7fffffffLL) return fail(GDN_ERR_INVALID_ARG, "decode_paged: B * Hk too large");
  if (n_pages < 0) return fail(GDN_ERR_INVALID_ARG, "decode_paged: n_pages = %d < 0", n_pages);
  if (!(eps >= 0)) return fail(GDN_ERR_INVALID_ARG, "decode_paged: eps must be >= 0");
  const int64_t vals = (int64_t)Hv * dv, page = vals * dk, taps = 3 * Cc;
  if (x_stride == 0) x_stride = Cc;
  if (z_stride == 0) z_stride = vals;
  if (conv_stride == 0) conv_stride = taps;
  if (state_stride == 0) state_stride = page;
  if (x_stride < Cc || x_stride % 8 || z_stride < vals || z_stride % 8 || conv_stride < taps || conv_stride % 8 ||
      state_stride < page || state_stride % 8)
    return fail(GDN_ERR_INVALID_ARG, "decode_paged: strides (x %lld, z %lld, conv %lld, state %lld) must cover a row "
                "or page and be multiples of 8", (long long)x_stride, (long long)z_stride, (long long)conv_stride,
                (long long)state_stride);
  if (B == 0) return ok();
  if (!x || !conv_w || !read_pages || !g || !beta || !o || (n_pages > 0 && (!conv_pool || !state_pool)))
    return fail(GDN_ERR_INVALID_ARG, "decode_paged: x, conv_w, the pools, read_pages, g, beta and o must be non-null");
  if (!z != !norm_w) return fail(GDN_ERR_INVALID_ARG, "decode_paged: z and norm_w come together");
  if (!aligned16(x) || !aligned16(conv_w) || !aligned16(conv_pool) || !aligned16(state_pool) || !aligned16(z) ||
      !aligned16(norm_w) || !aligned16(o))
    return fail(GDN_ERR_INVALID_ARG, "decode_paged: pointers must be 16-byte aligned");
  if (!aligned4(g) || !aligned4(beta) || !aligned4(read_pages) || !aligned4(write_pages) || !aligned4(n_valid))
    return fail(GDN_ERR_INVALID_ARG, "decode_paged: g, beta and the page lists must be 4-byte aligned");
  const size_t es = elt_size(dt), sts = elt_size(state_dt);
  const size_t toks = (size_t)B * n_tok, pages = (size_t)n_pages;
  const size_t cb = pages ? ((pages - 1) * conv_stride + taps) * es : 0;
  const size_t sb = pages ? ((pages - 1) * state_stride + page) * sts : 0;
  const size_t ob = toks * vals * es;
  const void* ro[9] = {x, conv_w, g, beta, z, norm_w, read_pages, write_pages, n_valid};
  const size_t rob[9] = {((toks - 1) * x_stride + Cc) * es, (size_t)Cc * 4 * es, toks * Hv * 4, toks * Hv * 4,
                         ((toks - 1) * z_stride + vals) * es, (size_t)dv * es, (size_t)B * 4, toks * 4, (size_t)B * 4};
  for (int i = 0; i < 9; ++i)
    if (overlap(ro[i], rob[i], conv_pool, cb) || overlap(ro[i], rob[i], state_pool, sb) || overlap(ro[i], rob[i], o, ob))
      return fail(GDN_ERR_INVALID_ARG, "decode_paged: an output or a pool overlaps an input");
  if (overlap(o, ob, conv_pool, cb) || overlap(o, ob, state_pool, sb))
    return fail(GDN_ERR_INVALID_ARG, "decode_paged: o overlaps a pool");
  if (overlap(conv_pool, cb, state_pool, sb)) {
    // interleaved pages: the state's place in a page's record, modulo the common stride
    const int64_t step = conv_stride * (int64_t)es;
    int64_t at = (int64_t)((intptr_t)state_pool - (intptr_t)conv_pool) % step;
    if (at < 0) at += step;
    if (step != state_stride * (int64_t)sts || at < taps * (int64_t)es || at + page * (int64_t)sts > step)
      return fail(GDN_ERR_INVALID_ARG, "decode_paged: conv_pool and state_pool overlap");
  }
  gdn::PagedDecode a{x, x_stride, conv_w, conv_pool, conv_stride, state_pool, state_stride, n_pages, read_pages,
                     write_pages, n_valid, g, beta, z, z_stride, norm_w, eps, o, B, n_tok, Hk, Hv, scale};
  return cuda_status(gdn::launch_decode_paged((int)dt, (int)state_dt, dk, a, (cudaStream_t)stream),
                     "decode_paged launch");
}

// The checks of a copy, before anything is launched; `a` becomes its launch, of no pool where there is
// nothing to copy.
static gdn_status_t pages_copy_args(gdn::PagesCopy& a, const gdn_page_pool_t* pools, int32_t n_pools, int32_t src_pages,
                                    int32_t dst_pages, const int32_t* src, const int32_t* dst, int32_t n, bool plain) {
  if (n < 0 || src_pages < 0 || dst_pages < 0) return fail(GDN_ERR_INVALID_ARG, "pages_copy: negative count");
  if (n_pools < 1 || n_pools > gdn::kPagesMaxPools || !pools)
    return fail(GDN_ERR_INVALID_ARG, "pages_copy: %d pools, expected 1 to %d", n_pools, gdn::kPagesMaxPools);
  if (n > gdn::kPagesMaxList)
    return fail(GDN_ERR_UNSUPPORTED, "pages_copy: %d entries, at most %d a call", n, gdn::kPagesMaxList);
  a = {};
  a.src_pages = src_pages; a.dst_pages = dst_pages; a.src = src; a.dst = dst; a.n = n;
  Pages from[gdn::kPagesMaxPools] = {}, to[gdn::kPagesMaxPools] = {};
  for (int i = 0; i < n_pools; ++i) {
    gdn_page_pool_t p = pools[i];
    if (p.page_bytes <= 0 || p.page_bytes % 16)
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: page_bytes = %lld must be a positive multiple of 16", (long long)p.page_bytes);
    if (p.layers < 0) return fail(GDN_ERR_INVALID_ARG, "pages_copy: negative count");
    if (p.src_page_stride == 0) p.src_page_stride = p.page_bytes;
    if (p.dst_page_stride == 0) p.dst_page_stride = p.page_bytes;
    if (!pages_apart(src_pages, p.src_page_stride, p.layers, p.src_layer_stride, p.page_bytes) ||
        !pages_apart(dst_pages, p.dst_page_stride, p.layers, p.dst_layer_stride, p.page_bytes))
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: strides must be multiples of 16 bytes that keep the pages apart");
    if (n == 0 || p.layers == 0 || src_pages == 0 || dst_pages == 0) continue;
    if (!p.src || !p.dst || !src || !dst)
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: pools and lists must be non-null");
    if (!aligned16(p.src) || !aligned16(p.dst) || !aligned4(src) || !aligned4(dst))
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: pools must be 16-byte aligned, lists 4-byte aligned");
    from[i] = {p.src, p.page_bytes, p.src_page_stride, p.src_layer_stride, src_pages, p.layers};
    to[i] = {p.dst, p.page_bytes, p.dst_page_stride, p.dst_layer_stride, dst_pages, p.layers};
    const bool same = p.src == p.dst;
    if (same && (src_pages != dst_pages || p.src_page_stride != p.dst_page_stride ||
                 (p.layers > 1 && p.src_layer_stride != p.dst_layer_stride)))
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: one pool, but different strides or page counts");
    if (!same && !pools_apart(from[i], to[i])) return fail(GDN_ERR_INVALID_ARG, "pages_copy: the pools overlap");
    if (overlap(src, (size_t)n * 4, p.dst, to[i].extent()) || overlap(dst, (size_t)n * 4, p.dst, to[i].extent()))
      return fail(GDN_ERR_INVALID_ARG, "pages_copy: a list overlaps a destination pool");
    for (int j = 0; j < i; ++j)
      if (!pools_apart(to[i], to[j]) || !pools_apart(to[i], from[j]) || !pools_apart(from[i], to[j]))
        return fail(GDN_ERR_INVALID_ARG, "pages_copy: the pools overlap");
    a.pool[a.n_pools++] = {(const char*)p.src, (char*)p.dst, p.page_bytes, p.src_page_stride, p.src_layer_stride,
                           p.dst_page_stride, p.dst_layer_stride, p.layers, same};
  }
  if (a.n_pools > 0 && !gdn::pages_copy_fits(a, plain))
    return fail(GDN_ERR_UNSUPPORTED, "pages_copy: too much for one launch; split the list");
  return GDN_OK;
}

gdn_status_t gdn_pages_copy(const gdn_page_pool_t* pools, int32_t n_pools, int32_t src_pages,
                            int32_t dst_pages, const int32_t* src, const int32_t* dst, int32_t n,
                            int32_t plain, gdn_stream_t stream) {
  gdn::PagesCopy a;
  const gdn_status_t s = pages_copy_args(a, pools, n_pools, src_pages, dst_pages, src, dst, n, plain != 0);
  if (s != GDN_OK) return s;
  if (a.n_pools == 0) return ok();
  return cuda_status(gdn::launch_pages_copy(a, plain != 0, (cudaStream_t)stream), "pages_copy launch");
}

static gdn_status_t pages_take_args(const int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n,
                                    const int32_t* out) {
  if (n < 0 || n_pages < 0) return fail(GDN_ERR_INVALID_ARG, "pages_take: negative count");
  if (n > gdn::kPagesMaxList)
    return fail(GDN_ERR_UNSUPPORTED, "pages_take: %d entries, at most %d a call", n, gdn::kPagesMaxList);
  if (n == 0) return GDN_OK;
  if (!out || (n_pages > 0 && !refs)) return fail(GDN_ERR_INVALID_ARG, "pages_take: refs and out must be non-null");
  if (!aligned4(refs) || !aligned4(src) || !aligned4(out))
    return fail(GDN_ERR_INVALID_ARG, "pages_take: arrays must be 4-byte aligned");
  if (overlap(out, (size_t)n * 4, refs, (size_t)n_pages * 4) || overlap(out, (size_t)n * 4, src, (size_t)n * 4) ||
      overlap(src, (size_t)n * 4, refs, (size_t)n_pages * 4))
    return fail(GDN_ERR_INVALID_ARG, "pages_take: arrays overlap");
  return GDN_OK;
}

gdn_status_t gdn_pages_take(int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n, int32_t* out,
                            gdn_stream_t stream) {
  const gdn_status_t s = pages_take_args(refs, n_pages, src, n, out);
  if (s != GDN_OK) return s;
  if (n == 0) return ok();
  return cuda_status(gdn::launch_pages_take(refs, n_pages, src, n, out, (cudaStream_t)stream), "pages_take launch");
}

gdn_status_t gdn_pages_ref(int32_t* refs, int32_t n_pages, const int32_t* pages, int32_t n, int32_t delta,
                           gdn_stream_t stream) {
  if (n < 0 || n_pages < 0) return fail(GDN_ERR_INVALID_ARG, "pages_ref: negative count");
  if ((int64_t)n * (delta < 0 ? -(int64_t)delta : delta) > 0x7fffffffLL)
    return fail(GDN_ERR_UNSUPPORTED, "pages_ref: %d entries of %d may pass the range of a count", n, delta);
  if (n == 0 || n_pages == 0) return ok();
  if (!refs || !pages) return fail(GDN_ERR_INVALID_ARG, "pages_ref: refs and pages must be non-null");
  if (!aligned4(refs) || !aligned4(pages)) return fail(GDN_ERR_INVALID_ARG, "pages_ref: arrays must be 4-byte aligned");
  if (overlap(refs, (size_t)n_pages * 4, pages, (size_t)n * 4))
    return fail(GDN_ERR_INVALID_ARG, "pages_ref: pages overlaps refs");
  return cuda_status(gdn::launch_pages_ref(refs, n_pages, pages, n, delta, (cudaStream_t)stream), "pages_ref launch");
}

static gdn_status_t pages_plan_args(const int32_t* refs, int32_t n_pages, const int32_t* table, int32_t n_table,
                                    const int32_t* src, const int32_t* dst, const int32_t* map, const int32_t* n_live) {
  if (n_table < 0 || n_pages < 0) return fail(GDN_ERR_INVALID_ARG, "pages_plan: negative count");
  if (!n_live || (n_pages > 0 && (!refs || !map)) || (n_pages > 1 && (!src || !dst)) || (n_table > 0 && !table))
    return fail(GDN_ERR_INVALID_ARG, "pages_plan: refs, src, dst, map, n_live (and table) must be non-null");
  const void* arr[6] = {refs, table, src, dst, map, n_live};
  const size_t half = (size_t)(n_pages / 2) * 4, all = (size_t)n_pages * 4;
  const size_t by[6] = {all, (size_t)n_table * 4, half, half, all, 4};
  for (int i = 0; i < 6; ++i) {
    if (!aligned4(arr[i])) return fail(GDN_ERR_INVALID_ARG, "pages_plan: arrays must be 4-byte aligned");
    for (int j = 0; j < i; ++j)
      if (overlap(arr[i], by[i], arr[j], by[j])) return fail(GDN_ERR_INVALID_ARG, "pages_plan: arrays overlap");
  }
  return GDN_OK;
}

gdn_status_t gdn_pages_plan(int32_t* refs, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* src,
                            int32_t* dst, int32_t* map, int32_t* n_live, gdn_stream_t stream) {
  const gdn_status_t s = pages_plan_args(refs, n_pages, table, n_table, src, dst, map, n_live);
  if (s != GDN_OK) return s;
  return cuda_status(gdn::launch_pages_plan(refs, n_pages, table, n_table, src, dst, map, n_live, (cudaStream_t)stream),
                     "pages_plan launch");
}

// What a call that changes counts before it copies asks of the pools besides: each is copied within
// itself, and [p, p + bytes) of its counts and lists lies outside.
static bool copies_within(const gdn::PagesCopy& a) {
  for (int i = 0; i < a.n_pools; ++i)
    if (!a.pool[i].same) return false;
  return true;
}
static bool in_pools(const gdn::PagesCopy& a, const void* p, size_t bytes) {
  for (int i = 0; i < a.n_pools; ++i) {
    const gdn::PagePool& q = a.pool[i];
    if (overlap(p, bytes, q.dst, Pages{q.dst, q.page_bytes, q.dst_page, q.dst_layer, a.dst_pages, q.layers}.extent()))
      return true;
  }
  return false;
}

gdn_status_t gdn_pages_fork(int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n, int32_t* out,
                            const gdn_page_pool_t* pools, int32_t n_pools, gdn_stream_t stream) {
  gdn_status_t s = pages_take_args(refs, n_pages, src, n, out);
  if (s != GDN_OK) return s;
  if (n > 0 && !src) return fail(GDN_ERR_INVALID_ARG, "pages_fork: src must be non-null");
  gdn::PagesCopy a;
  s = pages_copy_args(a, pools, n_pools, n_pages, n_pages, src, out, n, true);
  if (s != GDN_OK) return s;
  if (!copies_within(a)) return fail(GDN_ERR_INVALID_ARG, "pages_fork: a pool's src and dst differ");
  if (in_pools(a, refs, (size_t)n_pages * 4)) return fail(GDN_ERR_INVALID_ARG, "pages_fork: refs overlaps a pool");
  if (n == 0) return ok();
  s = cuda_status(gdn::launch_pages_take(refs, n_pages, src, n, out, (cudaStream_t)stream), "pages_fork: taking pages");
  if (s != GDN_OK || a.n_pools == 0) return s;
  return cuda_status(gdn::launch_pages_copy(a, true, (cudaStream_t)stream), "pages_fork: copying pages");
}

gdn_status_t gdn_pages_compact(int32_t* refs, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* src,
                               int32_t* dst, int32_t* map, int32_t* n_live, const gdn_page_pool_t* pools,
                               int32_t n_pools, gdn_stream_t stream) {
  gdn_status_t s = pages_plan_args(refs, n_pages, table, n_table, src, dst, map, n_live);
  if (s != GDN_OK) return s;
  const int32_t half = n_pages / 2, most = gdn::kPagesMaxList;
  gdn::PagesCopy a;
  s = pages_copy_args(a, pools, n_pools, n_pages, n_pages, src, dst, half < most ? half : most, true);
  if (s != GDN_OK) return s;
  if (!copies_within(a)) return fail(GDN_ERR_INVALID_ARG, "pages_compact: a pool's src and dst differ");
  if (half > most && half % most != 0 && a.n_pools > 0) {       // the last part, which may be cut into more tiles
    gdn::PagesCopy b = a;
    b.n = half % most;
    if (!gdn::pages_copy_fits(b, true)) return fail(GDN_ERR_UNSUPPORTED, "pages_compact: too much for one launch");
  }
  if (in_pools(a, refs, (size_t)n_pages * 4) || in_pools(a, table, (size_t)n_table * 4) ||
      in_pools(a, src, (size_t)half * 4) || in_pools(a, dst, (size_t)half * 4) ||
      in_pools(a, map, (size_t)n_pages * 4) || in_pools(a, n_live, 4))
    return fail(GDN_ERR_INVALID_ARG, "pages_compact: counts, lists or table overlap a pool");
  s = cuda_status(gdn::launch_pages_plan(refs, n_pages, table, n_table, src, dst, map, n_live, (cudaStream_t)stream),
                  "pages_compact: planning");
  // the plan's sources and destinations are distinct, so a long list is copied in parts
  for (int32_t i = 0; s == GDN_OK && a.n_pools > 0 && i < half; i += most) {
    a.src = src + i; a.dst = dst + i; a.n = half - i < most ? half - i : most;
    s = cuda_status(gdn::launch_pages_copy(a, true, (cudaStream_t)stream), "pages_compact: copying pages");
  }
  return s;
}

size_t gdn_norm_bwd_workspace_size(int32_t D) { return D > 0 ? (size_t)D * gdn::kNormParts * sizeof(float) : 0; }

static gdn_status_t gated_norm(const char* who, gdn::GatedNorm a, int64_t T, int32_t dv, gdn_dtype_t dt,
                               void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
  if (!valid_dtype(dt)) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, (int)dt);
  if (T < 0) return fail(GDN_ERR_INVALID_ARG, "%s: T = %lld < 0", who, (long long)T);
  if (a.H <= 0) return fail(GDN_ERR_INVALID_ARG, "%s: Hv must be > 0", who);
  if (!supported_head_dim(dv)) return fail(GDN_ERR_UNSUPPORTED, "%s: dv = %d (need 16, 32, 64 or 128)", who, dv);
  if (!(a.eps >= 0)) return fail(GDN_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  if (T > 0x7fffffffLL || T * a.H > 0x7fffffffLL)
    return fail(GDN_ERR_UNSUPPORTED, "%s: %lld tokens of %d heads pass 2^31 - 1 rows; split the call", who, (long long)T, a.H);
  const int64_t vals = (int64_t)a.H * dv;
  if (a.z_stride == 0) a.z_stride = vals;
  if (a.dz_stride == 0) a.dz_stride = vals;
  if (a.z_stride < vals || a.z_stride % 8 || a.dz_stride < vals || a.dz_stride % 8)
    return fail(GDN_ERR_INVALID_ARG, "%s: gate strides must cover a token's heads and be multiples of 8", who);
  if (!aligned16(a.o) || !aligned16(a.z) || !aligned16(a.w) || !aligned16(a.y) || !aligned16(a.dy) ||
      !aligned16(a.dout) || !aligned16(a.dz) || !aligned16(a.dw) || !aligned16(workspace))
    return fail(GDN_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const size_t es = elt_size(dt), ob = (size_t)T * vals * es, wb = (size_t)dv * es;
  const size_t zb = T ? ((size_t)(T - 1) * a.z_stride + vals) * es : 0;
  const size_t dzb = T ? ((size_t)(T - 1) * a.dz_stride + vals) * es : 0;
  const size_t need = a.dw ? gdn_norm_bwd_workspace_size(dv) : 0, dwb = a.dw ? (size_t)dv * 4 : 0;
  a.rows = T * a.H;
  if (!a.back) {
    if (T == 0) return ok();
    if (!a.o || !a.z || !a.w || !a.y) return fail(GDN_ERR_INVALID_ARG, "%s: o, z, w and y must be non-null", who);
    if ((a.y != a.o && overlap(a.y, ob, a.o, ob)) || overlap(a.y, ob, a.z, zb) || overlap(a.y, ob, a.w, wb))
      return fail(GDN_ERR_INVALID_ARG, "%s: y overlaps an input", who);
  } else {
    if (T > 0 && (!a.o || !a.z || !a.w || !a.dy || !a.dout || !a.dz))
      return fail(GDN_ERR_INVALID_ARG, "%s: o, z, w, dy, do and dz must be non-null", who);
    if (workspace_bytes < need || (need > 0 && !workspace))
      return fail(GDN_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", who, workspace_bytes, need);
    a.part = (float*)workspace;
    const void* ro[5] = {a.o, a.z, a.w, a.dy, nullptr};
    const size_t rob[5] = {ob, zb, wb, ob, 0};
    const void* out[4] = {a.dout, a.dz, a.dw, workspace};
    const size_t outb[4] = {ob, dzb, dwb, need};
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < 4; ++j)
        if (!(i == 0 && j == 3 && out[i] == ro[j]) && overlap(out[i], outb[i], ro[j], rob[j]))
          return fail(GDN_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], outb[i], out[j], outb[j])) return fail(GDN_ERR_INVALID_ARG, "%s: outputs overlap", who);
    }
    if (T == 0) {
      if (!a.dw) return ok();
      return cuda_status(cudaMemsetAsync(a.dw, 0, dwb, (cudaStream_t)stream), "gated_norm_bwd: clearing dw");
    }
  }
  return cuda_status(gdn::launch_gated_norm((int)dt, dv, a, (cudaStream_t)stream), who);
}

gdn_status_t gdn_gated_norm(const void* o, const void* z, int64_t z_stride, const void* w, float eps, void* y,
                            gdn_dtype_t dt, int64_t T, int32_t Hv, int32_t dv, gdn_stream_t stream) {
  gdn::GatedNorm a{};
  a.o = o; a.z = z; a.z_stride = z_stride; a.w = w; a.eps = eps; a.y = y; a.H = Hv;
  return gated_norm("gated_norm", a, T, dv, dt, nullptr, 0, stream);
}

gdn_status_t gdn_gated_norm_bwd(const void* o, const void* z, int64_t z_stride, const void* w, float eps,
                                const void* dy, void* dout, void* dz, int64_t dz_stride, float* dw,
                                gdn_dtype_t dt, int64_t T, int32_t Hv, int32_t dv, void* workspace,
                                size_t workspace_bytes, gdn_stream_t stream) {
  gdn::GatedNorm a{};
  a.o = o; a.z = z; a.z_stride = z_stride; a.w = w; a.eps = eps; a.H = Hv; a.back = true;
  a.dy = dy; a.dout = dout; a.dz = dz; a.dz_stride = dz_stride; a.dw = dw;
  return gated_norm("gated_norm_bwd", a, T, dv, dt, workspace, workspace_bytes, stream);
}

static gdn_status_t add_norm_args(const char* who, const gdn::AddNorm& a, gdn_dtype_t dt, gdn_dtype_t res_dt) {
  if (!valid_dtype(dt) || !valid_dtype(res_dt))
    return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d or %d", who, (int)dt, (int)res_dt);
  if (a.rows < 0 || a.rows > 0x7fffffffLL) return fail(GDN_ERR_INVALID_ARG, "%s: T = %lld outside [0, 2^31)", who, (long long)a.rows);
  if (a.D < 1) return fail(GDN_ERR_INVALID_ARG, "%s: D = %d < 1", who, a.D);
  if (a.D > 16384) return fail(GDN_ERR_UNSUPPORTED, "%s: D = %d > 16384", who, a.D);
  if (!(a.eps >= 0)) return fail(GDN_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  return GDN_OK;
}

gdn_status_t gdn_add_norm(const void* x, const void* residual, const void* w, float scale, float w_add, float eps,
                          void* h, gdn_dtype_t res_dt, void* n, gdn_dtype_t dt, int64_t T, int32_t D,
                          gdn_stream_t stream) {
  gdn::AddNorm a{};
  a.x = x; a.w = w; a.scale = scale; a.w_add = w_add; a.eps = eps; a.res = residual; a.h = h; a.n = n;
  a.rows = T; a.D = D;
  const gdn_status_t s = add_norm_args("add_norm", a, dt, res_dt);
  if (s != GDN_OK) return s;
  if (T == 0) return ok();
  if (!x || !residual || !w || !h || !n)
    return fail(GDN_ERR_INVALID_ARG, "add_norm: x, residual, w, h and n must be non-null");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(h) || !aligned16(n))
    return fail(GDN_ERR_INVALID_ARG, "add_norm: pointers must be 16-byte aligned");
  const size_t xb = (size_t)T * D * elt_size(dt), rb = (size_t)T * D * elt_size(res_dt), wb = (size_t)D * elt_size(dt);
  if ((h != residual && overlap(h, rb, residual, rb)) || overlap(h, rb, x, xb) || overlap(h, rb, w, wb) ||
      overlap(n, xb, x, xb) || overlap(n, xb, residual, rb) || overlap(n, xb, w, wb) || overlap(n, xb, h, rb))
    return fail(GDN_ERR_INVALID_ARG, "add_norm: an output overlaps an input or the other output");
  return cuda_status(gdn::launch_add_norm((int)dt, (int)res_dt, a, (cudaStream_t)stream), "add_norm launch");
}

gdn_status_t gdn_add_norm_bwd(const void* h, const void* w, const void* dn, const void* dh, float scale, float w_add,
                              float eps, void* dres, gdn_dtype_t res_dt, void* dx, float* dw, gdn_dtype_t dt,
                              int64_t T, int32_t D, void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
  gdn::AddNorm a{};
  a.w = w; a.scale = scale; a.w_add = w_add; a.eps = eps; a.res = dh; a.h = const_cast<void*>(h);
  a.n = const_cast<void*>(dn); a.dres = dres; a.dx = dx; a.dw = dw; a.part = (float*)workspace;
  a.rows = T; a.D = D; a.back = true;
  const gdn_status_t s = add_norm_args("add_norm_bwd", a, dt, res_dt);
  if (s != GDN_OK) return s;
  if (T > 0 && (!h || !w || !dn || !dres))
    return fail(GDN_ERR_INVALID_ARG, "add_norm_bwd: h, w, dn and dres must be non-null");
  if (!aligned16(h) || !aligned16(w) || !aligned16(dn) || !aligned16(dh) || !aligned16(dres) || !aligned16(dx) ||
      !aligned16(dw) || !aligned16(workspace))
    return fail(GDN_ERR_INVALID_ARG, "add_norm_bwd: pointers must be 16-byte aligned");
  const size_t need = dw ? gdn_norm_bwd_workspace_size(D) : 0;
  if (workspace_bytes < need || (need > 0 && !workspace))
    return fail(GDN_ERR_WORKSPACE, "add_norm_bwd: workspace %zu bytes < %zu needed", workspace_bytes, need);
  const size_t xb = (size_t)T * D * elt_size(dt), rb = (size_t)T * D * elt_size(res_dt);
  const void* ro[4] = {h, w, dn, dh};
  const size_t rob[4] = {rb, (size_t)D * elt_size(dt), xb, rb};
  const void* out[4] = {dres, dx, dw, workspace};
  const size_t outb[4] = {rb, xb, dw ? (size_t)D * 4 : 0, need};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (!(i == 0 && j == 3 && out[i] == ro[j]) && overlap(out[i], outb[i], ro[j], rob[j]))
        return fail(GDN_ERR_INVALID_ARG, "add_norm_bwd: an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], outb[i], out[j], outb[j])) return fail(GDN_ERR_INVALID_ARG, "add_norm_bwd: outputs overlap");
  }
  if (T == 0) {
    if (!dw) return ok();
    return cuda_status(cudaMemsetAsync(dw, 0, (size_t)D * 4, (cudaStream_t)stream), "add_norm_bwd: clearing dw");
  }
  return cuda_status(gdn::launch_add_norm((int)dt, (int)res_dt, a, (cudaStream_t)stream), "add_norm_bwd launch");
}

}  // extern "C"
