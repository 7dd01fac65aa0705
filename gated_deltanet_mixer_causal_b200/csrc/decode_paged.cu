// decode_paged.cu -- up to n_tok (1..8) tokens for each of B sequences whose conv taps and
// states lie in pages of a pool: every sequence reads one page and writes the state after each
// of its tokens to a page of its own choice (or after its last token back to the page it read).
//
// Same update as decode_tokens.cu (Qwen3.5 page, section 5: decay, then the delta write along
// k; section 8: decode is a state-update stream). With s a row of the state:
//   sk = s.k_t, sq = s.q_t;  u = beta_t (v_t,i - alpha_t sk);  s <- alpha_t s + u k_t
//   o_t,i = scale (alpha_t sq + u (k_t.q_t))
// and, when a gate is given, the block's output norm is applied where the head's whole output
// lies in shared memory:  o_t <- o_t / sqrt(mean(o_t^2) + eps) * w * SiLU(z_t).
//
// One CTA owns one (sequence, key head): the conv channels of its q and k and of its G value
// heads, so the in-place tap shift is race-free.
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kEps = 1e-6f;
constexpr int kMaxTok = 8;
constexpr int kSeg = 16;           // state columns per lane
constexpr int kRows = 2;           // state rows per lane and pass

// Four consecutive state values, streamed (evict-first).
template <typename S> struct Quad;
template <> struct Quad<float> {
  static __device__ __forceinline__ float4 load(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
  static __device__ __forceinline__ void store(float* p, float4 v) { __stcs(reinterpret_cast<float4*>(p), v); }
};
template <> struct Quad<bf16> {
  static __device__ __forceinline__ float4 load(const bf16* p) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  static __device__ __forceinline__ void store(bf16* p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)));
  }
};

// z * sigmoid(z) for the activations' type: fp32 with the accurate exponential and division,
// whose errors would otherwise show in fp32 results; bf16 with the fast ones.
template <typename T> __device__ __forceinline__ float silu_for(float z);
template <> __device__ __forceinline__ float silu_for<bf16>(float z) { return silu(z); }
template <> __device__ __forceinline__ float silu_for<float>(float z) { return z / (1.0f + expf(-z)); }

template <typename T, typename S, int D>
__global__ void __launch_bounds__(kThreads, 2)
decode_paged_kernel(const PagedDecode a) {
  constexpr int L = D / kSeg;              // lanes per state row
  constexpr int RPW = 32 / L;              // rows a warp covers at once
  constexpr int RPP = RPW * kRows;         // rows of a warp's pass
  const int G = a.Hv / a.Hk, n_tok = a.n_tok;
  const int32_t Cc = 2 * a.Hk * D + a.Hv * D;
  const int64_t b = blockIdx.x / a.Hk;
  const int hk = blockIdx.x % a.Hk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = G * D;

  int nv = n_tok;
  if (a.n_valid) nv = min(max(a.n_valid[b], 0), n_tok);
  if (nv == 0) return;                     // nothing of this sequence is read or written
  const int32_t rp = a.read_pages[b];
  const bool fresh = rp < 0 || rp >= a.n_pages;

  extern __shared__ float smem[];
  float* qk = smem;                        // [n_tok][2 D] q | k
  float* vo = qk + n_tok * 2 * D;          // [n_tok][rows] v, then o in its place
  float* kqs = vo + n_tok * rows;          // [kMaxTok] k_t.q_t
  float2* ab = reinterpret_cast<float2*>(kqs + kMaxTok);        // [G][n_tok] (alpha, beta)
  __shared__ int32_t wp[kMaxTok];          // page of the state after token t, -1: not stored

  if (threadIdx.x < kMaxTok) {
    const int t = threadIdx.x;
    int32_t p = -1;
    if (t < nv) {
      if (a.write_pages) p = a.write_pages[b * n_tok + t];
      else if (t == nv - 1) p = rp;
      if (p < 0 || p >= a.n_pages) p = -1;
    }
    wp[t] = p;
  }
  __syncthreads();

  // 1. conv + SiLU over this CTA's channels; the window slides in registers
  const T* x = static_cast<const T*>(a.x);
  T* conv = static_cast<T*>(a.conv_pool);
  for (int lc = threadIdx.x * 4; lc < 2 * D + rows; lc += kThreads * 4) {
    int gc;
    if (lc < D) gc = hk * D + lc;
    else if (lc < 2 * D) gc = a.Hk * D + hk * D + (lc - D);
    else gc = 2 * a.Hk * D + hk * G * D + (lc - 2 * D);
    float w0[4], w1[4], w2[4], cur[4], wr[16];
    VecIO<T, 16>::load(static_cast<const T*>(a.conv_w) + (int64_t)gc * 4, wr);
    if (fresh) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w0[i] = w1[i] = w2[i] = 0.f;
    } else {
      const T* cs = conv + (int64_t)rp * a.conv_stride + gc;
      VecIO<T, 4>::load(cs, w0); VecIO<T, 4>::load(cs + Cc, w1); VecIO<T, 4>::load(cs + 2 * Cc, w2);
    }
    for (int t = 0; t < nv; ++t) {
      VecIO<T, 4>::load(x + (b * n_tok + t) * a.x_stride + gc, cur);
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float z = wr[i * 4] * w0[i];
        z = fmaf(wr[i * 4 + 1], w1[i], z);
        z = fmaf(wr[i * 4 + 2], w2[i], z);
        z = fmaf(wr[i * 4 + 3], cur[i], z);
        y[i] = silu_for<T>(z);
      }
      float* dst = lc < 2 * D ? qk + t * 2 * D + lc : vo + t * rows + (lc - 2 * D);
      *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
      if (wp[t] >= 0) {
        T* cs = conv + (int64_t)wp[t] * a.conv_stride + gc;
        VecIO<T, 4>::store(cs, w1); VecIO<T, 4>::store(cs + Cc, w2); VecIO<T, 4>::store(cs + 2 * Cc, cur);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) { w0[i] = w1[i]; w1[i] = w2[i]; w2[i] = cur[i]; }
    }
  }
  __syncthreads();

  // 2. q_t and k_t L2-normalised in place (a warp per token), k_t.q_t beside them
  constexpr int VEC = D >= 32 ? D / 32 : 1;
  for (int t = warp; t < nv; t += kWarps) {
    float* yt = qk + t * 2 * D;
    const bool active = lane * VEC < D;
    float qv[VEC], kv[VEC], qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      qv[j] = active ? yt[lane * VEC + j] : 0.f;
      kv[j] = active ? yt[D + lane * VEC + j] : 0.f;
      qq = fmaf(qv[j], qv[j], qq); kk = fmaf(kv[j], kv[j], kk); kq = fmaf(kv[j], qv[j], kq);
    }
    qq = warp_sum(qq); kk = warp_sum(kk); kq = warp_sum(kq);
    const float iq = 1.0f / sqrtf(qq + kEps), ik = 1.0f / sqrtf(kk + kEps);
    if (active) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) { yt[lane * VEC + j] = qv[j] * iq; yt[D + lane * VEC + j] = kv[j] * ik; }
    }
    if (lane == 0) kqs[t] = kq * iq * ik;
  }
  for (int i = threadIdx.x; i < G * nv; i += kThreads) {
    const int hh = i / nv, t = i % nv;
    const int64_t gi = (b * n_tok + t) * a.Hv + hk * G + hh;
    ab[hh * n_tok + t] = make_float2(expf(a.g[gi]), a.beta[gi]);
  }
  __syncthreads();

  // 3. the state rows, each through every token
  const int seg = lane % L;
  const S* src = static_cast<const S*>(a.state_pool) + (fresh ? 0 : (int64_t)rp * a.state_stride);
  const int64_t head0 = (int64_t)hk * G * D * D;        // this CTA's first element in a page
  for (int p0 = warp * RPP; p0 < rows; p0 += kWarps * RPP) {
    float s[kRows][kSeg];
    int r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      r[i] = p0 + i * RPW + lane / L;
#pragma unroll
      for (int j = 0; j < kSeg; j += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!fresh && r[i] < rows) v = Quad<S>::load(src + head0 + (int64_t)r[i] * D + seg * 4 + j * L);
        s[i][j] = v.x; s[i][j + 1] = v.y; s[i][j + 2] = v.z; s[i][j + 3] = v.w;
      }
    }
    for (int t = 0; t < nv; ++t) {
      const float* qt = qk + t * 2 * D + seg * 4;
      float kv[kSeg], sk[kRows], sq[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) sk[i] = sq[i] = 0.f;
#pragma unroll
      for (int j = 0; j < kSeg; j += 4) {
        const float4 q4 = *reinterpret_cast<const float4*>(qt + j * L);
        const float4 k4 = *reinterpret_cast<const float4*>(qt + D + j * L);
        kv[j] = k4.x; kv[j + 1] = k4.y; kv[j + 2] = k4.z; kv[j + 3] = k4.w;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          sk[i] = fmaf(s[i][j], k4.x, sk[i]); sk[i] = fmaf(s[i][j + 1], k4.y, sk[i]);
          sk[i] = fmaf(s[i][j + 2], k4.z, sk[i]); sk[i] = fmaf(s[i][j + 3], k4.w, sk[i]);
          sq[i] = fmaf(s[i][j], q4.x, sq[i]); sq[i] = fmaf(s[i][j + 1], q4.y, sq[i]);
          sq[i] = fmaf(s[i][j + 2], q4.z, sq[i]); sq[i] = fmaf(s[i][j + 3], q4.w, sq[i]);
        }
      }
#pragma unroll
      for (int m = L / 2; m >= 1; m >>= 1)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], m);
          sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], m);
        }
      const int32_t to = wp[t];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool live = r[i] < rows;
        const int rr = live ? r[i] : 0;
        const float2 sc = ab[(rr / D) * n_tok + t];
        const float u = sc.y * (vo[t * rows + rr] - sc.x * sk[i]);
#pragma unroll
        for (int j = 0; j < kSeg; ++j) s[i][j] = fmaf(sc.x, s[i][j], u * kv[j]);
        __syncwarp();                       // every lane of the row has read v before o replaces it
        if (live && seg == 0) vo[t * rows + rr] = a.scale * fmaf(sc.x, sq[i], u * kqs[t]);
        if (live && to >= 0) {
          S* dst = static_cast<S*>(a.state_pool) + (int64_t)to * a.state_stride + head0 + (int64_t)rr * D + seg * 4;
#pragma unroll
          for (int j = 0; j < kSeg; j += 4)
            Quad<S>::store(dst + j * L, make_float4(s[i][j], s[i][j + 1], s[i][j + 2], s[i][j + 3]));
        }
      }
    }
  }
  __syncthreads();

  // 4. outputs, normalised and gated when asked (a warp per token and head)
  T* o = static_cast<T*>(a.o);
  for (int e = warp; e < nv * G; e += kWarps) {
    const int t = e / G, hh = e % G;
    const float* row = vo + t * rows + hh * D;
    const int64_t tok = b * n_tok + t;
    T* dst = o + (tok * a.Hv + hk * G + hh) * D;
    float rstd = 1.f;
    if (a.z) {
      float ss = 0.f;
      for (int i = lane; i < D; i += 32) ss = fmaf(row[i], row[i], ss);
      rstd = 1.0f / sqrtf(warp_sum(ss) / D + a.eps);
    }
    for (int i = lane; i < D; i += 32) {
      float v = row[i];
      if (a.z) {
        const float z = to_f(static_cast<const T*>(a.z)[tok * a.z_stride + (hk * G + hh) * D + i]);
        v = v * rstd * to_f(static_cast<const T*>(a.norm_w)[i]) * silu_for<T>(z);
      }
      dst[i] = from_f<T>(v);
    }
  }
}

template <typename T, typename S, int D>
cudaError_t launch_d(const PagedDecode& a, cudaStream_t st) {
  const size_t smem = decode_paged_smem(a.n_tok, a.Hv / a.Hk, D);
  if (smem > 40 * 1024) {   // beside the kernel's few static bytes
    cudaError_t e = cudaFuncSetAttribute(decode_paged_kernel<T, S, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  decode_paged_kernel<T, S, D><<<(unsigned)((int64_t)a.B * a.Hk), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, typename S>
cudaError_t launch_ts(const PagedDecode& a, int d, cudaStream_t st) {
  switch (d) {
    case 16: return launch_d<T, S, 16>(a, st);
    case 32: return launch_d<T, S, 32>(a, st);
    case 64: return launch_d<T, S, 64>(a, st);
    default: return launch_d<T, S, 128>(a, st);
  }
}

}  // namespace

size_t decode_paged_smem(int n_tok, int64_t G, int d) {
  // q | k, v (then o), k.q, (alpha, beta)
  return sizeof(float) * (size_t)((int64_t)n_tok * (2 + G) * d + kMaxTok + 2 * G * n_tok);
}

cudaError_t launch_decode_paged(int dtype, int state_dtype, int d, const PagedDecode& a, cudaStream_t st) {
  if (dtype == kF32)
    return state_dtype == kF32 ? launch_ts<float, float>(a, d, st) : launch_ts<float, bf16>(a, d, st);
  return state_dtype == kF32 ? launch_ts<bf16, float>(a, d, st) : launch_ts<bf16, bf16>(a, d, st);
}

}  // namespace gdn
