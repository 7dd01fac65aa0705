// norms.cu -- the norms around a block, forward and backward: the gated norm of the mixer's
// output (per value head) and the residual add with the norm before a block.
//
//   gated:  y = xh w SiLU(z),  xh = o r,  r = 1 / sqrt(mean(o^2) + eps)          per head
//     da = dy SiLU(z) w;  do = r (da - xh mean(da xh));  dz = dy xh w SiLU'(z)
//     dw = sum over rows of dy xh SiLU(z),  SiLU'(z) = p (1 + z (1 - p)), p = sigmoid(z)
//   add:    h = residual + scale x;  n = hh (w + c),  hh = h r                      per token
//     da = dn (w + c);  dres = dh + r (da - hh mean(da hh));  dx = scale dres
//     dw = sum over tokens of dn hh
//
// All four are bound by HBM: every element is read once and written once, the rows stay in
// registers between their reduction and their use. Weight gradients are summed in fp32 in a
// fixed order: registers of a thread over its rows, the threads of a CTA, then the CTAs.
//
// Measured, share of the bytes at the copy rate, bf16: gated 65,536 x 48 x 128 344 us (107 %:
// two reads for a write), its backward 8,192 x 48 x 128 85 us (90 %; the second launch that adds
// up dw and the fp32 instructions of two sigmoid factors an element take the rest); add norm
// backward 16,384 x 4,096 with an fp32 residual 172 us (95 %). A decode batch of 64 tokens takes
// 2.8 and 2.4 us, of which a launch is about 2.
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kGatedThreads = 256;
constexpr int kGatedWarps = kGatedThreads / 32;
constexpr int kGatedBwdBlocks = 3;    // resident CTAs per SM of the backward pass

// sigmoid for the activations' type: accurate for fp32, fast (about 2 ulp) for bf16
template <typename T> __device__ __forceinline__ float sigmoid_for(float z);
template <> __device__ __forceinline__ float sigmoid_for<bf16>(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
template <> __device__ __forceinline__ float sigmoid_for<float>(float z) { return 1.0f / (1.0f + expf(-z)); }

template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// VEC elements as they lie in memory: loads that are ahead of their use hold half the registers
// that bf16 values widened to fp32 would.
template <typename T, int VEC> struct Raw {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr int kWords = kBytes >= 16 ? kBytes / 16 : 1;
  uint4 u[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      static_assert(VEC == 1, "single elements or whole 16-byte words");
      if constexpr (sizeof(T) == 4) u[0].x = *reinterpret_cast<const uint32_t*>(p);
      else u[0].x = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (VEC == 1) {
      f[0] = __uint_as_float(sizeof(T) == 4 ? u[0].x : u[0].x << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            f[i * 4 + j] = __uint_as_float(w[j]);
          } else {
            f[i * 8 + 2 * j] = __uint_as_float(w[j] << 16);
            f[i * 8 + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      }
    }
  }
};

// ------------------------------------------------------------------------ gated norm
//
// A lane holds 16 bytes of a row, D / VEC lanes a row; a lane's loads of U rows are in flight
// together.

// r / H and r % H for r < 2^31, magic = (2^32 - 1) / H: the high product is the quotient or one less
__device__ __forceinline__ uint2 div_rows(uint32_t r, uint32_t H, uint32_t magic) {
  uint32_t q = __umulhi(r, magic), m = r - q * H;
  if (m >= H) { ++q; m -= H; }
  return make_uint2(q, m);
}

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads, 4)
gated_norm_kernel(const T* o, const T* __restrict__ z, int64_t z_stride, const T* __restrict__ w, float eps, T* y,
                  uint32_t rows, uint32_t H, uint32_t magic) {
  constexpr int VEC = 16 / sizeof(T), LANES = D / VEC, RPW = 32 / LANES, U = 4;
  allow_next_grid();
  wait_for_previous_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LANES * VEC;
  const uint32_t r0 = (blockIdx.x * kGatedWarps + warp) * (RPW * U) + lane / LANES;
  Raw<T, VEC> wv, ov[U], zv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPW;
    ov[u].zero(); zv[u].zero();
    if (r < rows) {
      const uint2 th = div_rows(r, H, magic);
      ov[u].load(o + (int64_t)r * D + col);
      zv[u].load(z + (int64_t)th.x * z_stride + th.y * D + col);
    }
  }
  wv.load(w + col);
  float wf[VEC];
  wv.get(wf);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPW;
    float x[VEC], g[VEC], ss = 0.f;
    ov[u].get(x); zv[u].get(g);
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(x[i], x[i], ss);
    const float rstd = rsqrtf(lanes_sum<LANES>(ss) * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = x[i] * rstd * wf[i] * (g[i] * sigmoid_for<T>(g[i]));
    if (r < rows) VecIO<T, VEC>::store(y + (int64_t)r * D + col, x);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads, kGatedBwdBlocks)
gated_norm_bwd_kernel(const T* __restrict__ o, const T* __restrict__ z, int64_t z_stride, const T* __restrict__ w,
                      float eps, const T* dy, T* dout, T* __restrict__ dz, int64_t dz_stride,
                      float* __restrict__ part, uint32_t rows, uint32_t H, uint32_t magic) {
  constexpr int VEC = 16 / sizeof(T), LANES = D / VEC, RPW = 32 / LANES, U = 2;
  wait_for_previous_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LANES * VEC;
  float wf[VEC], dw[VEC];
  VecIO<T, VEC>::load(w + col, wf);
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = 0.f;
  for (uint64_t g = blockIdx.x * kGatedWarps + warp; g * (RPW * U) < rows; g += (uint64_t)gridDim.x * kGatedWarps) {
    const uint32_t r0 = (uint32_t)(g * (RPW * U)) + lane / LANES;
    Raw<T, VEC> ov[U], zv[U], dv[U];
    uint2 th[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = r0 + u * RPW;
      ov[u].zero(); zv[u].zero(); dv[u].zero();
      th[u] = div_rows(r, H, magic);
      if (r < rows) {
        ov[u].load(o + (int64_t)r * D + col);
        zv[u].load(z + (int64_t)th[u].x * z_stride + th[u].y * D + col);
        dv[u].load(dy + (int64_t)r * D + col);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = r0 + u * RPW;
      float x[VEC], gz[VEC], d[VEC], da[VEC], ss = 0.f, ax = 0.f;
      ov[u].get(x); zv[u].get(gz); dv[u].get(d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float p = sigmoid_for<T>(gz[i]), dw_ = d[i] * wf[i];
        const float slope = p * fmaf(gz[i], 1.0f - p, 1.0f);
        d[i] *= gz[i] * p;                                     // dy SiLU(z)
        gz[i] = dw_ * x[i] * slope;                            // dz / r
        da[i] = d[i] * wf[i];
        ss = fmaf(x[i], x[i], ss);
        ax = fmaf(da[i], x[i], ax);
      }
      ss = lanes_sum<LANES>(ss); ax = lanes_sum<LANES>(ax);
      const float r1 = rsqrtf(ss * (1.0f / D) + eps), c = ax * r1 * r1 * (1.0f / D);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[i] = fmaf(d[i], x[i] * r1, dw[i]);
        da[i] = r1 * fmaf(-c, x[i], da[i]);
        gz[i] *= r1;
      }
      if (r < rows) {
        VecIO<T, VEC>::store(dout + (int64_t)r * D + col, da);
        VecIO<T, VEC>::store(dz + (int64_t)th[u].x * dz_stride + th[u].y * D + col, gz);
      }
    }
  }
  if (part == nullptr) return;
  allow_next_grid();
  __shared__ float acc[kGatedWarps][D];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
#pragma unroll
    for (int m = LANES; m < 32; m <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], m);
    if (lane < LANES) acc[warp][col + i] = dw[i];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kGatedWarps; ++k) s += acc[k][threadIdx.x];
    part[(int64_t)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw[c] = sum over the CTAs' parts, in a fixed order: 32 columns x 32 slices of the parts a CTA
__global__ void __launch_bounds__(1024)
norm_dw_kernel(const float* __restrict__ part, int n_part, int D, float* __restrict__ dw) {
  __shared__ float acc[32][33];
  allow_next_grid();
  wait_for_previous_grid();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < D)
    for (int p = threadIdx.y; p < n_part; p += 32) s += part[(int64_t)p * D + c];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += acc[k][threadIdx.x];
    dw[c] = s;
  }
}

// -------------------------------------------------------------------------- add norm
//
// blockDim = (threads a row, rows a CTA); a thread holds NV runs of VEC elements of its row,
// run k at column (k * blockDim.x + threadIdx.x) * VEC.

// Sums of v and u over the threads of a row; every thread of the CTA calls it. The first exchange
// of a warp leaves v's half sums in its lower lanes and u's in its upper ones, so one tree of
// shuffles serves both. sm holds two buffers that successive calls use in turn (`turn`), so one
// barrier a call is enough: a buffer is written again only behind the next call's barrier.
__device__ __forceinline__ float2 row_sum(float v, float u, float (*sm)[64], int turn) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool up = lane & 16;
  float a = (up ? u : v) + __shfl_xor_sync(0xffffffffu, up ? v : u, 16);
  a = lanes_sum<16>(a);
  if (warps > 1) {
    float* mine = sm[turn & 1] + threadIdx.y * warps * 2 + (up ? warps : 0);
    if ((lane & 15) == 0) mine[threadIdx.x >> 5] = a;
    __syncthreads();
    const int i = lane & 15;
    a = i < warps ? mine[i] : 0.f;
    if (i + 16 < warps) a += mine[i + 16];
    a = lanes_sum<16>(a);
  }
  return make_float2(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, a, 16));
}

template <typename T, typename R, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT)
add_norm_kernel(const T* __restrict__ x, const R* res, const T* __restrict__ w, float scale, float w_add, float eps,
                R* h, T* __restrict__ n, int64_t rows, int D) {
  __shared__ float sm[2][64];
  allow_next_grid();
  wait_for_previous_grid();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < rows;
  float v[NV][VEC], ss = 0.f;
  Raw<T, VEC> wv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
    Raw<T, VEC> xr;
    Raw<R, VEC> rr;
    xr.zero(); rr.zero(); wv[k].zero();
    if (live && c < D) {
      xr.load(x + row * D + c);
      rr.load(res + row * D + c);
      wv[k].load(w + c);
    }
    float xv[VEC];
    xr.get(xv); rr.get(v[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[k][i] = fmaf(scale, xv[i], v[k][i]);
      ss = fmaf(v[k][i], v[k][i], ss);
    }
  }
  const float rstd = rsqrtf(row_sum(ss, 0.f, sm, 0).x * (1.0f / D) + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
    if (live && c < D) {
      VecIO<R, VEC>::store(h + row * D + c, v[k]);
      float wf[VEC];
      wv[k].get(wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[k][i] *= rstd * (wf[i] + w_add);
      VecIO<T, VEC>::store(n + row * D + c, v[k]);
    }
  }
}

// A CTA takes every gridDim.x-th group of rows; a thread keeps its columns' weight gradient in
// registers over them and has the next row's loads in flight while it works on one.
template <typename T, typename R, int VEC, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
add_norm_bwd_kernel(const R* __restrict__ h, const T* __restrict__ w, const T* __restrict__ dn, const R* dh,
                    float scale, float w_add, float eps, R* dres, T* __restrict__ dx,
                    float* __restrict__ part, int64_t rows, int D) {
  __shared__ float sm[2][64];
  wait_for_previous_grid();
  const float inv_d = 1.0f / D;
  float dw[NV][VEC];
  Raw<T, VEC> wv[NV], dr[NV];
  Raw<R, VEC> hr[NV], gr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
    wv[k].zero();
    if (c < D) wv[k].load(w + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[k][i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  auto fetch_row = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * VEC;
      hr[k].zero(); dr[k].zero();
      if (r < rows && c < D) { hr[k].load(h + r * D + c); dr[k].load(dn + r * D + c); }
    }
  };
  auto fetch_dh = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * VEC;
      gr[k].zero();
      if (dh && r < rows && c < D) gr[k].load(dh + r * D + c);
    }
  };
  fetch_row(row);
  fetch_dh(row);
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += step, row += step, ++turn) {
    float hv[NV][VEC], da[NV][VEC], ss = 0.f, ax = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) { hr[k].get(hv[k]); dr[k].get(da[k]); }
    fetch_row(row + step);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float wf[VEC];
      wv[k].get(wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(hv[k][i], hv[k][i], ss);
        ax = fmaf(da[k][i] * (wf[i] + w_add), hv[k][i], ax);
      }
    }
    const float2 s = row_sum(ss, ax, sm, turn);
    const float r1 = rsqrtf(fmaf(s.x, inv_d, eps)), cc = -s.y * r1 * r1 * inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * VEC;
      float wf[VEC], gv[VEC];
      wv[k].get(wf);
      gr[k].get(gv);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[k][i] = fmaf(da[k][i], hv[k][i] * r1, dw[k][i]);
        gv[i] = fmaf(r1, fmaf(da[k][i], wf[i] + w_add, cc * hv[k][i]), gv[i]);
      }
      if (row < rows && c < D) {
        VecIO<R, VEC>::store(dres + row * D + c, gv);
        if (dx) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) gv[i] *= scale;
          VecIO<T, VEC>::store(dx + row * D + c, gv);
        }
      }
    }
    fetch_dh(row + step);
  }
  if (part == nullptr) return;
  allow_next_grid();
  // the rows of the CTA take their turns at one row of parts
  float* mine = part + (int64_t)blockIdx.x * D;
  for (int y = 0; y < blockDim.y; ++y) {
    if (threadIdx.y == y) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c < D) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) mine[c + i] = y ? mine[c + i] + dw[k][i] : dw[k][i];
        }
      }
    }
    __syncthreads();
  }
}

struct AddShape { int tx, ty; };

// Threads a row when each holds nv runs of vec elements, in whole warps; rows narrower than 256
// threads share a CTA.
AddShape add_shape(int D, int vec, int nv) {
  const int runs = (D + vec - 1) / vec;
  AddShape s;
  s.tx = ((runs + nv - 1) / nv + 31) / 32 * 32;
  s.ty = s.tx >= 256 ? 1 : 256 / s.tx;
  return s;
}

template <typename T, typename R, int VEC, int NV, int MAXT>
cudaError_t add_fwd(const AddNorm& a, cudaStream_t st) {
  const AddShape s = add_shape(a.D, VEC, NV);
  return launch_overlapped(add_norm_kernel<T, R, VEC, NV, MAXT>, dim3((unsigned)((a.rows + s.ty - 1) / s.ty)),
                           dim3(s.tx, s.ty), 0, st, (const T*)a.x, (const R*)a.res, (const T*)a.w, a.scale, a.w_add,
                           a.eps, (R*)a.h, (T*)a.n, a.rows, a.D);
}

// MINB CTAs of the backward pass are resident on each of 148 SMs; no more are launched, so that
// every CTA begins at once and takes the same number of rows.
template <typename T, typename R, int VEC, int NV, int MAXT, int MINB>
cudaError_t add_bwd(const AddNorm& a, cudaStream_t st) {
  static_assert(MINB * 148 <= kNormParts, "parts in the workspace");
  const AddShape s = add_shape(a.D, VEC, NV);
  const int64_t groups = (a.rows + s.ty - 1) / s.ty;
  const int parts = (int)(groups < MINB * 148 ? groups : MINB * 148);
  const cudaError_t e = launch_overlapped(add_norm_bwd_kernel<T, R, VEC, NV, MAXT, MINB>, dim3(parts), dim3(s.tx, s.ty),
                                          0, st, (const R*)a.h, (const T*)a.w, (const T*)a.n, (const R*)a.res, a.scale,
                                          a.w_add, a.eps, (R*)a.dres, (T*)a.dx, a.dw ? a.part : nullptr, a.rows, a.D);
  return e != cudaSuccess || !a.dw ? e : launch_overlapped(norm_dw_kernel, dim3((a.D + 31) / 32), dim3(32, 32), 0, st,
                                                           a.part, parts, a.D, a.dw);
}

template <typename T, typename R>
cudaError_t add_tr(const AddNorm& a, cudaStream_t st) {
  // runs of 8 elements where every row begins on a run's boundary, single elements else
  if (a.D % 8 == 0) {
    if (a.back) {
      if (a.D <= 2048) return add_bwd<T, R, 8, 1, 256, 4>(a, st);
      if (a.D <= 4096) return add_bwd<T, R, 8, 2, 256, 2>(a, st);
      if (a.D <= 8192) return add_bwd<T, R, 8, 2, 512, 1>(a, st);
      return add_bwd<T, R, 8, 2, 1024, 1>(a, st);
    }
    if (a.D <= 2048) return add_fwd<T, R, 8, 1, 256>(a, st);
    if (a.D <= 8192) return add_fwd<T, R, 8, 1, 1024>(a, st);
    return add_fwd<T, R, 8, 2, 1024>(a, st);
  }
  if (a.back) {
    if (a.D <= 1024) return add_bwd<T, R, 1, 4, 256, 4>(a, st);
    if (a.D <= 4096) return add_bwd<T, R, 1, 8, 512, 2>(a, st);
    return add_bwd<T, R, 1, 16, 1024, 1>(a, st);
  }
  if (a.D <= 1024) return add_fwd<T, R, 1, 4, 256>(a, st);
  if (a.D <= 4096) return add_fwd<T, R, 1, 8, 512>(a, st);
  return add_fwd<T, R, 1, 16, 1024>(a, st);
}

template <typename T, int D>
cudaError_t gated_d(const GatedNorm& a, cudaStream_t st) {
  constexpr int RPW = 32 / (D / (16 / (int)sizeof(T)));
  if (!a.back) {
    const int64_t per = (int64_t)kGatedWarps * RPW * 4;
    return launch_overlapped(gated_norm_kernel<T, D>, dim3((unsigned)((a.rows + per - 1) / per)), dim3(kGatedThreads), 0,
                             st, (const T*)a.o, (const T*)a.z, a.z_stride, (const T*)a.w, a.eps, (T*)a.y,
                             (uint32_t)a.rows, (uint32_t)a.H, 0xFFFFFFFFu / (uint32_t)a.H);
  }
  const int64_t per = (int64_t)kGatedWarps * RPW * 2;
  const int64_t groups = (a.rows + per - 1) / per;
  const int parts = (int)(groups < kGatedBwdBlocks * 148 ? groups : kGatedBwdBlocks * 148);   // one wave
  const cudaError_t e = launch_overlapped(
      gated_norm_bwd_kernel<T, D>, dim3(parts), dim3(kGatedThreads), 0, st, (const T*)a.o, (const T*)a.z, a.z_stride,
      (const T*)a.w, a.eps, (const T*)a.dy, (T*)a.dout, (T*)a.dz, a.dz_stride, a.dw ? a.part : nullptr, (uint32_t)a.rows,
      (uint32_t)a.H, 0xFFFFFFFFu / (uint32_t)a.H);
  return e != cudaSuccess || !a.dw ? e : launch_overlapped(norm_dw_kernel, dim3((D + 31) / 32), dim3(32, 32), 0, st,
                                                           a.part, parts, D, a.dw);
}

template <typename T>
cudaError_t gated_t(int d, const GatedNorm& a, cudaStream_t st) {
  switch (d) {
    case 16: return gated_d<T, 16>(a, st);
    case 32: return gated_d<T, 32>(a, st);
    case 64: return gated_d<T, 64>(a, st);
    default: return gated_d<T, 128>(a, st);
  }
}

}  // namespace

cudaError_t launch_gated_norm(int dtype, int d, const GatedNorm& a, cudaStream_t st) {
  return dtype == kF32 ? gated_t<float>(d, a, st) : gated_t<bf16>(d, a, st);
}

cudaError_t launch_add_norm(int dtype, int res_dtype, const AddNorm& a, cudaStream_t st) {
  if (dtype == kF32) return res_dtype == kF32 ? add_tr<float, float>(a, st) : add_tr<float, bf16>(a, st);
  return res_dtype == kF32 ? add_tr<bf16, float>(a, st) : add_tr<bf16, bf16>(a, st);
}

}  // namespace gdn
