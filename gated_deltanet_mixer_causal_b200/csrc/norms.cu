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
#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kGatedThreads = 256;
constexpr int kGatedWarps = kGatedThreads / 32;
constexpr int kAddMaxThreads = 1024;

// sigmoid for the activations' type: accurate for fp32, fast (about 2 ulp) for bf16
template <typename T> __device__ __forceinline__ float sigmoid_for(float z);
template <> __device__ __forceinline__ float sigmoid_for<bf16>(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
template <> __device__ __forceinline__ float sigmoid_for<float>(float z) { return 1.0f / (1.0f + expf(-z)); }

template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// ------------------------------------------------------------------------ gated norm
//
// A lane holds 16 bytes of a row, D / VEC lanes a row; a warp takes U rows per lane at a time,
// so that enough loads are in flight.

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads)
gated_norm_kernel(const T* __restrict__ o, const T* __restrict__ z, int64_t z_stride, const T* __restrict__ w,
                  float eps, T* __restrict__ y, uint32_t rows, uint32_t H) {
  constexpr int VEC = 16 / sizeof(T), LANES = D / VEC, RPW = 32 / LANES, U = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LANES * VEC;
  const uint32_t r0 = (blockIdx.x * kGatedWarps + warp) * (RPW * U) + lane / LANES;
  float wv[VEC], ov[U][VEC], zv[U][VEC];
  VecIO<T, VEC>::load(w + col, wv);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPW;
    if (r < rows) {
      VecIO<T, VEC>::load(o + (int64_t)r * D + col, ov[u]);
      VecIO<T, VEC>::load(z + (int64_t)(r / H) * z_stride + r % H * D + col, zv[u]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) ov[u][i] = zv[u][i] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPW;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(ov[u][i], ov[u][i], ss);
    const float rstd = 1.0f / sqrtf(lanes_sum<LANES>(ss) / D + eps);
    float out[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = ov[u][i] * rstd * wv[i] * (zv[u][i] * sigmoid_for<T>(zv[u][i]));
    if (r < rows) VecIO<T, VEC>::store(y + (int64_t)r * D + col, out);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads)
gated_norm_bwd_kernel(const T* __restrict__ o, const T* __restrict__ z, int64_t z_stride, const T* __restrict__ w,
                      float eps, const T* __restrict__ dy, T* __restrict__ dout, T* __restrict__ dz,
                      int64_t dz_stride, float* __restrict__ part, uint32_t rows, uint32_t H) {
  constexpr int VEC = 16 / sizeof(T), LANES = D / VEC, RPW = 32 / LANES;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % LANES * VEC;
  float wv[VEC], dw[VEC];
  VecIO<T, VEC>::load(w + col, wv);
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = 0.f;
  for (uint64_t g = blockIdx.x * kGatedWarps + warp; g * RPW < rows; g += (uint64_t)gridDim.x * kGatedWarps) {
    const uint32_t r = (uint32_t)(g * RPW) + lane / LANES;
    const bool live = r < rows;
    float ov[VEC], zv[VEC], dv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) ov[i] = zv[i] = dv[i] = 0.f;
    if (live) {
      VecIO<T, VEC>::load(o + (int64_t)r * D + col, ov);
      VecIO<T, VEC>::load(z + (int64_t)(r / H) * z_stride + r % H * D + col, zv);
      VecIO<T, VEC>::load(dy + (int64_t)r * D + col, dv);
    }
    float ss = 0.f, ax = 0.f, da[VEC], dg[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float p = sigmoid_for<T>(zv[i]);
      const float gate = zv[i] * p;
      dg[i] = dv[i] * wv[i] * ov[i] * (p * (1.0f + zv[i] * (1.0f - p)));     // dz / r
      dv[i] *= gate;                                                         // dy SiLU(z)
      da[i] = dv[i] * wv[i];
      ss = fmaf(ov[i], ov[i], ss);
      ax = fmaf(da[i], ov[i], ax);
    }
    ss = lanes_sum<LANES>(ss); ax = lanes_sum<LANES>(ax);
    const float r1 = 1.0f / sqrtf(ss / D + eps), c = ax * r1 * r1 / D;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      dw[i] = fmaf(dv[i], ov[i] * r1, dw[i]);
      da[i] = r1 * (da[i] - c * ov[i]);
      dg[i] *= r1;
    }
    if (live) {
      VecIO<T, VEC>::store(dout + (int64_t)r * D + col, da);
      VecIO<T, VEC>::store(dz + (int64_t)(r / H) * dz_stride + r % H * D + col, dg);
    }
  }
  if (part == nullptr) return;
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

// Sum of v (and u) over the threads of a row; every thread of the CTA calls it.
__device__ __forceinline__ float2 row_sum(float v, float u, float2* sm) {
  v = warp_sum(v); u = warp_sum(u);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(v, u);
  float2* mine = sm + threadIdx.y * warps;
  __syncthreads();                       // the previous row's sums have been read
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(v, u);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int i = 0; i < warps; ++i) { s.x += mine[i].x; s.y += mine[i].y; }
  return s;
}

template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(kAddMaxThreads)
add_norm_kernel(const T* __restrict__ x, const R* res, const T* __restrict__ w, float scale, float w_add, float eps,
                R* h, T* __restrict__ n, int64_t rows, int D) {
  __shared__ float2 sm[32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < rows;
  float v[NV][VEC], wv[NV][VEC], ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
    float xv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[k][i] = xv[i] = wv[k][i] = 0.f;
    if (live && c < D) {
      VecIO<T, VEC>::load(x + row * D + c, xv);
      VecIO<R, VEC>::load(res + row * D + c, v[k]);
      VecIO<T, VEC>::load(w + c, wv[k]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[k][i] = fmaf(scale, xv[i], v[k][i]);
      ss = fmaf(v[k][i], v[k][i], ss);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(ss, 0.f, sm).x / D + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
    if (live && c < D) {
      VecIO<R, VEC>::store(h + row * D + c, v[k]);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[k][i] *= rstd * (wv[k][i] + w_add);
      VecIO<T, VEC>::store(n + row * D + c, v[k]);
    }
  }
}

template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(kAddMaxThreads)
add_norm_bwd_kernel(const R* __restrict__ h, const T* __restrict__ w, const T* __restrict__ dn, const R* dh,
                    float scale, float w_add, float eps, R* dres, T* __restrict__ dx,
                    float* __restrict__ part, int64_t rows, int D) {
  __shared__ float2 sm[32];
  float wv[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) wv[k][i] = dw[k][i] = 0.f;
    if (c < D) VecIO<T, VEC>::load(w + c, wv[k]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) wv[k][i] += w_add;
  }
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < rows;
    float hv[NV][VEC], da[NV][VEC], gv[NV][VEC], ss = 0.f, ax = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) hv[k][i] = da[k][i] = gv[k][i] = 0.f;
      if (live && c < D) {
        VecIO<R, VEC>::load(h + row * D + c, hv[k]);
        VecIO<T, VEC>::load(dn + row * D + c, da[k]);
        if (dh) VecIO<R, VEC>::load(dh + row * D + c, gv[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(hv[k][i], hv[k][i], ss);
        ax = fmaf(da[k][i] * wv[k][i], hv[k][i], ax);
      }
    const float2 s = row_sum(ss, ax, sm);
    const float r1 = 1.0f / sqrtf(s.x / D + eps), cc = s.y * r1 * r1 / D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[k][i] = fmaf(da[k][i], hv[k][i] * r1, dw[k][i]);
        gv[k][i] += r1 * (da[k][i] * wv[k][i] - cc * hv[k][i]);
      }
      if (live && c < D) {
        VecIO<R, VEC>::store(dres + row * D + c, gv[k]);
        if (dx) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) gv[k][i] *= scale;
          VecIO<T, VEC>::store(dx + row * D + c, gv[k]);
        }
      }
    }
  }
  if (part == nullptr) return;
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

struct AddShape { int tx, ty, nv; };

// Threads a row: one run of VEC elements each up to 1024 threads, whole warps; rows narrower
// than 128 threads share a CTA.
AddShape add_shape(int D, int vec) {
  const int runs = (D + vec - 1) / vec;
  AddShape s;
  s.nv = 1;
  while ((runs + s.nv - 1) / s.nv > kAddMaxThreads) s.nv *= 2;
  s.tx = ((runs + s.nv - 1) / s.nv + 31) / 32 * 32;
  s.ty = s.tx >= 128 ? 1 : 128 / s.tx;
  return s;
}

int bwd_parts(int64_t groups) { return (int)(groups < kNormParts ? groups : kNormParts); }

template <typename T, typename R, int VEC, int NV>
cudaError_t add_nv(const AddNorm& a, const AddShape& s, cudaStream_t st) {
  const dim3 block(s.tx, s.ty);
  const int64_t groups = (a.rows + s.ty - 1) / s.ty;
  if (!a.back) {
    add_norm_kernel<T, R, VEC, NV><<<(unsigned)groups, block, 0, st>>>(
        (const T*)a.x, (const R*)a.res, (const T*)a.w, a.scale, a.w_add, a.eps, (R*)a.h, (T*)a.n, a.rows, a.D);
    return cudaGetLastError();
  }
  const int parts = bwd_parts(groups);
  add_norm_bwd_kernel<T, R, VEC, NV><<<parts, block, 0, st>>>(
      (const R*)a.h, (const T*)a.w, (const T*)a.n, (const R*)a.res, a.scale, a.w_add, a.eps, (R*)a.dres, (T*)a.dx,
      a.dw ? a.part : nullptr, a.rows, a.D);
  if (a.dw) norm_dw_kernel<<<(a.D + 31) / 32, dim3(32, 32), 0, st>>>(a.part, parts, a.D, a.dw);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t add_tr(const AddNorm& a, cudaStream_t st) {
  // runs of 8 elements where every row begins on a run's boundary, single elements else
  if (a.D % 8 == 0) {
    const AddShape s = add_shape(a.D, 8);
    return s.nv == 1 ? add_nv<T, R, 8, 1>(a, s, st) : add_nv<T, R, 8, 2>(a, s, st);
  }
  const AddShape s = add_shape(a.D, 1);
  switch (s.nv) {
    case 1: return add_nv<T, R, 1, 1>(a, s, st);
    case 2: return add_nv<T, R, 1, 2>(a, s, st);
    case 4: return add_nv<T, R, 1, 4>(a, s, st);
    case 8: return add_nv<T, R, 1, 8>(a, s, st);
    default: return add_nv<T, R, 1, 16>(a, s, st);
  }
}

template <typename T, int D>
cudaError_t gated_d(const GatedNorm& a, cudaStream_t st) {
  constexpr int RPW = 32 / (D / (16 / (int)sizeof(T)));
  if (!a.back) {
    const int64_t per = (int64_t)kGatedWarps * RPW * 4;
    gated_norm_kernel<T, D><<<(unsigned)((a.rows + per - 1) / per), kGatedThreads, 0, st>>>(
        (const T*)a.o, (const T*)a.z, a.z_stride, (const T*)a.w, a.eps, (T*)a.y, (uint32_t)a.rows, (uint32_t)a.H);
    return cudaGetLastError();
  }
  const int64_t per = (int64_t)kGatedWarps * RPW;
  const int parts = bwd_parts((a.rows + per - 1) / per);
  gated_norm_bwd_kernel<T, D><<<parts, kGatedThreads, 0, st>>>(
      (const T*)a.o, (const T*)a.z, a.z_stride, (const T*)a.w, a.eps, (const T*)a.dy, (T*)a.dout, (T*)a.dz, a.dz_stride,
      a.dw ? a.part : nullptr, (uint32_t)a.rows, (uint32_t)a.H);
  if (a.dw) norm_dw_kernel<<<(D + 31) / 32, dim3(32, 32), 0, st>>>(a.part, parts, D, a.dw);
  return cudaGetLastError();
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
