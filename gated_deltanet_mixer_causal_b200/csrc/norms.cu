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
// Measured by graph replay, share of the bytes at the copy rate, bf16: gated 65,536 x 48 x 128 344 us
// on one card and 373 on another (107 and 99 %: two reads for a write; 377 as a call), its backward
// 8,192 x 48 x 128 87 to 90 us (88 %; the second launch that adds up dw and the fp32 instructions of two
// sigmoid factors an element take the rest; 93 as a call); add norm backward 16,384 x 4,096 with an fp32
// residual 173 us (95 %; 179 as a call). All in fp32: gated 16,384 x 48 173 us (106 %), backward 8,192 x
// 48 157 (98 %), add norm 16,384 x 4,096 163 (100 %), backward 222 (92 %). A decode batch of 64 tokens
// takes 2.7 and 2.0 us, of which a launch is most.
#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

// No input is `const __restrict__`: these kernels begin while the grid before them, which may have
// made their inputs, still runs, and the qualifier would let their loads move ahead of the wait.

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

// VEC elements (whole 16-byte words) as they lie in memory: loads that are ahead of their use hold
// half the registers that bf16 values widened to fp32 would.
template <typename T, int VEC> struct Raw {
  static constexpr int kWords = VEC * (int)sizeof(T) / 16, kPer = 16 / (int)sizeof(T);
  uint4 u[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  // what the backward passes take for a value behind the last row: its 1 / rms is finite with any eps,
  // so that its zero gradients add zeros to dw (zeros and eps = 0 would give 0 * inf)
  __device__ __forceinline__ void ones() {
    const uint32_t w = sizeof(T) == 4 ? 0x3F800000u : 0x3F803F80u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = make_uint4(w, w, w, w);
  }
  // the elements [from, to) of the run one by one, zeros for the others
  __device__ __forceinline__ void load_part(const T* p, int from, int to) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = i * kPer + j;
        if (e < from || e >= to) continue;
        if constexpr (sizeof(T) == 4) w[j] = reinterpret_cast<const uint32_t*>(p)[e];
        else w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (j % 2 * 16);
      }
      u[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // zeros outside [from, to)
  __device__ __forceinline__ void keep(int from, int to) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = i * kPer + j;
        const uint32_t on = e >= from && e < to ? 0xFFFFFFFFu : 0u;
        if constexpr (sizeof(T) == 4) m[j] = on;
        else m[j / 2] |= on & (j % 2 ? 0xFFFF0000u : 0xFFFFu);
      }
      u[i].x &= m[0]; u[i].y &= m[1]; u[i].z &= m[2]; u[i].w &= m[3];
    }
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
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
gated_norm_kernel(const T* o, const T* z, int64_t z_stride, const T* w, float eps, T* y,
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
      zv[u].load(z + (int64_t)th.x * z_stride + (int64_t)th.y * D + col);
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
gated_norm_bwd_kernel(const T* o, const T* z, int64_t z_stride, const T* w,
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
      ov[u].ones(); zv[u].zero(); dv[u].zero();
      th[u] = div_rows(r, H, magic);
      if (r < rows) {
        ov[u].load(o + (int64_t)r * D + col);
        zv[u].load(z + (int64_t)th[u].x * z_stride + (int64_t)th[u].y * D + col);
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
        VecIO<T, VEC>::store(dz + (int64_t)th[u].x * dz_stride + (int64_t)th[u].y * D + col, gz);
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
norm_dw_kernel(const float* part, int n_part, int D, float* __restrict__ dw) {
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
// blockDim = (threads a row, rows a CTA); a thread holds NV runs of 8 elements of its row. All
// tensors of rows lie alike, so a run that is aligned in one is aligned in all. Where D is not a
// multiple of 8 (ODD) a row begins `lead` elements behind a run's boundary: its first and last run
// are partly the neighbours'. They are read whole, but for one that passes the tensor's end, and
// written element by element. A thread's rows are a multiple of 8 apart, so that `lead`, and with it
// the thread's columns of w and dw, stays the same.

constexpr int kRun = 8;

template <bool ODD> struct Columns {
  int lead, D;
  int64_t rows;
  __device__ __forceinline__ Columns(int64_t row, int64_t rows_, int D_)
      : lead(ODD ? (int)((row * D_) & (kRun - 1)) : 0), D(D_), rows(rows_) {}
  __device__ __forceinline__ int at(int k) const { return (k * (int)blockDim.x + (int)threadIdx.x) * kRun - lead; }
  template <typename T> __device__ __forceinline__ void load(Raw<T, kRun>& r, const T* base, int64_t row, int c) const {
    const int64_t at = row * D + c;        // a multiple of a run, so never below 0
    const T* p = base + at;
    const bool here = c < D && (!ODD || c > -kRun);
    if (here && (!ODD || at + kRun <= rows * D)) r.load(p);
    else if (ODD && here) r.load_part(p, -c, D - c);
    else r.zero();
  }
  // takes the neighbours' elements out of a loaded run: at its use, so that no load is waited for
  // before
  template <typename T> __device__ __forceinline__ void clip(Raw<T, kRun>& r, int c) const {
    if (ODD && c < D && (c < 0 || c + kRun > D)) r.keep(-c, D - c);
  }
  // of a vector that begins at column 0, whatever the row's lead
  template <typename T> __device__ __forceinline__ void load_w(Raw<T, kRun>& r, const T* w, int c) const {
    if (!ODD) load(r, w, 0, c);
    else if (c < D && c > -kRun) r.load_part(w + c, -c, D - c);
    else r.zero();
  }
  template <typename T> __device__ __forceinline__ void store(T* base, int64_t row, int c, const float (&v)[kRun]) const {
    T* p = base + row * D + c;
    if (c + kRun <= D && (!ODD || c >= 0)) {
      VecIO<T, kRun>::store(p, v);
    } else if (ODD && c < D && c > -kRun) {
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (c + i >= 0 && c + i < D) p[i] = from_f<T>(v[i]);
    }
  }
};

// Sums of v and u over the threads of a row; every thread of the CTA calls it. The first exchange
// of a warp leaves v's half sums in its lower lanes and u's in its upper ones, so one tree of
// shuffles serves both. sm holds two buffers that successive calls use in turn (`turn`), so one
// barrier a call is enough: a buffer is written again only behind the next call's barrier.
__device__ __forceinline__ float2 row_sum(float v, float u, float (*sm)[64], int turn) {
  if (blockDim.x < 32) {                 // a few rows a warp
    for (int m = blockDim.x >> 1; m >= 1; m >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, m);
      u += __shfl_xor_sync(0xffffffffu, u, m);
    }
    return make_float2(v, u);
  }
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

template <typename T, typename R, int NV, int MAXT, bool ODD>
__global__ void __launch_bounds__(MAXT)
add_norm_kernel(const T* x, const R* res, const T* w, float scale, float w_add, float eps,
                R* h, T* __restrict__ n, int64_t rows, int D) {
  __shared__ float sm[2][64];
  allow_next_grid();
  wait_for_previous_grid();
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const Columns<ODD> cols(row, rows, D);
  Raw<T, kRun> wv[NV];
  if (ODD) {
#pragma unroll
    for (int k = 0; k < NV; ++k) cols.load_w(wv[k], w, cols.at(k));
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  Raw<T, kRun> xr[NV];
  Raw<R, kRun> rr[NV];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      xr[k].zero(); rr[k].zero();
      if (r < rows) { cols.load(xr[k], x, r, cols.at(k)); cols.load(rr[k], res, r, cols.at(k)); }
    }
  };
  fetch(row);
  if (!ODD) {
#pragma unroll
    for (int k = 0; k < NV; ++k) cols.load_w(wv[k], w, cols.at(k));
  }
  int turn = 0;
  do {
    const bool live = row < rows;
    float v[NV][kRun], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      cols.clip(xr[k], cols.at(k)); cols.clip(rr[k], cols.at(k));
      float xv[kRun];
      xr[k].get(xv); rr[k].get(v[k]);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        v[k][i] = fmaf(scale, xv[i], v[k][i]);
        ss = fmaf(v[k][i], v[k][i], ss);
      }
    }
    if (ODD) fetch(row + step);
    const float rstd = rsqrtf(row_sum(ss, 0.f, sm, turn++).x * (1.0f / D) + eps);
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        cols.store(h, row, cols.at(k), v[k]);
        float wf[kRun];
        wv[k].get(wf);
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[k][i] *= rstd * (wf[i] + w_add);
        cols.store(n, row, cols.at(k), v[k]);
      }
    }
    row += step;
  } while (ODD && row - threadIdx.y < rows);      // aligned rows have a CTA each
}

// A CTA takes every gridDim.x-th group of rows; a thread keeps its columns' weight gradient in
// registers over them and has the next row's loads in flight while it works on one.
template <typename T, typename R, int NV, int MAXT, int MINB, bool ODD>
__global__ void __launch_bounds__(MAXT, MINB)
add_norm_bwd_kernel(const R* h, const T* w, const T* dn, const R* dh,
                    float scale, float w_add, float eps, R* dres, T* __restrict__ dx,
                    float* __restrict__ part, int64_t rows, int D) {
  // the next row's dh is asked for with its h and dn where the registers allow (bf16), else once
  // this row's has been used
  constexpr bool kEarly = sizeof(R) == 2;
  __shared__ float sm[2][64];
  extern __shared__ float sum_w[];          // [D] where several rows share a CTA
  wait_for_previous_grid();
  const float inv_d = 1.0f / D;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const Columns<ODD> cols(row, rows, D);
  float dw[NV][kRun];
  Raw<T, kRun> wv[NV], dr[NV];
  Raw<R, kRun> hr[NV], gr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    cols.load_w(wv[k], w, cols.at(k));
#pragma unroll
    for (int i = 0; i < kRun; ++i) dw[k][i] = 0.f;
  }
  auto fetch_row = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      hr[k].ones(); dr[k].zero();
      if (r < rows) { cols.load(hr[k], h, r, cols.at(k)); cols.load(dr[k], dn, r, cols.at(k)); }
    }
  };
  auto fetch_dh = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      gr[k].zero();
      if (dh && r < rows) cols.load(gr[k], dh, r, cols.at(k));
    }
  };
  fetch_row(row);
  fetch_dh(row);
  int turn = 0;
  for (int64_t r0 = row - threadIdx.y; r0 < rows; r0 += step, row += step, ++turn) {
    float hv[NV][kRun], da[NV][kRun], ss = 0.f, ax = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      cols.clip(hr[k], cols.at(k)); cols.clip(dr[k], cols.at(k));
      hr[k].get(hv[k]); dr[k].get(da[k]);
    }
    Raw<R, kRun> now[NV];                   // this row's dh
#pragma unroll
    for (int k = 0; k < NV; ++k) now[k] = gr[k];
    fetch_row(row + step);
    if (kEarly) fetch_dh(row + step);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float wf[kRun];
      wv[k].get(wf);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        ss = fmaf(hv[k][i], hv[k][i], ss);
        ax = fmaf(da[k][i] * (wf[i] + w_add), hv[k][i], ax);
      }
    }
    const float2 s = row_sum(ss, ax, sm, turn);
    const float r1 = rsqrtf(fmaf(s.x, inv_d, eps)), cc = -s.y * r1 * r1 * inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float wf[kRun], gv[kRun];
      wv[k].get(wf);
      now[k].get(gv);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        dw[k][i] = fmaf(da[k][i], hv[k][i] * r1, dw[k][i]);
        gv[i] = fmaf(r1, fmaf(da[k][i], wf[i] + w_add, cc * hv[k][i]), gv[i]);
      }
      if (row < rows) {
        cols.store(dres, row, cols.at(k), gv);
        if (dx) {
#pragma unroll
          for (int i = 0; i < kRun; ++i) gv[i] *= scale;
          cols.store(dx, row, cols.at(k), gv);
        }
      }
    }
    if (!kEarly) fetch_dh(row + step);
  }
  if (part == nullptr) return;
  allow_next_grid();
  float* mine = part + (int64_t)blockIdx.x * D;
  if (blockDim.y == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int c = cols.at(k) + i;
        if (c >= 0 && c < D) mine[c] = dw[k][i];
      }
    return;
  }
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  for (int c = tid; c < D; c += threads) sum_w[c] = 0.f;
  for (int y = 0; y < blockDim.y; ++y) {    // the rows of the CTA in turn
    __syncthreads();
    if (threadIdx.y != y) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int c = cols.at(k) + i;
        if (c >= 0 && c < D) sum_w[c] += dw[k][i];
      }
  }
  __syncthreads();
  for (int c = tid; c < D; c += threads) mine[c] = sum_w[c];
}

// Rows too long for registers: a CTA reads its row twice, the second time from the caches, and
// keeps the weight gradient in shared memory.
template <typename T, typename R, bool ODD>
__global__ void __launch_bounds__(1024, 1)
add_norm_bwd_long_kernel(const R* h, const T* w, const T* dn, const R* dh,
                         float scale, float w_add, float eps, R* dres, T* __restrict__ dx,
                         float* __restrict__ part, int64_t rows, int D) {
  __shared__ float sm[2][64];
  extern __shared__ float sum_w[];          // [runs * 8], from the first run's first column
  wait_for_previous_grid();
  const float inv_d = 1.0f / D;
  const Columns<ODD> cols(blockIdx.x, rows, D);
  const int runs = (D + cols.lead + kRun - 1) / kRun, nv = (runs + blockDim.x - 1) / blockDim.x;
  for (int c = threadIdx.x; c < runs * kRun; c += blockDim.x) sum_w[c] = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, ++turn) {
    float ss = 0.f, ax = 0.f;
    for (int k = 0; k < nv; ++k) {
      Raw<R, kRun> hr;
      Raw<T, kRun> dr, wr;
      cols.load(hr, h, row, cols.at(k)); cols.load(dr, dn, row, cols.at(k)); cols.load_w(wr, w, cols.at(k));
      cols.clip(hr, cols.at(k)); cols.clip(dr, cols.at(k));
      float hv[kRun], da[kRun], wf[kRun];
      hr.get(hv); dr.get(da); wr.get(wf);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        ss = fmaf(hv[i], hv[i], ss);
        ax = fmaf(da[i] * (wf[i] + w_add), hv[i], ax);
      }
    }
    const float2 s = row_sum(ss, ax, sm, turn);
    const float r1 = rsqrtf(fmaf(s.x, inv_d, eps)), cc = -s.y * r1 * r1 * inv_d;
    for (int k = 0; k < nv; ++k) {
      const int c = cols.at(k);
      if (c >= D) break;
      Raw<R, kRun> hr, gr;
      Raw<T, kRun> dr, wr;
      cols.load(hr, h, row, c); cols.load(dr, dn, row, c); cols.load_w(wr, w, c);
      gr.zero();
      if (dh) cols.load(gr, dh, row, c);
      cols.clip(hr, c); cols.clip(dr, c);
      float hv[kRun], da[kRun], wf[kRun], gv[kRun];
      hr.get(hv); dr.get(da); wr.get(wf); gr.get(gv);
      float* mw = sum_w + c + cols.lead;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        mw[i] = fmaf(da[i], hv[i] * r1, mw[i]);
        gv[i] = fmaf(r1, fmaf(da[i], wf[i] + w_add, cc * hv[i]), gv[i]);
      }
      cols.store(dres, row, c, gv);
      if (dx) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) gv[i] *= scale;
        cols.store(dx, row, c, gv);
      }
    }
  }
  if (part == nullptr) return;
  allow_next_grid();
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += blockDim.x) part[(int64_t)blockIdx.x * D + c] = sum_w[c + cols.lead];
}

struct AddShape { int tx, ty; };

int runs_of(int D) { return D % kRun == 0 ? D / kRun : (D + 2 * kRun - 2) / kRun; }    // with any lead

// Threads a row when each holds nv runs: whole warps, or a power of two below; rows of up to 128
// threads share a CTA of 256 (a power of two of them, see grid_of).
AddShape add_shape(int D, int nv) {
  AddShape s;
  const int threads = (runs_of(D) + nv - 1) / nv;
  s.tx = (threads + 31) / 32 * 32;
  if (threads <= 16)
    for (s.tx = 1; s.tx < threads;) s.tx *= 2;
  s.ty = s.tx > 128 ? 1 : s.tx > 64 ? 2 : s.tx > 32 ? 4 : 256 / s.tx;
  return s;
}

// At most `most` CTAs (a multiple of 8), for odd rows a multiple of 8 of them: a thread's rows are
// then a multiple of 8 apart. CTAs without a row add zeros.
unsigned grid_of(int64_t groups, int64_t most, bool odd) {
  const int64_t n = groups < most ? groups : most;
  return (unsigned)(odd ? (n + 7) / 8 * 8 : n);
}

template <typename T, typename R, int NV, int MAXT, bool ODD>
cudaError_t add_fwd(const AddNorm& a, cudaStream_t st) {
  const AddShape s = add_shape(a.D, NV);
  // aligned rows: a CTA for each group of rows; odd ones: resident CTAs, which load w's parts once
  const unsigned grid = grid_of((a.rows + s.ty - 1) / s.ty, ODD ? 148 * (1024 / MAXT) : 1LL << 31, ODD);
  return launch_overlapped(add_norm_kernel<T, R, NV, MAXT, ODD>, dim3(grid), dim3(s.tx, s.ty), 0, st, (const T*)a.x,
                           (const R*)a.res, (const T*)a.w, a.scale, a.w_add, a.eps, (R*)a.h, (T*)a.n, a.rows, a.D);
}

cudaError_t sum_parts(const AddNorm& a, cudaError_t e, int parts, cudaStream_t st) {
  return e != cudaSuccess || !a.dw ? e : launch_overlapped(norm_dw_kernel, dim3((a.D + 31) / 32), dim3(32, 32), 0, st,
                                                           a.part, parts, a.D, a.dw);
}

// MINB CTAs of the backward pass are resident on each of 148 SMs; no more are launched, so that
// every CTA begins at once and takes the same number of rows.
template <typename T, typename R, int NV, int MAXT, int MINB, bool ODD>
cudaError_t add_bwd(const AddNorm& a, cudaStream_t st) {
  static_assert(MINB * 148 <= kNormParts, "parts in the workspace");
  const AddShape s = add_shape(a.D, NV);
  const unsigned parts = grid_of((a.rows + s.ty - 1) / s.ty, ODD ? MINB * 148 / 8 * 8 : MINB * 148, ODD);
  const cudaError_t e = launch_overlapped(
      add_norm_bwd_kernel<T, R, NV, MAXT, MINB, ODD>, dim3(parts), dim3(s.tx, s.ty), s.ty > 1 ? a.D * sizeof(float) : 0,
      st, (const R*)a.h, (const T*)a.w, (const T*)a.n, (const R*)a.res, a.scale, a.w_add, a.eps, (R*)a.dres, (T*)a.dx,
      a.dw ? a.part : nullptr, a.rows, a.D);
  return sum_parts(a, e, parts, st);
}

template <typename T, typename R, bool ODD>
cudaError_t add_bwd_long(const AddNorm& a, cudaStream_t st) {
  static std::atomic<uint64_t> prepared{0};
  const cudaError_t p = raise_smem_limit(add_norm_bwd_long_kernel<T, R, ODD>, 96 * 1024, prepared);
  if (p != cudaSuccess) return p;
  const unsigned parts = grid_of(a.rows, ODD ? 144 : 148, ODD);
  const cudaError_t e = launch_overlapped(
      add_norm_bwd_long_kernel<T, R, ODD>, dim3(parts), dim3(1024), runs_of(a.D) * kRun * sizeof(float), st,
      (const R*)a.h, (const T*)a.w, (const T*)a.n, (const R*)a.res, a.scale, a.w_add, a.eps, (R*)a.dres, (T*)a.dx,
      a.dw ? a.part : nullptr, a.rows, a.D);
  return sum_parts(a, e, parts, st);
}

// Runs of a thread and CTAs of an SM: as few threads a row as the registers allow (their barrier and
// shuffles are paid by all of them), as many CTAs as fit. (Backward, 16,384 x 4,096, fp32 residual:
// two runs by 256 threads 172 us, one run by 512 226; 8,000 x 8,192, bf16: forward by 512 threads 79
// us, by 1,024 95; 4,000 x 16,384: backward reading the row twice 198 us, by registers that spill
// 484. Odd rows: 5,000 x 7,001, bf16: forward 66 us and backward 77, element by element 204 and
// 588; 20,000 x 1,001 31 and 50, element by element 45 and 80. Odd rows of more than 8,190 columns
// spill in the forward pass, whose three runs a thread and prefetch do not fit 64 registers: 3,000 x
// 12,001, bf16, 104 us and backward 139 for 44 and 55 of bytes; fp32 381 and 210 for 88 and 110.)
template <typename T, typename R, bool ODD>
cudaError_t add_odd(const AddNorm& a, cudaStream_t st) {
  const int runs = runs_of(a.D);
  if (a.back) {
    if (runs <= 256) return add_bwd<T, R, 1, 256, 4, ODD>(a, st);
    if (runs <= 512) return add_bwd<T, R, 2, 256, 2, ODD>(a, st);
    if (runs <= 1024) return add_bwd<T, R, 2, 512, 1, ODD>(a, st);
    return add_bwd_long<T, R, ODD>(a, st);
  }
  if (runs <= 256) return add_fwd<T, R, 1, 256, ODD>(a, st);
  if (runs <= 512) return add_fwd<T, R, 1, 512, ODD>(a, st);
  if (runs <= 1024) return add_fwd<T, R, 2, 512, ODD>(a, st);
  return add_fwd<T, R, ODD ? 3 : 2, 1024, ODD>(a, st);      // an odd row may take 2,049 runs
}

template <typename T, typename R>
cudaError_t add_tr(const AddNorm& a, cudaStream_t st) {
  return a.D % kRun == 0 ? add_odd<T, R, false>(a, st) : add_odd<T, R, true>(a, st);
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
