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
// One cluster of C CTAs owns KH neighbouring key heads of a sequence: the conv channels of their q
// and k and of their G value heads, whose G D state rows (one run of a page) are split evenly over
// the cluster. C is 1 where the batch fills the GPU and grows as it shrinks; KH is 1 for heads of
// 128 and grows for narrower ones, whose rows alone would not pay for a CTA's start.
//
// Bound by HBM: the state is read once and written once per stored token. What costs the
// bandwidth is time in which an SM has no loads in flight (a page number is looked up, a conv
// computed, before a row is used), so every lane runs a ring of asynchronous copies of the row
// parts that it will itself consume, started before the conv: it needs no barrier, only the
// lane's own wait. CTAs of 128 threads, four an SM: the start of one overlaps the rows of the
// others (bf16 states: 114 us by two CTAs of 256 threads, 77 by four of 128).
//
// Measured, 16 / 48 heads of 128 (16 / 32 for 192 sequences), share of 2 x state bytes and the
// rest at the copy rate: 256 sequences, fp32 states 261 us (97 %); 192, bf16 states 79 us (82 %,
// the last of its 5.2 waves of CTAs is nearly empty); one sequence 6.7 us, with the output norm 8.4.
// From four tokens on the row loop's fp32 instructions bind instead: per token and element two
// multiply-adds for the sums and one or two for the update (64 sequences of 4 tokens, fp32 states
// 79 us, 81 %; of 8 tokens 106 us, 61 %; 128 of 4 with bf16 states 109 us, 61 %). Taking the sums
// of all tokens from matrix instructions on the state as it was, with a triangular recursion
// behind them, was right but slower (135 us for the last): its chain of shuffles and shared-memory
// reads leaves three warps a scheduler idle for most of the time.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocks = 4;         // resident CTAs per SM
constexpr int kWarps = kThreads / 32;
constexpr float kEps = 1e-6f;
constexpr int kMaxTok = 8;
constexpr int kMaxSmem = 224 * 1024;
constexpr int kSeg = 16;           // state columns per lane
constexpr int kRows = 4;           // state rows per lane and pass
constexpr int kAhead = 4;          // tokens whose channels are loaded together
constexpr int kPass = 32 * kSeg * kRows;   // state elements of a warp's pass

// Stages of the ring: 8 KB a warp.
template <typename S> constexpr int kStages = sizeof(S) == 4 ? 1 : 2;

// z * sigmoid(z) for the activations' type: fp32 with the accurate exponential and division,
// whose errors would otherwise show in fp32 results; bf16 with the fast ones.
template <typename T> __device__ __forceinline__ float silu_for(float z);
template <> __device__ __forceinline__ float silu_for<bf16>(float z) { return silu(z); }
template <> __device__ __forceinline__ float silu_for<float>(float z) { return z / (1.0f + expf(-z)); }

// a * b + c. With fp32 activations every product and sum on the state's way is rounded on its own, in one
// fixed order of sums (plain_dots), as in a form of elementary operations; fused operations made about
// 1 in 10^4 of the states stored in bf16 round to the other neighbour than such a form's. Nothing more is
// promised than the bound of fp32 sums: in which order such a form adds is its own affair.
// The price is in the row loop, whose instructions bind from four tokens on: 64 sequences of 1 / 4 / 8
// tokens, fp32 states, 74 / 103 / 159 us, with bf16 activations and fused operations 70 / 79 / 106; 256 of
// one token 271 and 258.
template <typename T> __device__ __forceinline__ float mul_add(float a, float b, float c);
template <> __device__ __forceinline__ float mul_add<bf16>(float a, float b, float c) { return fmaf(a, b, c); }
template <> __device__ __forceinline__ float mul_add<float>(float a, float b, float c) { return __fadd_rn(__fmul_rn(a, b), c); }

// Pairs of fp32 values: one instruction for two products or sums.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(f2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a + b c with the product rounded before it is added, which the paired instructions, put together
// by the assembler, would not be
__device__ __forceinline__ f2 add_product(f2 a, f2 b, f2 c) {
  const float2 x = unpair(a), y = unpair(b), z = unpair(c);
  return pair(__fadd_rn(x.x, __fmul_rn(y.x, z.x)), __fadd_rn(x.y, __fmul_rn(y.y, z.y)));
}

// Eight channels as they lie in memory.
template <typename T> struct Raw8 {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  // element i (a constant once unrolled)
  __device__ __forceinline__ float get(int i) const {
    const uint4 q = u[i * sizeof(T) / 16];
    const int b = i % (16 / (int)sizeof(T));
    if constexpr (sizeof(T) == 4) return __uint_as_float(b == 0 ? q.x : b == 1 ? q.y : b == 2 ? q.z : q.w);
    const uint32_t w = b < 2 ? q.x : b < 4 ? q.y : b < 6 ? q.z : q.w;
    return __uint_as_float(b & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

// N consecutive elements of a state row (a word of 8 or 16 bytes) as pairs, and back (rounded to
// nearest even once for bf16).
template <typename S, int N> struct Chunk;
template <> struct Chunk<float, 4> {
  typedef uint4 Word;
  static __device__ __forceinline__ void get(uint4 u, f2* p) {
    p[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
    p[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 put(const f2* p) {
    const float2 a = unpair(p[0]), b = unpair(p[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
__device__ __forceinline__ f2 widen(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t narrow(f2 p) {
  const float2 f = unpair(p);
  __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <> struct Chunk<bf16, 8> {
  typedef uint4 Word;
  static __device__ __forceinline__ void get(uint4 u, f2* p) {
    p[0] = widen(u.x); p[1] = widen(u.y); p[2] = widen(u.z); p[3] = widen(u.w);
  }
  static __device__ __forceinline__ uint4 put(const f2* p) {
    return make_uint4(narrow(p[0]), narrow(p[1]), narrow(p[2]), narrow(p[3]));
  }
};
template <> struct Chunk<bf16, 4> {
  typedef uint2 Word;
  static __device__ __forceinline__ void get(uint2 u, f2* p) { p[0] = widen(u.x); p[1] = widen(u.y); }
  static __device__ __forceinline__ uint2 put(const f2* p) { return make_uint2(narrow(p[0]), narrow(p[1])); }
};

// What the row loop needs of a token and value head. The state is carried as gamma times the
// registers: a token that is neither stored nor near the ends of fp32 only multiplies gamma by its
// alpha and adds (u / gamma) k, one instruction for two elements instead of two.
struct __align__(16) Step {
  float gamma;                     // alpha times the factor the registers carried before the token
  float beta;
  float inv;                       // 1 / gamma where the registers keep the factor, else 0: they
                                   // become the state itself
  float pad;
};

// Shared memory: the ring, then in floats steps, q | k, v (then o), k.q, sums of o^2, 1 / rms.
int64_t smem_bytes(int n_tok, int64_t KH, int64_t G, int d, int64_t rows) {
  return kWarps * kStages<float> * kPass * (int64_t)sizeof(float) +
         (int64_t)sizeof(float) * n_tok * (KH * 2 * d + rows + KH + 6 * G);
}

// N sums (over the L lanes of a row) of each lane: every exchange leaves half of the sums with each
// lane, 4 shuffles for 4 sums of 8 lanes instead of 12. The sums end in v[0 .. N / L - 1] (v[0] for
// N < L), lane seg holding those from seg * N / L on.
template <int L, int N> __device__ __forceinline__ void scatter_sums(float* v, int seg) {
  if constexpr (L > 1 && N > 1) {
    const bool up = seg & (L / 2);
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      v[i] = (up ? v[i + N / 2] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + N / 2], L / 2);
    scatter_sums<L / 2, N / 2>(v, seg);
  } else if constexpr (L > 1) {             // one sum left, shared by L lanes
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
  }
}

// Whether the registers may carry a factor: not with fp32 activations (see mul_add), and only where
// the rows of a pass share one head's factor.
template <typename T, int D> constexpr bool kCarry = sizeof(T) == 2 && kPass / D <= D;

template <typename T, typename S, int D>
__global__ void __launch_bounds__(kThreads, kBlocks)
decode_paged_kernel(const PagedDecode a, int C, int KH) {
  constexpr int L = D / kSeg;              // lanes per state row
  constexpr int RPW = 32 / L;              // rows a warp covers at once
  constexpr int RPP = RPW * kRows;         // rows of a warp's pass
  constexpr bool kPlain = sizeof(T) == 4;  // fp32 activations: the definition's own operations (see mul_add)
  constexpr int CE = kPlain ? 4 : 16 / sizeof(S);      // elements of a lane's chunk
  constexpr int CH = kSeg / CE;            // chunks of a lane's row part
  typedef Chunk<S, CE> Part;
  typedef typename Part::Word Word;
  constexpr int NST = kStages<S>;
  const int G1 = a.Hv / a.Hk, G = KH * G1, W = KH * D, n_tok = a.n_tok;
  const int32_t Cc = 2 * a.Hk * D + a.Hv * D;
  const int rank = blockIdx.x % C;
  const int per_seq = a.Hk / KH;
  const int64_t b = blockIdx.x / C / per_seq;
  const int hk = blockIdx.x / C % per_seq * KH;        // the first key head
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = G * D / C, row0 = rank * rows;      // this CTA's rows of the G D

  allow_next_grid();
  wait_for_previous_grid();
  // what does not depend on the page is asked for beside the page's number: the first channels'
  // taps' weights and tokens
  const int32_t rp = a.read_pages[b];
  const int nv = a.n_valid ? min(max(a.n_valid[b], 0), n_tok) : n_tok;
  const T* x = static_cast<const T*>(a.x) + b * n_tok * a.x_stride;
  const int n_local = 2 * W + rows;
  int lc = threadIdx.x * 8;
  auto channel = [&](int c) {              // of this CTA's local channel c, in the layer
    return c < W ? hk * D + c : c < 2 * W ? a.Hk * D + hk * D + (c - W) : 2 * a.Hk * D + hk * G1 * D + row0 + (c - 2 * W);
  };
  Raw8<T> wr[4], xr[kAhead];
  auto fetch_x = [&](int t0) {
#pragma unroll
    for (int t = 0; t < kAhead; ++t)
      if (t0 + t < n_tok) xr[t].load(x + (t0 + t) * a.x_stride + channel(lc));
  };
  auto fetch_w = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) wr[j].load(static_cast<const T*>(a.conv_w) + (int64_t)channel(lc) * 4 + j * 8);
  };
  if (lc < n_local) { fetch_w(); fetch_x(0); }
  if (nv == 0) return;                     // nothing of this sequence is computed, written or stored
  const bool fresh = rp < 0 || rp >= a.n_pages;

  extern __shared__ __align__(16) char smem_raw[];
  Word* ring = reinterpret_cast<Word*>(smem_raw) + warp * (NST * kRows * CH * 32) + lane;     // [stage][row][chunk][lane]
  Step* steps = reinterpret_cast<Step*>(smem_raw + kWarps * NST * kPass * sizeof(S));         // [n_tok][G]
  float* qk = reinterpret_cast<float*>(steps + n_tok * G);      // [n_tok][KH][2 D] q | k
  float* vo = qk + n_tok * 2 * W;          // [n_tok][rows] v, then o in its place
  float* kqs = vo + n_tok * rows;          // [n_tok][KH] k_t.q_t
  float* sqs = kqs + n_tok * KH;           // [n_tok][G] sums of o^2 over this CTA's rows
  float* rms = sqs + n_tok * G;            // [n_tok][G] 1 / rms of a head's o
  __shared__ int32_t wp[kMaxTok];          // page of the state after token t, -1: not stored

  // 0. the first row parts are on their way before anything else is done
  const int seg = lane % L;
  const int64_t at0 = ((int64_t)hk * G1 * D + row0) * D + seg * CE;        // this lane's place in a page
  const S* src = static_cast<const S*>(a.state_pool) + (fresh ? 0 : (int64_t)rp * a.state_stride) + at0;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  // a pass lies in one key head: its key head, first row and the row behind that key head's last
  const int krows = rows / KH, kpasses = (krows + RPP - 1) / RPP, passes = KH * kpasses;
  struct Pass { int head, row, end; };
  auto pass_of = [&](int pass) {
    const int j = KH > 1 ? pass / kpasses : 0;
    return Pass{j, j * krows + (pass - j * kpasses) * RPP, j * krows + krows};
  };
  auto fetch = [&](int pass, int stage) {
    if (!fresh && pass < passes) {
      const Pass w = pass_of(pass);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = w.row + i * RPW + lane / L;
        if (r < w.end) {
#pragma unroll
          for (int j = 0; j < CH; ++j)
            copy_async<sizeof(Word)>(ring_at + ((stage * kRows + i) * CH + j) * (32 * sizeof(Word)),
                                     src + (int64_t)r * D + j * CE * L);
        }
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int st = 0; st < NST; ++st) fetch(warp + st * kWarps, st);

  // 1. conv + SiLU over this CTA's channels, eight a thread; the window slides in registers. q and
  //    k are laid out as the lanes of a row read them: quad i of a lane at 4 L i + 4 seg.
  const auto place = [](int c) {           // of column c in a vector of q or k
    return (c / (CE * L) * CE + c % CE) / 4 * (4 * L) + c % (CE * L) / CE * 4 + c % 4;
  };
  T* conv = static_cast<T*>(a.conv_pool);
  Raw8<T> w0, w1, w2;
  auto fetch_taps = [&]() {
    w0.zero(); w1.zero(); w2.zero();
    if (!fresh && lc < n_local) {
      const T* cs = conv + (int64_t)rp * a.conv_stride + channel(lc);
      w0.load(cs); w1.load(cs + Cc); w2.load(cs + 2 * Cc);
    }
  };
  fetch_taps();
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
  for (int i = threadIdx.x; i < G * nv; i += kThreads) {
    const int64_t gi = (b * n_tok + i / G) * a.Hv + hk * G1 + i % G;
    steps[i].gamma = expf(a.g[gi]);
    steps[i].beta = a.beta[gi];
  }
  // the taps of q and k are read by the whole cluster before rank 0 writes them (all channels are
  // in the loop's first round then); wp is visible behind the barrier
  if (C > 1) cg::this_cluster().sync();
  else __syncthreads();
  while (lc < n_local) {
    const int gc = channel(lc);
    const bool keeps = rank == 0 || lc >= 2 * W;
    const auto quad_at = [&](int c) {      // where four channels of q or k, or v, begin in shared memory
      if (c >= 2 * W) return (int)(vo - qk) + c - 2 * W;
      const int h = c < W ? 0 : D, cw = c < W ? c : c - W;
      return cw / D * (2 * D) + h + place(cw % D);
    };
    const int at_a = quad_at(lc), at_b = quad_at(lc + 4), at_step = lc < 2 * W ? 2 * W : rows;
    for (int t0 = 0; t0 < nv; t0 += kAhead) {
      if (t0) fetch_x(t0);
#pragma unroll
      for (int t = 0; t < kAhead; ++t) {
        if (t0 + t >= nv) break;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float z = wr[i / 2].get(i % 2 * 4) * w0.get(i);
          z = mul_add<T>(wr[i / 2].get(i % 2 * 4 + 1), w1.get(i), z);
          z = mul_add<T>(wr[i / 2].get(i % 2 * 4 + 2), w2.get(i), z);
          z = mul_add<T>(wr[i / 2].get(i % 2 * 4 + 3), xr[t].get(i), z);
          y[i] = silu_for<T>(z);
        }
        float* dst = qk + (t0 + t) * at_step;
        *reinterpret_cast<float4*>(dst + at_a) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(dst + at_b) = make_float4(y[4], y[5], y[6], y[7]);
        if (keeps && wp[t0 + t] >= 0) {
          T* cs = conv + (int64_t)wp[t0 + t] * a.conv_stride + gc;
          w1.store(cs); w2.store(cs + Cc); xr[t].store(cs + 2 * Cc);
        }
        w0 = w1; w1 = w2; w2 = xr[t];
      }
    }
    lc += kThreads * 8;
    if (lc < n_local) { fetch_w(); fetch_x(0); fetch_taps(); }
  }
  __syncthreads();

  // 2. q_t and k_t L2-normalised in place (a warp per token and key head), k_t.q_t beside them
  constexpr int VEC = D >= 32 ? D / 32 : 1;
  for (int e = warp; e < nv * KH; e += kWarps) {        // qk and kqs lie by token, then key head
    float* yt = qk + e * 2 * D;
    const bool active = lane * VEC < D;
    float qv[VEC], kv[VEC], qq = 0.f, kk = 0.f, kq = 0.f;
    int at[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      at[j] = place((D == 128 ? lane * VEC + j : lane + 32 * j) % D);
      qv[j] = active ? yt[at[j]] : 0.f;
      kv[j] = active ? yt[D + at[j]] : 0.f;
      qq = mul_add<T>(qv[j], qv[j], qq); kk = mul_add<T>(kv[j], kv[j], kk); kq = fmaf(kv[j], qv[j], kq);
    }
    qq = warp_sum(qq); kk = warp_sum(kk); kq = warp_sum(kq);
    const float nq = sqrtf(qq + kEps), nk = sqrtf(kk + kEps);
    if (active) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) { yt[at[j]] = qv[j] / nq; yt[D + at[j]] = kv[j] / nk; }
    }
    if (lane == 0) kqs[e] = kq / (nq * nk);
  }
  // the factor that the registers carry through the tokens of a head: it stays within 2^-40 and
  // 2^40 (else, and where the token's state is stored, the registers become the state itself)
  for (int hh = threadIdx.x; hh < G; hh += kThreads) {
    constexpr float kLow = 0x1p-40f, kHigh = 0x1p40f;
    float carried = 1.f;
    for (int t = 0; t < nv; ++t) {
      Step& st = steps[t * G + hh];
      const float gamma = carried * st.gamma;
      const float next = t + 1 < nv ? gamma * steps[(t + 1) * G + hh].gamma : 0.f;
      const bool keep = kCarry<T, D> && wp[t] < 0 && gamma >= kLow && gamma <= kHigh && next >= kLow && next <= kHigh;
      st.gamma = gamma;
      st.inv = keep ? 1.0f / gamma : 0.f;
      carried = keep ? gamma : 1.f;
    }
  }
  __syncthreads();

  // 3. the state rows, each through every token
  S* pool = static_cast<S*>(a.state_pool) + at0;
  int stage = 0;
  for (int pass = warp; pass < passes; pass += kWarps) {
    const Pass w = pass_of(pass);
    const int ra = w.row + lane / L, end = w.end;    // this lane's first row; the others follow by RPW
    f2 s[kRows][kSeg / 2];
    copy_wait<NST - 1>();
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        Word u = {};
        if (!fresh && ra + i * RPW < end) u = ring[((stage * kRows + i) * CH + j) * 32];
        Part::get(u, &s[i][j * CE / 2]);
      }
    fetch(pass + NST * kWarps, stage);
    stage = stage + 1 == NST ? 0 : stage + 1;
    const float* qt = qk + w.head * 2 * D + seg * 4;
    const Step* st = steps;
    float* vt = vo;
    for (int t = 0; t < nv; ++t, qt += 2 * W, st += G, vt += rows) {
      // S k of the lane's rows: first its own columns, then the row's lanes together, which leaves
      // each lane the sums of NR rows from r0 on (two lanes of 8 the same row's). S q is added up
      // while S k's shuffles are under way: u waits for S k only.
      constexpr int NR = kRows > L ? kRows / L : 1, SAME = L > kRows ? L / kRows : 1;
      const int r0 = seg * kRows / L;
      float sk[kRows], sq[kRows];
      // fp32 activations: the state decays first, and its products with k are rounded and added up one
      // by one. The order depends on the width: at 128 columns fours of neighbours first, then halves of
      // the row; below, halves of the row only.
      auto plain_dots = [&](const float* vec, float (&sums)[kRows]) {
        float tot[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          float q[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(vec + j * 4 * L);
            const float2 lo = unpair(mul2(s[i][2 * j], v4.x)), hi = unpair(mul2(s[i][2 * j + 1], v4.y));
            q[j][0] = lo.x; q[j][1] = lo.y; q[j][2] = hi.x; q[j][3] = hi.y;
          }
          if constexpr (D == 128) {
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              f[j] = __fadd_rn(__fadd_rn(__fadd_rn(q[j][0], q[j][1]), q[j][2]), q[j][3]);
            tot[i] = __fadd_rn(__fadd_rn(f[0], f[2]), __fadd_rn(f[1], f[3]));
#pragma unroll
            for (int m = L / 2; m >= 1; m >>= 1) tot[i] += __shfl_xor_sync(0xffffffffu, tot[i], m);
          } else {
            float f[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f[x] = __fadd_rn(__fadd_rn(q[0][x], q[2][x]), __fadd_rn(q[1][x], q[3][x]));
#pragma unroll
              for (int m = L / 2; m >= 1; m >>= 1) f[x] += __shfl_xor_sync(0xffffffffu, f[x], m);
            }
            tot[i] = __fadd_rn(__fadd_rn(f[0], f[2]), __fadd_rn(f[1], f[3]));
          }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {       // this lane's rows, as scatter_sums leaves them
          sums[i] = tot[0];
#pragma unroll
          for (int c = 1; c < kRows; ++c) sums[i] = r0 + i == c ? tot[c] : sums[i];
        }
      };
      auto dots = [&](const float* vec, float (&sums)[kRows]) {
        f2 acc[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) acc[i] = 0ull;
#pragma unroll
        for (int j = 0; j < kSeg / 4; ++j) {
          const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(vec + j * 4 * L);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            acc[i] = fma2(s[i][2 * j], v4.x, acc[i]);
            acc[i] = fma2(s[i][2 * j + 1], v4.y, acc[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float2 f = unpair(acc[i]);
          sums[i] = f.x + f.y;
        }
        scatter_sums<L, kRows>(sums, seg);
      };
      if constexpr (kPlain) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = ra + i * RPW;
          const float alpha = r < end ? st[(row0 + r) / D].gamma : 0.f;
          const f2 aa = pair(alpha, alpha);
#pragma unroll
          for (int j = 0; j < kSeg / 2; ++j) s[i][j] = mul2(aa, s[i][j]);
        }
        plain_dots(qt + D, sk);
      } else {
        dots(qt + D, sk);
      }
      dots(qt, sq);
      float u[NR], gam[kRows], inv[kRows];
      if constexpr (RPP <= D) {             // a pass lies in one head
        const float4 p = *reinterpret_cast<const float4*>(st + (row0 + w.row) / D);
#pragma unroll
        for (int i = 0; i < kRows; ++i) { gam[i] = p.x; inv[i] = p.z; }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = ra + (r0 + i) * RPW;
          u[i] = p.y * ((r < end ? vt[r] : 0.f) - (kPlain ? sk[i] : p.x * sk[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = ra + i * RPW;
          gam[i] = r < end ? st[(row0 + r) / D].gamma : 0.f;
          inv[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = ra + (r0 + i) * RPW, rr = r < end ? r : 0;
          u[i] = st[(row0 + rr) / D].beta * (vt[rr] - (kPlain ? sk[i] : st[(row0 + rr) / D].gamma * sk[i]));
        }
      }
      f2 uu[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float ui = L > 1 ? __shfl_sync(0xffffffffu, u[i % NR], (lane & ~(L - 1)) + i / NR * SAME) : u[i % NR];
        uu[i] = pair(ui, ui);
      }
      __syncwarp();                         // v has been read where o is written
      if (seg % SAME == 0) {
        const float kq = kqs[t * KH + w.head];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = ra + (r0 + i) * RPW;
          if (r < end) {
            const float gm = RPP <= D ? gam[0] : st[(row0 + r) / D].gamma;
            vt[r] = a.scale * fmaf(kPlain ? 1.f : gm, sq[i], u[i] * kq);
          }
        }
      }
      if (kCarry<T, D> && inv[0] != 0.f) {
        const f2 iv = pair(inv[0], inv[0]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) uu[i] = mul2(uu[i], iv);
#pragma unroll
        for (int j = 0; j < kSeg / 4; ++j) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(qt + D + j * 4 * L);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            s[i][2 * j] = fma2(uu[i], k4.x, s[i][2 * j]);
            s[i][2 * j + 1] = fma2(uu[i], k4.y, s[i][2 * j + 1]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kSeg / 4; ++j) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(qt + D + j * 4 * L);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const f2 aa = pair(gam[i], gam[i]);
            s[i][2 * j] = kPlain ? add_product(s[i][2 * j], uu[i], k4.x) : fma2(aa, s[i][2 * j], mul2(uu[i], k4.x));
            s[i][2 * j + 1] = kPlain ? add_product(s[i][2 * j + 1], uu[i], k4.y) : fma2(aa, s[i][2 * j + 1], mul2(uu[i], k4.y));
          }
        }
        const int32_t to = wp[t];
        if (to >= 0) {
          S* dst = pool + (int64_t)to * a.state_stride + (int64_t)ra * D;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (ra + i * RPW < end) {
#pragma unroll
              for (int j = 0; j < CH; ++j)
                __stcs(reinterpret_cast<Word*>(dst + i * RPW * D + j * CE * L), Part::put(&s[i][j * CE / 2]));
            }
        }
      }
    }
  }
  __syncthreads();

  // 4. outputs, normalised and gated when asked: sums of squares per token and head, over the
  //    cluster where its CTAs share a head
  if (a.z) {
    for (int e = warp; e < nv * G; e += kWarps) {
      const int t = e / G, hh = e % G;
      const int lo = max(hh * D, row0) - row0, hi = min(hh * D + D, row0 + rows) - row0;
      float ss = 0.f;
      for (int i = lo + lane; i < hi; i += 32) ss = fmaf(vo[t * rows + i], vo[t * rows + i], ss);
      ss = warp_sum(ss);
      if (lane == 0) sqs[e] = ss;
    }
    if (C > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      for (int e = threadIdx.x; e < nv * G; e += kThreads) {
        float ss = 0.f;
        for (int k = 0; k < C; ++k) ss += cl.map_shared_rank(sqs, k)[e];
        rms[e] = 1.0f / sqrtf(ss / D + a.eps);
      }
      cl.sync();                            // no CTA leaves while another reads its sums
    } else {
      __syncthreads();
      for (int e = threadIdx.x; e < nv * G; e += kThreads) rms[e] = 1.0f / sqrtf(sqs[e] / D + a.eps);
      __syncthreads();
    }
  }
  T* o = static_cast<T*>(a.o);
  for (int e = threadIdx.x * 4; e < nv * rows; e += kThreads * 4) {
    const int t = e / rows, i = e % rows, r = row0 + i;
    const int64_t tok = b * n_tok + t;
    float v[4];
    VecIO<float, 4>::load(vo + e, v);
    if (a.z) {
      float z[4], w[4];
      VecIO<T, 4>::load(static_cast<const T*>(a.z) + tok * a.z_stride + hk * G1 * D + r, z);
      VecIO<T, 4>::load(static_cast<const T*>(a.norm_w) + r % D, w);
      const float rstd = rms[t * G + r / D];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = v[k] * rstd * w[k] * silu_for<T>(z[k]);
    }
    VecIO<T, 4>::store(o + (tok * a.Hv + hk * G1) * D + r, v);
  }
}

template <typename T, typename S, int D>
cudaError_t launch_d(const PagedDecode& a, cudaStream_t st) {
  const int G = a.Hv / a.Hk, places = kBlocks * 148;
  // Key heads a CTA: for heads below 128, neighbours up to 768 rows in all, while the CTAs still
  // fill the GPU's places and four of them an SM's shared memory. (256 sequences of 16 / 48 heads,
  // heads of 64, fp32 states: 82.8 -> 78.5 us; heads of 32,
  // bf16 states: 34.3 -> 20.4 us.)
  int KH = 1;
  while (D < 128 && a.Hk % (KH * 2) == 0 && KH * 2 * G * D <= 768 && (int64_t)a.B * a.Hk / (KH * 2) >= places &&
         smem_bytes(a.n_tok, KH * 2, KH * 2 * G, D, KH * 2 * G * D) <= 56 * 1024)
    KH *= 2;
  // The cluster: CTAs until the GPU's places are taken, two where a second wave would be half
  // empty or less.
  const int64_t ctas = (int64_t)a.B * (a.Hk / KH);
  const auto splits = [&](int c) { return G * D % (c * (kPass / D)) == 0 && 2 * D + G * D / c <= kThreads * 8; };
  int C = 1;
  if (KH == 1) {
    while (C < 8 && ctas * C * 2 <= places && splits(C * 2)) C *= 2;
    if (ctas > places && ctas * 2 <= places * 3 && splits(2)) C = 2;
  }
  const size_t smem = (size_t)smem_bytes(a.n_tok, KH, KH * G, D, KH * G * D / C);
  static std::atomic<uint64_t> prepared{0};
  cudaError_t e = raise_smem_limit(decode_paged_kernel<T, S, D>, kMaxSmem, prepared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C; attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return launch_result(cudaLaunchKernelEx(&cfg, decode_paged_kernel<T, S, D>, a, C, KH));
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

size_t decode_paged_smem(int n_tok, int64_t G, int d) { return (size_t)smem_bytes(n_tok, 1, G, d, G * d); }

cudaError_t launch_decode_paged(int dtype, int state_dtype, int d, const PagedDecode& a, cudaStream_t st) {
  if (dtype == kF32)
    return state_dtype == kF32 ? launch_ts<float, float>(a, d, st) : launch_ts<float, bf16>(a, d, st);
  return state_dtype == kF32 ? launch_ts<bf16, float>(a, d, st) : launch_ts<bf16, bf16>(a, d, st);
}

}  // namespace gdn
