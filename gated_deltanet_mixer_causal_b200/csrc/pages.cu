// pages.cu -- the pages of a state pool: copy, take, reference counts, compaction plan.
//
// A page holds one sequence's state (or its conv taps) of one layer. A copy moves whole pages,
// so it is bound by HBM: 2 x page bytes for each entry. The lists, counts and plans are a few
// ints per page and run in one CTA (3 to 4 us for 256 pages).
//
// Measured, share of the bytes at the copy rate: 200 pages of 2 MB 129 us (100 %); 256 pages of
// 3.2 MB compacted, plan included, 70 us (89 %; 75 to 78 as a call); one page into 8 new ones in 4
// layers, with the taking of the pages, 26 us (68 %; writes alone are 17 us; 29 to 31 as a call); 64
// beams of 1.1 MB in 4 layers reordered in place 84 us (83 %: short runs of every page in turn, see
// below).
#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kPlainThreads = 256;
constexpr int kPlainLog = 14;           // log2 of a plain tile's bytes
constexpr int kPlanThreads = 1024;

// Exclusive prefix sum of v over a CTA of WARPS warps, and the total.
template <int WARPS> __device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();                    // the previous call's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < WARPS ? warp_sums[lane] : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, m);
      if (lane >= m) s += y;
    }
    if (lane < WARPS) warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[WARPS - 1];
  return (warp ? warp_sums[warp - 1] : 0) + x - v;
}

// ------------------------------------------------------------------------------- copy
//
// Entry i moves page src[i] to page dst[i], as if every source were read before any destination
// is written. Bound by HBM. A CTA copies a tile, its loads into registers before its stores. Tiles
// are not looped over by resident CTAs: taken up in the order of the pages by the hardware's
// scheduler, they keep the reads and writes of the moment close together (419 MB copied: 127 us,
// 6.6 TB/s; by a grid of resident CTAs that stride over the tiles 145 us, by bulk copies through
// shared memory 138 us).
//
// Where the caller knows that no destination repeats and none is another entry's source (plain), a
// tile is a run of 16 KB of one page. Else it is a column of ALL entries, so that no other CTA
// touches its bytes and the barrier between its loads and its stores is the only order needed; a
// hash table of the destinations in shared memory, made by each CTA for itself, gives the last
// entry of each, the one that counts. There the run of one page is a tile's bytes by the entries
// (512 of 32 KB, 1 KB of 64 KB for 64 entries), and short runs cost bandwidth: 64 chained pages of
// 2 MB 5.6 TB/s, 256 6.1, 1,000 of 256 KB 3.5, 2,000 of them (32-byte runs) 2.0.

struct Table {
  int32_t* key;    // destination page, -1: empty
  int32_t* val;    // its last entry
  uint32_t mask;
};

__device__ __forceinline__ uint32_t slot_of(int32_t page, uint32_t mask) { return ((uint32_t)page * 2654435761u >> 7) & mask; }

__device__ __forceinline__ int find(const Table& t, int32_t page) {
  uint32_t s = slot_of(page, t.mask);
  while (true) {                      // the table is at most half full, so an empty slot ends it
    const int32_t k = t.key[s];
    if (k == page) return t.val[s];
    if (k == -1) return -1;
    s = (s + 1) & t.mask;
  }
}

// log2 of a tile's bytes: U 16-byte words of each of T threads
__host__ __device__ constexpr int tile_log(int T, int U) {
  int log = 4;
  while (16 << (log - 4) < T * U * 16) ++log;
  return log;
}

// first[k]: the first CTA of pool k
struct CopyTiles { uint32_t first[kPagesMaxPools]; };

__device__ __forceinline__ int pool_of(const CopyTiles& t, int n_pools) {
  int k = 0;
  while (k + 1 < n_pools && blockIdx.x >= t.first[k + 1]) ++k;
  return k;
}

template <int T, int U>
__global__ void __launch_bounds__(T, 1024 / T)
pages_copy_kernel(const PagesCopy a, const CopyTiles t, uint32_t slots, int log_n) {
  extern __shared__ int32_t sm[];
  Table tab{sm, sm + slots, slots - 1};
  int32_t* ms = sm + 2 * slots;       // [n] sources, -1: the entry does not count
  int32_t* md = ms + a.n;
  wait_for_previous_grid();
  for (uint32_t h = threadIdx.x; h < slots; h += T) { tab.key[h] = -1; tab.val[h] = -1; }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += T) {
    const int32_t s = a.src[i], d = a.dst[i];
    const bool in = s >= 0 && s < a.src_pages && d >= 0 && d < a.dst_pages;
    ms[i] = in ? s : -1;
    md[i] = d;
    if (!in) continue;
    uint32_t at = slot_of(d, tab.mask);
    while (true) {
      const int32_t was = atomicCAS(&tab.key[at], -1, d);
      if (was == -1 || was == d) break;
      at = (at + 1) & tab.mask;
    }
    atomicMax(&tab.val[at], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += T)
    if (ms[i] >= 0 && find(tab, md[i]) != i) ms[i] = -1;
  __syncthreads();
  constexpr int kLog = tile_log(T, U);
  const int k = pool_of(t, a.n_pools);
  const PagePool& p = a.pool[k];
  const int lw = kLog - log_n, lu = lw - 4;
  const uint32_t cta = blockIdx.x - t.first[k], cols = (uint32_t)((p.page_bytes + (1LL << lw) - 1) >> lw), layer = cta / cols;
  const int64_t col = (int64_t)(cta - layer * cols) << lw, left = p.page_bytes - col;
  const char* from = p.src + layer * p.src_layer + col;
  char* to = p.dst + layer * p.dst_layer + col;
  uint4 v[U];
  int32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int idx = u * T + threadIdx.x, off = (idx & ((1 << lu) - 1)) << 4;
    e[u] = idx >> lu;
    int32_t m = -1;
    if (e[u] < a.n && off < left) m = ms[e[u]];
    if (m < 0) e[u] = -1;
    else v[u] = *reinterpret_cast<const uint4*>(from + m * p.src_page + off);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int off = ((u * T + threadIdx.x) & ((1 << lu) - 1)) << 4;
    if (e[u] >= 0) *reinterpret_cast<uint4*>(to + md[e[u]] * p.dst_page + off) = v[u];
  }
}

// Groups of entries of a pool: 2^(kPlainLog - lw) entries each, 2^lw bytes of a page (its power of
// two, at most a tile's). In a long list a CTA takes its columns of every step-th group, fold of
// them: a plan's list is padded, and a CTA that only finds an entry void costs its place for about
// 1 us (compacting 256 pages of 3 MB, 128 entries of which half are void: 100 us by one group a
// CTA, 69 by four).
struct PlainShape {
  int lw;
  uint32_t cols, groups, fold, step;
};
__host__ __device__ inline PlainShape plain_shape(int64_t page_bytes, int n) {
  PlainShape s;
  s.lw = 4;
  while (s.lw < kPlainLog && (1LL << s.lw) < page_bytes) ++s.lw;
  s.cols = (uint32_t)((page_bytes + (1LL << s.lw) - 1) >> s.lw);
  s.groups = ((uint32_t)(n - 1) >> (kPlainLog - s.lw)) + 1;
  s.fold = s.groups >= 32 ? 4 : 1;
  s.step = (s.groups + s.fold - 1) / s.fold;
  return s;
}

__global__ void __launch_bounds__(kPlainThreads, 6)
pages_copy_plain_kernel(const PagesCopy a, const CopyTiles t) {
  constexpr int U = (1 << kPlainLog) / (kPlainThreads * 16);
  wait_for_previous_grid();
  const int k = pool_of(t, a.n_pools);
  const PagePool& p = a.pool[k];
  const PlainShape sh = plain_shape(p.page_bytes, a.n);
  const uint32_t cta = blockIdx.x - t.first[k], rest = cta / sh.cols, layer = rest / sh.step;
  const int64_t col = (int64_t)(cta - rest * sh.cols) << sh.lw, left = p.page_bytes - col;
  const int lu = sh.lw - 4;
  for (uint32_t g = rest - layer * sh.step; g < sh.groups; g += sh.step) {
    if (sh.lw == kPlainLog) {           // one entry a tile
      const int32_t s = a.src[g], d = a.dst[g];
      if (s < 0 || s >= a.src_pages || d < 0 || d >= a.dst_pages || (p.same && s == d)) continue;
      const int off = threadIdx.x * 16;
      const char* from = p.src + layer * p.src_layer + s * p.src_page + col + off;
      char* to = p.dst + layer * p.dst_layer + d * p.dst_page + col + off;
      constexpr int kStep = kPlainThreads * 16;
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (off + u * kStep < left) v[u] = *reinterpret_cast<const uint4*>(from + u * kStep);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (off + u * kStep < left) *reinterpret_cast<uint4*>(to + u * kStep) = v[u];
    } else {                            // whole pages of some entries
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int idx = u * kPlainThreads + threadIdx.x;
        const int off = (idx & ((1 << lu) - 1)) << 4, e = (int)(g << (kPlainLog - sh.lw)) + (idx >> lu);
        if (e >= a.n || off >= left) continue;
        const int32_t s = a.src[e], d = a.dst[e];
        if (s < 0 || s >= a.src_pages || d < 0 || d >= a.dst_pages || (p.same && s == d)) continue;
        *reinterpret_cast<uint4*>(p.dst + layer * p.dst_layer + d * p.dst_page + off) =
            *reinterpret_cast<const uint4*>(p.src + layer * p.src_layer + s * p.src_page + off);
      }
    }
  }
}

// ------------------------------------------------------------------- lists and counts

// out[i] = the next lowest free page for every entry that wants one, -1 for the others. The sources
// are looked at before any page is taken, so none of them is among the pages taken.
__global__ void __launch_bounds__(kPlanThreads)
pages_take_kernel(int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n, int32_t* out) {
  __shared__ int sums[32];
  __shared__ int32_t want[kPagesMaxList];
  allow_next_grid();
  int n_want = 0, total;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const bool w = i < n && (!src || (src[i] >= 0 && src[i] < n_pages && refs[src[i]] > 0));
    const int at = n_want + block_scan<kPlanThreads / 32>(w, sums, total);
    if (w) want[at] = i;
    if (i < n) out[i] = -1;
    n_want += total;
  }
  __syncthreads();
  int taken = 0;
  for (int64_t p0 = 0; p0 < n_pages && taken < n_want; p0 += kPlanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool is_free = p < n_pages && refs[p] <= 0;
    const int at = taken + block_scan<kPlanThreads / 32>(is_free, sums, total);
    if (is_free && at < n_want) { out[want[at]] = (int32_t)p; refs[p] = 1; }
    taken += total;
  }
}

// refs[p] += delta for each entry, never below 0
__global__ void __launch_bounds__(kPlanThreads)
pages_ref_kernel(int32_t* refs, int32_t n_pages, const int32_t* pages, int32_t n, int32_t delta) {
  for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
    const int32_t p = pages[i];
    if (p >= 0 && p < n_pages) atomicAdd(&refs[p], delta);
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
    const int32_t p = pages[i];
    if (p >= 0 && p < n_pages) atomicMax(&refs[p], 0);
  }
}

// The i-th hole below the number of live pages takes the i-th live page behind it.
__global__ void __launch_bounds__(kPlanThreads)
pages_plan_kernel(int32_t* refs, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* src,
                  int32_t* dst, int32_t* map, int32_t* n_live) {
  __shared__ int sums[32];
  allow_next_grid();
  int total, live_all = 0;
  for (int64_t p0 = 0; p0 < n_pages; p0 += kPlanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool live = p < n_pages && refs[p] > 0;
    block_scan<kPlanThreads / 32>(live, sums, total);
    live_all += total;
    if (p < n_pages) map[p] = live ? (int32_t)p : -1;
  }
  const int half = n_pages / 2;
  for (int i = threadIdx.x; i < half; i += kPlanThreads) src[i] = dst[i] = -1;
  __syncthreads();
  int holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < n_pages; p0 += kPlanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool in = p < n_pages, live = in && refs[p] > 0;
    const bool hole = in && !live && p < live_all, mover = live && p >= live_all;
    const int hat = holes + block_scan<kPlanThreads / 32>(hole, sums, total);
    holes += total;
    const int mat = movers + block_scan<kPlanThreads / 32>(mover, sums, total);
    movers += total;
    if (hole) dst[hat] = (int32_t)p;
    if (mover) src[mat] = (int32_t)p;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) {
    const int32_t s = src[i], d = dst[i];
    refs[d] = refs[s];
    refs[s] = 0;
    map[s] = d;
  }
  // a free page's count is 0, also where a caller left it below
  __syncthreads();
  for (int64_t p = live_all + threadIdx.x; p < n_pages; p += kPlanThreads) refs[p] = 0;
  for (int64_t i = threadIdx.x; i < n_table; i += kPlanThreads) {
    const int32_t p = table[i];
    if (p >= 0 && p < n_pages) table[i] = map[p];
  }
  if (threadIdx.x == 0) *n_live = live_all;
}

// CTAs of a call, and the first of each pool.
int64_t plain_ctas(const PagesCopy& a, CopyTiles& t) {
  int64_t ctas = 0;
  for (int k = 0; k < a.n_pools; ++k) {
    const PlainShape s = plain_shape(a.pool[k].page_bytes, a.n);
    t.first[k] = (uint32_t)ctas;
    const int64_t cols = (a.pool[k].page_bytes + (1LL << s.lw) - 1) >> s.lw;     // s.cols may have wrapped
    ctas += cols * s.step * a.pool[k].layers;
  }
  return ctas;
}

int log_of(int n) {
  int log = 0;
  while ((1 << log) < n) ++log;
  return log;
}

int64_t general_ctas(const PagesCopy& a, int log_tile, CopyTiles& t) {
  const int lw = log_tile - log_of(a.n);
  int64_t ctas = 0;
  for (int k = 0; k < a.n_pools; ++k) {
    t.first[k] = (uint32_t)ctas;
    ctas += ((a.pool[k].page_bytes + (1LL << lw) - 1) >> lw) * a.pool[k].layers;
  }
  return ctas;
}

template <int T, int U>
cudaError_t launch_general(const PagesCopy& a, cudaStream_t st) {
  CopyTiles t{};
  const int64_t ctas = general_ctas(a, tile_log(T, U), t);
  const uint32_t slots = 2u << log_of(a.n < 16 ? 16 : a.n);
  const size_t smem = 8 * ((size_t)slots + a.n);
  static std::atomic<uint64_t> prepared{0};
  const cudaError_t e = raise_smem_limit(pages_copy_kernel<T, U>, 64 * 1024, prepared);
  if (e != cudaSuccess) return e;
  return launch_overlapped(pages_copy_kernel<T, U>, dim3((unsigned)ctas), dim3(T), smem, st, a, t, slots, log_of(a.n));
}

// The general form's two tiles: 32 KB by 256 threads up to 128 entries (64 pages of 2 MB 48 us, 128
// 91; by 64 KB 47 and 98), 64 KB by 512 threads beyond (256 of them 176 us, by 32 KB 187; 1,000 of
// 256 KB 149, by 32 KB 284).
constexpr int kSmallList = 128;
static_assert(kPagesMaxList << 4 <= 1 << tile_log(512, 8), "a tile holds 16 bytes of every entry");

}  // namespace

bool pages_copy_fits(const PagesCopy& a, bool plain) {
  CopyTiles t;
  const int64_t ctas = plain ? plain_ctas(a, t) : general_ctas(a, a.n <= kSmallList ? tile_log(256, 8) : tile_log(512, 8), t);
  return ctas <= 0x7fffffffLL;
}

cudaError_t launch_pages_copy(const PagesCopy& a, bool plain, cudaStream_t st) {
  if (plain) {
    CopyTiles t{};
    const int64_t ctas = plain_ctas(a, t);
    return launch_overlapped(pages_copy_plain_kernel, dim3((unsigned)ctas), dim3(kPlainThreads), 0, st, a, t);
  }
  return a.n <= kSmallList ? launch_general<256, 8>(a, st) : launch_general<512, 8>(a, st);
}

cudaError_t launch_pages_take(int32_t* refs, int32_t n_pages, const int32_t* src, int32_t n, int32_t* out,
                              cudaStream_t st) {
  pages_take_kernel<<<1, kPlanThreads, 0, st>>>(refs, n_pages, src, n, out);
  return cudaGetLastError();
}

cudaError_t launch_pages_ref(int32_t* refs, int32_t n_pages, const int32_t* pages, int32_t n, int32_t delta,
                             cudaStream_t st) {
  pages_ref_kernel<<<1, kPlanThreads, 0, st>>>(refs, n_pages, pages, n, delta);
  return cudaGetLastError();
}

cudaError_t launch_pages_plan(int32_t* refs, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* src,
                              int32_t* dst, int32_t* map, int32_t* n_live, cudaStream_t st) {
  pages_plan_kernel<<<1, kPlanThreads, 0, st>>>(refs, n_pages, table, n_table, src, dst, map, n_live);
  return cudaGetLastError();
}

}  // namespace gdn
