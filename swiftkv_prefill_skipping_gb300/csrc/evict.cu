// Eviction from the paged cache by accumulated attention weight. Per (cache, sequence, KV head)
// with n keys: the first `sinks` and the last `recent` stay, and of the others those with the
// largest scores (ties: lower index first; NaN ranks last), `keep` in all; the kept keys move, in
// order, to rows 0 .. of the destination pages, K, V, FP8 scales and scores alike.
//
// evict_select_kernel: one CTA per list. Scores become order-preserving 32-bit keys in shared
// memory (protected keys the largest); three rounds of histograms over 11, 11 and 10 bits find the
// keep-th largest key, and one ordered pass writes the kept indices, ties by index. The floats of a
// kept key (its score, FP8 scales) move here. Bound by latency: every round is a pass over shared
// memory and three barriers. 512 lists of 7000 keys: 39 us. Lists of more than 49152 keys, what shared
// memory holds, are read from memory in every round: one of 49152 keys takes 62 us, of 49153 90.
//
// evict_copy_kernel, evict_shift_kernel: the bound, HBM: kept rows are read once and written once.
// To other pages (copy), CTAs split the kept list freely. In place (shift) every destination row lies
// at or below its source, so a CTA walks one list in order: a chunk is loaded whole before any of it
// is written, and the next chunk is loaded before that, which only reads rows that no earlier write
// reaches. Rows of a list are cut into 64-byte columns, each its own CTA, so that one sequence still
// fills the GPU. 16 sequences of ~7000 keys to 2048, 4 caches of 8 heads x 128, bf16, to other pages:
// 1.07 GB in 172 us, 6.2 TB/s of a copy's 6.8; 221 us with the selection, which comes before every move
// though lists do not depend on one another. In place 484 us: a list is walked by 8 CTAs in order, a chunk
// at a time. FP8 139 and 261 us.
#include <climits>

#include "common.cuh"
#include "pdl.cuh"
#include "serving.h"

namespace skv {

namespace {

constexpr int ET = 512;               // threads of the selection
constexpr int EWARPS = ET / 32;
constexpr int kSelectSmemKeys = 49152;  // lists up to this long keep their keys in shared memory

// Order-preserving map of scores; NaN is the least, and only protected keys are UINT_MAX.
__device__ __forceinline__ unsigned score_key(float x) {
  if (x != x) return 0;
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct List {
  int c, s, h, n;  // cache (within the call), sequence, KV head, keys
};
// The lengths and pool pointers of a call.
struct Pools {
  const int* lens;
  void* const* ptrs;
  int n;  // caches of the model
  __device__ __forceinline__ Pools(const EvictArgs& a, const InlineInts& inl)
      : lens(list_base(a.lists, inl)), ptrs(reinterpret_cast<void* const*>(lens + a.o_ptrs)), n(a.num_ptrs) {}
  __device__ __forceinline__ unsigned char* k(int c) const { return static_cast<unsigned char*>(ptrs[c]); }
  __device__ __forceinline__ unsigned char* v(int c) const { return static_cast<unsigned char*>(ptrs[n + c]); }
  __device__ __forceinline__ float* scores(int c) const { return static_cast<float*>(ptrs[2 * n + c]); }
  __device__ __forceinline__ float* ks(int c) const { return static_cast<float*>(ptrs[3 * n + c]); }
  __device__ __forceinline__ float* vs(int c) const { return static_cast<float*>(ptrs[4 * n + c]); }
};
__device__ __forceinline__ List list_at(const EvictArgs& a, const Pools& pools, int i) {
  List l;
  l.h = i % a.n_kv;
  l.s = i / a.n_kv % a.P;
  l.c = i / a.n_kv / a.P;
  l.n = pools.lens[l.s];
  return l;
}
// Row index (page, head, slot) of key j of a list in the pools, -1 on a page outside them.
__device__ __forceinline__ long long row_of(const int* bt, int width, int num_pages, int n_kv, const List& l, int j) {
  const int page = bt[(size_t)l.s * width + (j >> 4)];
  if (page < 0 || page >= num_pages) return -1;
  return ((long long)page * n_kv + l.h) * kPageSize + (j & 15);
}

// Digits of a key, most significant first: 11 + 11 + 10 bits. Scores crowd into few exponents, and
// two more bits a digit than a byte spread their first histogram over enough bins to need no
// aggregation within the warp.
constexpr int EBINS = 2048;
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }

__global__ void __launch_bounds__(ET) evict_select_kernel(const EvictArgs a, const __grid_constant__ InlineInts inl,
                                                          int in_smem) {
  extern __shared__ __align__(16) unsigned keys[];  // [n rounded up to pages] when in_smem
  __shared__ unsigned hist[EBINS];
  __shared__ unsigned s_sum[EWARPS], s_key, s_left;
  __shared__ int s_cnt[2][EWARPS];
  griddep_launch_dependents();
  griddep_wait();
  const Pools pools(a, inl);
  const List l = list_at(a, pools, blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* scores = pools.scores(a.first_cache + l.c);
  int* kept = a.kept + (size_t)blockIdx.x * a.keep;
  const int n = l.n, pages = (n + kPageSize - 1) / kPageSize;
  const int* bt = a.src_bt + (size_t)l.s * a.src_pages;
  // an entry outside the pool: the status says so, and the list is left as it is
  int bad = 0;
  const int out_pages = (min(n, a.keep) + kPageSize - 1) / kPageSize;
  for (int p = tid; p < pages; p += ET) bad |= bt[p] < 0 || bt[p] >= a.num_pages;
  for (int p = tid; p < out_pages; p += ET) {
    const int page = a.dst_bt[(size_t)l.s * a.dst_pages + p];
    bad |= page < 0 || page >= a.num_pages;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(a.status, kStatusBadPage);
    for (int i = tid; i < a.keep; i += ET) kept[i] = -1;
    return;
  }
  // keys of rows 4 q .. 4 q + 3 (a quarter of a page); rows behind the list: 0, never counted
  auto quad = [&](int q) -> uint4 {
    const float4 v = *reinterpret_cast<const float4*>(
        scores + ((size_t)bt[q >> 2] * a.n_kv + l.h) * kPageSize + (q & 3) * 4);
    const float f[4] = {v.x, v.y, v.z, v.w};
    unsigned k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 4 * q + e;
      k[e] = j >= n ? 0u : j < a.sinks || j >= n - a.recent ? UINT_MAX : score_key(f[e]);
    }
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  if (n <= a.keep) {
    for (int i = tid; i < a.keep; i += ET) kept[i] = i < n ? i : -1;
  } else {
    const int quads = pages * 4;
    if (in_smem) {
      constexpr int U = 4;
      for (int q0 = tid; q0 < quads; q0 += ET * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (q0 + u * ET < quads) v[u] = quad(q0 + u * ET);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (q0 + u * ET < quads) reinterpret_cast<uint4*>(keys)[q0 + u * ET] = v[u];
      }
    }
    auto key4 = [&](int q) { return in_smem ? reinterpret_cast<const uint4*>(keys)[q] : quad(q); };
    // the keep-th largest key, a digit a round
    unsigned prefix = 0, left = (unsigned)a.keep;
    for (int d = 0; d < 3; ++d) {
      const int shift = digit_shift(d), bits = d == 2 ? 10 : 11;
      for (int b = tid; b < EBINS; b += ET) hist[b] = 0;
      __syncthreads();
      const unsigned mask = d == 0 ? 0u : ~0u << (shift + bits);
      for (int q = tid; q < quads; q += ET) {
        const uint4 v = key4(q);
        const unsigned k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((k[e] & mask) == prefix && 4 * q + e < n) atomicAdd(&hist[(k[e] >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // descending: thread t owns bins top - 4 t .. top - 4 t - 3
      constexpr int PER = EBINS / ET;
      unsigned c[PER], mine = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) mine += c[e] = hist[EBINS - 1 - PER * tid - e];
      unsigned upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) s_sum[warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += s_sum[w];
      unsigned before = upto - mine;
      if (before < left && left <= upto) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          if (before < left && left <= before + c[e]) {
            s_key = prefix | ((unsigned)(EBINS - 1 - PER * tid - e) << shift);
            s_left = left - before;
          }
          before += c[e];
        }
      }
      __syncthreads();
      prefix = s_key;
      left = s_left;
    }
    // ordered pass: everything above the key, and the first `left` at it
    int above = 0, ties = 0;  // before this round
    for (int q0 = 0; q0 < quads; q0 += ET) {
      const int q = q0 + tid, par = (q0 / ET) & 1;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (q < quads) v = key4(q);
      const unsigned k[4] = {v.x, v.y, v.z, v.w};
      unsigned gt = 0, eq = 0;  // of the thread's four keys
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = q < quads && 4 * q + e < n;
        gt |= (unsigned)(in && k[e] > prefix) << e;
        eq |= (unsigned)(in && k[e] == prefix) << e;
      }
      int both = __popc(gt) | __popc(eq) << 16, upto = both;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) s_cnt[par][warp] = upto;
      __syncthreads();
      int first = upto - both, all = 0;
#pragma unroll
      for (int w = 0; w < EWARPS; ++w) {
        const int c = s_cnt[par][w];
        if (w < warp) first += c;
        all += c;
      }
      int g = above + (first & 0xffff), t = ties + (first >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_gt = gt >> e & 1, is_eq = eq >> e & 1;
        if (is_gt || (is_eq && t < (int)left)) kept[g + min(t, (int)left)] = 4 * q + e;
        g += is_gt;
        t += is_eq;
      }
      above += all & 0xffff;
      ties += all >> 16;
    }
  }
  __syncthreads();  // kept, written by this CTA, is read below
  // the kept keys' floats; a round is read whole before it is written (in place, rows move down)
  const int m = min(n, a.keep);
  const int c = a.first_cache + l.c;
  float* arrays[3] = {pools.scores(c), a.fp8 ? pools.ks(c) : nullptr, a.fp8 ? pools.vs(c) : nullptr};
  constexpr int U = 4;
  for (int i0 = 0; i0 < m; i0 += ET * U) {
    float v[U][3];
    long long to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * ET + tid;
      to[u] = -1;
      if (i < m) {
        const long long from = row_of(a.src_bt, a.src_pages, a.num_pages, a.n_kv, l, kept[i]);
        to[u] = row_of(a.dst_bt, a.dst_pages, a.num_pages, a.n_kv, l, i);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (arrays[t]) v[u][t] = arrays[t][from];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0)
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (arrays[t]) arrays[t][to[u]] = v[u][t];
  }
}

constexpr int MT = 256;  // threads of the move

// To other pages: CTA (list, part of the kept list); K and V of a row by neighbouring threads.
constexpr int kPartBytes = 32768;
__global__ void __launch_bounds__(MT) evict_copy_kernel(const EvictArgs a, const __grid_constant__ InlineInts inl, int parts) {
  griddep_launch_dependents();
  griddep_wait();
  const int li = blockIdx.x / parts, part = blockIdx.x - li * parts;
  const Pools pools(a, inl);
  const List l = list_at(a, pools, li);
  const int* kept = a.kept + (size_t)li * a.keep;
  const int vecs = a.row_bytes / 16, rows = kPartBytes / a.row_bytes;
  const int i0 = part * rows, i1 = min(min(l.n, a.keep), i0 + rows);
  unsigned char* k = pools.k(a.first_cache + l.c);
  unsigned char* v = pools.v(a.first_cache + l.c);
  const int count = (i1 - i0) * vecs;
  constexpr int U = 4;
  for (int e0 = threadIdx.x; e0 < count; e0 += MT * U) {
    uint4 x[U], y[U];
    long long to[U];
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int e = e0 + t * MT;
      to[t] = -1;
      if (e < count) {
        const int i = i0 + e / vecs, src = kept[i];
        if (src >= 0) {
          const size_t off = (size_t)row_of(a.src_bt, a.src_pages, a.num_pages, a.n_kv, l, src) * a.row_bytes + e % vecs * 16;
          x[t] = __ldcs(reinterpret_cast<const uint4*>(k + off));
          y[t] = __ldcs(reinterpret_cast<const uint4*>(v + off));
          to[t] = row_of(a.dst_bt, a.dst_pages, a.num_pages, a.n_kv, l, i) * a.row_bytes + e % vecs * 16;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < U; ++t)
      if (to[t] >= 0) {
        *reinterpret_cast<uint4*>(k + to[t]) = x[t];
        *reinterpret_cast<uint4*>(v + to[t]) = y[t];
      }
  }
}

// In place: CTA (list, K or V, 64-byte column). 4 threads a row, 64 U rows a chunk, the next chunk
// loaded before the current one is written.
__global__ void __launch_bounds__(MT) evict_shift_kernel(const EvictArgs a, const __grid_constant__ InlineInts inl, int cols) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int U = 8, RPC = MT / 4 * U;
  const int col = blockIdx.x % cols, sel = blockIdx.x / cols % 2, li = blockIdx.x / cols / 2;
  const Pools pools(a, inl);
  const List l = list_at(a, pools, li);
  const int* kept = a.kept + (size_t)li * a.keep;
  const int m = min(l.n, a.keep);
  unsigned char* pool = sel ? pools.v(a.first_cache + l.c) : pools.k(a.first_cache + l.c);
  const size_t at = col * 64 + threadIdx.x % 4 * 16;  // this thread's 16 bytes of a row
  uint4 x[U], y[U];
  auto row_off = [&](const int* bt, int width, int j) {
    return (size_t)row_of(bt, width, a.num_pages, a.n_kv, l, j) * a.row_bytes + at;
  };
  // chunk c of the list: kept rows that move (src > i; a row at its place stays untouched)
  auto load = [&](int c, uint4* v) {
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int i = c * RPC + t * (MT / 4) + threadIdx.x / 4;
      const int src = i < m ? kept[i] : -1;
      if (src > i) v[t] = *reinterpret_cast<const uint4*>(pool + row_off(a.src_bt, a.src_pages, src));
    }
  };
  auto store = [&](int c, const uint4* v) {
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int i = c * RPC + t * (MT / 4) + threadIdx.x / 4;
      const int src = i < m ? kept[i] : -1;
      if (src > i) *reinterpret_cast<uint4*>(pool + row_off(a.dst_bt, a.dst_pages, i)) = v[t];
    }
  };
  const int chunks = (m + RPC - 1) / RPC;
  if (chunks > 0) load(0, x);
  for (int c = 0; c < chunks; c += 2) {
    if (c + 1 < chunks) load(c + 1, y);
    __syncthreads();  // every thread holds its rows of chunk c
    store(c, x);
    if (c + 1 >= chunks) break;
    if (c + 2 < chunks) load(c + 2, x);
    __syncthreads();
    store(c + 1, y);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, const InlineInts& inl, int max_len, cudaStream_t s) {
  const long long lists = (long long)a.num_caches * a.P * a.n_kv;
  const int parts = (int)(((long long)a.keep * a.row_bytes + kPartBytes - 1) / kPartBytes);
  const int cols = a.row_bytes / 64;
  const long long ctas = a.in_place ? lists * 2 * cols : lists * parts;
  if (lists <= 0) return cudaSuccess;
  if (ctas > INT_MAX || a.row_bytes % 64) return cudaErrorNotSupported;
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(evict_select_kernel), kSelectSmemKeys * 4, once);
  if (e != cudaSuccess) return e;
  const int in_smem = max_len <= kSelectSmemKeys;
  e = launch_pdl(evict_select_kernel, dim3((unsigned)lists), dim3(ET), in_smem ? (size_t)(max_len + 15) / 16 * 64 : 0, s, a, inl, in_smem);
  if (e != cudaSuccess) return e;
  if (a.in_place) return launch_pdl(evict_shift_kernel, dim3((unsigned)ctas), dim3(MT), 0, s, a, inl, cols);
  return launch_pdl(evict_copy_kernel, dim3((unsigned)ctas), dim3(MT), 0, s, a, inl, parts);
}

}  // namespace skv
