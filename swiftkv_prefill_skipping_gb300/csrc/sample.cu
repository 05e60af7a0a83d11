// Next-token sampling with temperature, top-k, top-p and min-p from given uniform numbers.
//
// Per row, with logits l (NaN counts as -inf), m = max l and temperature T > 0 (T <= 0: the
// argmax, lowest id on ties):
//   w_i = exp((l_i - m) / T); order: l descending, then id ascending
//   top-k: the first k of the order; top-p: of those, the ones with less than top_p of their
//   mass before them; min-p: of those, the ones with w_i >= min_p
//   token = the lowest kept id i with sum_{kept j <= i} w_j > u * sum_{kept j} w_j
// All three filters keep a prefix of one order, so together they are one prefix: every element
// above a threshold key, and the first few ids at it.
//
// The chosen token is a whole number that hangs on comparisons of sums of up to 10^5 weights,
// which float32 cannot decide. Weights are therefore fixed-point numbers in 64 bits, w * 2^44
// (weight_fx: the exponent as a pair of floats, a 256-entry table of 2^(j/256) and a short
// polynomial, within 2^-40 of w), and every sum is an integer sum: exact, the same in any
// order, so atomics, the cluster size and the launch shape never change a token.
//
// One thread-block cluster per row: each CTA keeps its slice of the row in shared memory (one
// read of the logits from HBM), and the CTAs exchange maxima, histograms and prefix sums
// through distributed shared memory. A threshold is found by a histogram over 1024 bins that
// are linear in (m - l) / T (masses as three 16-bit limbs, 32-bit shared atomics). The elements of
// the one bin that holds it meet in the cluster's first CTA, if they are at most 2048, which narrows
// their keys ten bits a round; more of them are narrowed by histograms over the cluster.
//
// Bound by latency for few rows (a cluster barrier is 1 us) and by instructions for many: a weight is
// some 45 of them and its histogram up to three shared atomics. 128256 logits, us for 1 / 64 / 256 rows
// (131 MB, 19 us of reading): argmax 4.2 / 12 / 47, no filter 9.4 / 31 / 106, top-k 50 16 / 41 / 146, top-p 0.95
// 25 / 69 / 235, both 23 / 58 / 212, min-p 0.1 11 / 27 / 95.
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "swiftkv.h"

namespace skv {

namespace {

typedef unsigned long long u64;

constexpr int ST = 512;            // threads per CTA
constexpr int SWARPS = ST / 32;
constexpr int NB = 1024;           // histogram bins
constexpr int TAB = 256;           // 2^(j / TAB) table
constexpr int MAXCAND = 2048;      // elements of one bin that one CTA searches (in the room of its bins)
constexpr int FX = 44;             // fixed-point weights: w * 2^FX (360448 of them, times 2^(1/256), stay below 2^63)
constexpr int kMaxSlice = 45056;   // floats of a row one CTA holds (176 KB)
constexpr int kMaxVocab = 8 * kMaxSlice;
constexpr int MAXCHUNK = kMaxSlice / SWARPS / 32 + 1;  // 32-element chunks of a warp's segment

struct SampleParams {
  const float* logits;
  long long ld;
  int V, slice;  // slice: elements per CTA of the cluster, a multiple of 4
  bool vec;      // rows start 16-byte aligned
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  int* tokens;
};

// round(2^(j / 256) * 2^44) by the exponential series, at compile time
struct Pow2Table {
  u64 v[TAB];
  constexpr Pow2Table() : v() {
    for (int j = 0; j < TAB; ++j) {
      const double y = 0.69314718055994530942 * j / TAB;
      double term = 1.0, sum = 0.0;
      for (int k = 1; k < 24; ++k) {
        sum += term;
        term *= y / k;
      }
      v[j] = (u64)(sum * (double)(1ull << FX) + 0.5);
    }
  }
};
__device__ constexpr Pow2Table kPow2 = Pow2Table();

// Shared-memory state of one CTA (ahead of its slice); the cluster's other CTAs read it.
struct alignas(16) Share {  // the slice behind it is written 16 bytes at a time
  u64 mass[NB];                 // this CTA's bins
  u64 tab[TAB];
  unsigned limb[3][NB];         // 16-bit limbs of the bins while they are summed
  u64 warp_mass[SWARPS];
  u64 sums[NB];                 // the cluster's sums of the bins this CTA scans
  u64 part[SWARPS];
  // the row's settings
  float set_t, set_p, set_m, set_u, set_ch, set_cl;
  int set_k;
  // the search for the drawn id: masses, or kept and tied elements, of 32-element chunks
  u64 chunk_mass[MAXCHUNK];
  unsigned chunk_gt[MAXCHUNK], chunk_eq[MAXCHUNK];
  int len[SWARPS];
  int pos;
  float red_f[SWARPS];
  unsigned red_a[SWARPS], red_b[SWARPS];
  // read by the cluster's other CTAs
  float x_max;
  unsigned x_kmin, x_ties;
  unsigned x_key;  // of this CTA alone: min-p's smallest key
  u64 x_mass, x_sum;
  // the bin that a search found
  unsigned d_bin;
  u64 d_before, d_inside;
  // a bin's elements on their way to one key: counted and kept by the cluster's first CTA
  unsigned cand;
};

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared variable in CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ uint32_t remote(const T* p, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ unsigned ld_remote(const unsigned* p, unsigned rank) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_remote(const float* p, unsigned rank) {
  return __uint_as_float(ld_remote(reinterpret_cast<const unsigned*>(p), rank));
}
__device__ __forceinline__ u64 ld_remote(const u64* p, unsigned rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ unsigned add_remote(unsigned* p, unsigned rank, unsigned v) {
  unsigned old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(p, rank)), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void st_remote(float* p, unsigned rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote(p, rank)), "f"(v) : "memory");
}

// Order-preserving map of floats to unsigned (no NaN); -0 and +0 share a key.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// How a row's logits become exponents: c = log2(e) / T as a pair of floats, and a reference
// exponent near m c on the 1/256 grid. All weights of a row are scaled by the one factor
// 2^(m c - ref), which no comparison sees. Far from zero (|m c| > 256, tiny temperatures) l c
// would lose too many bits, and l - m is taken first (`diff`, ref = 0).
struct Scale {
  float m, ch, cl, ref;
  bool diff;
};

// w * 2^FX for w = 2^((l - m) c) up to the row's common factor, within 2^-40 of it. l c is a
// pair p + lo; p = ref + k / 256 + r with |r| <= 2^-9, exactly; 2^(r + lo) - 1 is its Taylor
// series in L (r + lo), L = ln 2, to the fourth term, the leading one again as a pair. Scaled by
// 2^40 it fits 32 bits; the table entry times it is a 64-bit product, shifted into place. The
// shift drops bits and sets the lowest one, the middle of what was dropped, so that 10^5 small
// weights carry no bias.
// No branches, so that a thread's loop runs several weights at once.
template <bool DIFF>
__device__ __forceinline__ u64 weight_of(float l, const Scale& s, const u64* tab) {
  float p, lo;
  if (DIFF) {
    const float dh = l - s.m, bb = dh - l;
    const float dl = (l - (dh - bb)) - (s.m + bb);  // l - m = dh + dl exactly
    p = dh * s.ch;
    lo = fmaf(dl, s.ch, fmaf(dh, s.cl, fmaf(dh, s.ch, -p)));
  } else {
    p = l * s.ch;
    lo = fmaf(l, s.cl, fmaf(l, s.ch, -p));
  }
  const float d = p - s.ref;
  const bool none = !(d > -(float)(FX + 1));  // also l = -inf (c may be 0 or infinite)
  const float magic = 12582912.f;  // 1.5 * 2^23: rounds to an integer held in the low bits
  const float kf = fmaf(none ? 0.f : d, 256.f, magic);
  const int k = __float_as_int(kf) - 0x4b400000;
  const float r = p - fmaf(kf - magic, 1.f / 256.f, s.ref);
  constexpr float S40 = 1099511627776.f;
  constexpr double L = 0.69314718055994530942;
  constexpr float Lh = (float)L * S40;
  constexpr float Ll = (float)(L - (double)(float)L) * S40;
  constexpr float C2 = (float)(L * L / 2 * S40), C3 = (float)(L * L * L / 6 * S40), C4 = (float)(L * L * L * L / 24 * S40);
  const float qh = r * Lh, rs = r + lo;
  float ql = fmaf(lo, Lh, fmaf(r, Ll, fmaf(r, Lh, -qh)));
  ql = fmaf(fmaf(fmaf(C4, rs, C3), rs, C2), rs * rs, ql);
  const int q = __float2int_rn(qh) + __float2int_rn(ql);
  const u64 t = tab[k & (TAB - 1)];               // 2^(j / 256) * 2^FX, below 2^46
  const int t30 = (int)(t >> (FX - 30));          // 30 bits of it and one before the point
  const u64 x = t + (u64)(((long long)t30 * q) >> (70 - FX));
  u64 w = (x >> -(k >> 8)) | 1ull;                // k <= 1, so the shift is 0 .. FX + 1
  if (DIFF && l == s.m) w = 1ull << FX;           // c may be infinite
  return none && !(DIFF && l == s.m) ? 0 : w;
}
__device__ __forceinline__ u64 weight_fx(float l, const Scale& s, const u64* tab) {
  return s.diff ? weight_of<true>(l, s, tab) : weight_of<false>(l, s, tab);
}

// floor(f * w) for a float 0 <= f < 1 and whether that is exact: f = mant * 2^-sh.
__device__ __forceinline__ u64 floor_mul(float f, u64 w, bool* exact = nullptr) {
  const unsigned b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const u64 mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (e ? e : 1);  // at least 24
  const u64 lo = mant * w, hi = __umul64hi(mant, w);  // below 2^87
  u64 q, rest;
  if (sh < 64) {
    q = (lo >> sh) | (hi << (64 - sh));
    rest = lo & ((1ull << sh) - 1);
  } else {
    const int s = min(sh - 64, 63);
    q = hi >> s;
    rest = lo | (hi & ((1ull << s) - 1));
  }
  if (exact) *exact = rest == 0;
  return q;
}
__device__ __forceinline__ u64 ceil_mul(float f, u64 w) {
  if (!(f > 0.f)) return 0;
  bool exact;
  const u64 q = floor_mul(f, w, &exact);
  return exact ? q : q + 1;
}

// The prefix of the order that ends with the first `ties` ids of key `key`.
struct Prefix {
  unsigned key, ties;
  __device__ __forceinline__ bool shorter(const Prefix& o) const {
    return key > o.key || (key == o.key && ties < o.ties);
  }
  // Whether the lane's element (of 32 in ascending order; all lanes call) belongs to it; t0
  // counts the elements at `key` seen so far.
  __device__ __forceinline__ bool keeps(bool in, unsigned k, unsigned& t0, int lane) const {
    if (ties == UINT_MAX) return in && k >= key;
    const unsigned eq = __ballot_sync(0xffffffffu, in && k == key);
    const bool keep = in && (k > key || (k == key && t0 + __popc(eq & ((1u << lane) - 1)) < ties));
    t0 += __popc(eq);
    return keep;
  }
};

template <int C>
__global__ void __launch_bounds__(ST, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Share& sh = *reinterpret_cast<Share*>(smem);
  float* row = reinterpret_cast<float*>(smem + sizeof(Share));
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const int r = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int base = (int)rank * p.slice;
  const int n = max(0, min(p.slice, p.V - base));  // this CTA's ids: [base, base + n)
  const float* src = p.logits + (long long)r * p.ld + base;
  auto sync_all = [&]() {
    if (C > 1) cluster_barrier();
    else __syncthreads();
  };

  griddep_launch_dependents();
  static_assert(TAB <= ST, "one table entry a thread");
  const u64 entry = tid < TAB ? kPow2.v[tid] : 0;
  griddep_wait();
  // ---- the slice and its maximum (NaN becomes -inf): all loads of a round before their use
  float mx = -INFINITY;
  constexpr int LD = 8;
  if (p.vec) {
    const int n4 = n >> 2;
    for (int i0 = tid; i0 < n4; i0 += LD * ST) {
      float4 v[LD];
#pragma unroll
      for (int e = 0; e < LD; ++e)
        if (i0 + e * ST < n4) v[e] = __ldcs(reinterpret_cast<const float4*>(src) + i0 + e * ST);
#pragma unroll
      for (int e = 0; e < LD; ++e) {
        if (i0 + e * ST >= n4) break;
        float4 x = v[e];
        x.x = fmaxf(x.x, -INFINITY);
        x.y = fmaxf(x.y, -INFINITY);
        x.z = fmaxf(x.z, -INFINITY);
        x.w = fmaxf(x.w, -INFINITY);
        mx = fmaxf(fmaxf(mx, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
        *reinterpret_cast<float4*>(row + 4 * (i0 + e * ST)) = x;
      }
    }
    for (int i = 4 * n4 + tid; i < n; i += ST) mx = fmaxf(mx, row[i] = fmaxf(src[i], -INFINITY));
  } else {
    for (int i0 = tid; i0 < n; i0 += 2 * LD * ST) {
      float v[2 * LD];
#pragma unroll
      for (int e = 0; e < 2 * LD; ++e)
        if (i0 + e * ST < n) v[e] = __ldcs(src + i0 + e * ST);
#pragma unroll
      for (int e = 0; e < 2 * LD; ++e)
        if (i0 + e * ST < n) mx = fmaxf(mx, row[i0 + e * ST] = fmaxf(v[e], -INFINITY));
    }
  }
  if (tid < TAB) sh.tab[tid] = entry;
  if (tid == 0) sh.cand = 0;
  if (tid == ST - 1) {
    const float t = p.temperature ? p.temperature[r] : p.temperature_all;
    sh.set_t = t;
    sh.set_k = p.top_k ? p.top_k[r] : p.top_k_all;
    sh.set_p = p.top_p ? p.top_p[r] : p.top_p_all;
    sh.set_m = p.min_p ? p.min_p[r] : p.min_p_all;
    sh.set_u = p.u[r];
    // log2(e) / T as a pair: the quotient and what its product with T leaves
    const float c = 1.442695041f / t;
    sh.set_ch = c;
    sh.set_cl = c > 0.f && c < INFINITY ? (fmaf(-c, t, 1.442695041f) + 1.925963033e-8f) / t : 0.f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) sh.red_f[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < SWARPS; ++w) mx = fmaxf(mx, sh.red_f[w]);
  if (C > 1) {
    if (tid == 0) sh.x_max = mx;
    cluster_barrier();
#pragma unroll
    for (unsigned c = 0; c < (unsigned)C; ++c) mx = fmaxf(mx, ld_remote(&sh.x_max, c));
  }
  const float T = sh.set_t;
  if (!(T > 0.f) || mx == -INFINITY) {  // greedy; a row with no logit above -inf gives id 0
    unsigned at = UINT_MAX;
    for (int i = tid; i < n; i += ST)
      if (row[i] == mx) at = min(at, (unsigned)(base + i));
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sh.red_a[warp] = at;
    __syncthreads();
    for (int w = 0; w < SWARPS; ++w) at = min(at, sh.red_a[w]);
    if (C > 1) {
      if (tid == 0) sh.x_kmin = at;
      cluster_barrier();
      for (unsigned c = 0; c < (unsigned)C; ++c) at = min(at, ld_remote(&sh.x_kmin, c));
    }
    if (rank == 0 && tid == 0) p.tokens[r] = (int)at;
    if (C > 1) cluster_barrier();  // no CTA leaves while another may read its x_kmin
    return;
  }
  const int tk = sh.set_k;
  const float tp = sh.set_p, mp = sh.set_m;
  const bool use_k = tk > 0 && tk < p.V;
  const bool use_p = tp < 1.f;  // NaN: off
  Scale sc;
  sc.m = mx;
  sc.ch = sh.set_ch;
  sc.cl = sh.set_cl;
  sc.diff = !(fabsf(mx * sc.ch) <= 256.f);
  sc.ref = sc.diff ? 0.f : rintf(mx * sc.ch * 256.f) * (1.f / 256.f);
  // Warp w owns the slice's segment [s0, s1), ids ascending. Filters compact the segments in
  // place (lower positions only), so later passes read what is left.
  const int seg = ((n + SWARPS - 1) / SWARPS + 31) & ~31;
  const int s0 = min(n, warp * seg);
  int s1 = min(n, s0 + seg);

  // linear bins over the range where weights are not zero; the last bin takes the rest
  const float bin_scale = fminf(sc.ch * ((float)(NB - 1) / (float)(FX + 1)), FLT_MAX);
  auto bin_of = [&](float l) {
    const float b = (mx - l) * bin_scale;  // NaN (l = m = inf, or inf * 0): bin 0
    return (int)fminf(b > 0.f ? b : 0.f, (float)(NB - 1));
  };
  auto add_mass = [&](int b, u64 w) {
    const unsigned lo = (unsigned)w, hi = (unsigned)(w >> 32);
    atomicAdd(&sh.limb[0][b], lo & 0xffffu);
    if (lo >> 16) atomicAdd(&sh.limb[1][b], lo >> 16);
    if (hi) atomicAdd(&sh.limb[2][b], hi);
  };
  // f(row element, weight function) over this warp's elements, the kind of scale hoisted out
  auto each = [&](auto f) {
    auto go = [&](auto kind) {
      auto weight = [&](float l) { return weight_of<decltype(kind)::value>(l, sc, sh.tab); };
#pragma unroll 4
      for (int i = s0 + lane; i < s1; i += 32) f(row[i], weight);
    };
    if (sc.diff) go(std::true_type());
    else go(std::false_type());
  };
  auto clear = [&]() {
    for (int b = tid; b < NB; b += ST) sh.limb[0][b] = sh.limb[1][b] = sh.limb[2][b] = 0;
    __syncthreads();
  };
  // this CTA's bins as 64-bit masses (or counts, in the first limb), visible to the cluster
  auto publish = [&]() {
    __syncthreads();
    for (int b = tid; b < NB; b += ST)
      sh.mass[b] = (u64)sh.limb[0][b] + ((u64)sh.limb[1][b] << 16) + ((u64)sh.limb[2][b] << 32);
    sync_all();
  };
  // The first bin, in descending order of the logits, at which the cluster's running sum reaches
  // `want`; the sum above it is returned in `before`, the bin's own in `inside`. fraction >= 0: want is
  // that part of all the bins (at least 1). Each CTA sums its NB / C bins over the cluster's copies, so a bin crosses
  // between CTAs once (all CTAs reading all bins took 3 us a search), and only the totals and the
  // decision are exchanged after that.
  auto find = [&](u64& want, float fraction, u64& before, u64& inside) -> int {
    constexpr int BPC = NB / C;
    constexpr int PER = ST >= BPC ? ST / BPC : 1;  // threads per bin, each with C / PER copies
#pragma unroll
    for (int b = tid / PER; b < BPC; b += ST / PER) {
      u64 x = 0;
#pragma unroll
      for (int c = 0; c < C / PER; ++c) x += ld_remote(&sh.mass[rank * BPC + b], (tid % PER) * (C / PER) + c);
#pragma unroll
      for (int o = 1; o < PER; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (tid % PER == 0) sh.sums[b] = x;
    }
    __syncthreads();
    constexpr int PL = BPC / 32;  // bins per lane of the scanning warp
    if (warp == 0) {
      u64 x = 0;
#pragma unroll
      for (int e = 0; e < PL; ++e) x += sh.sums[lane * PL + e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) sh.x_sum = x;
    }
    sync_all();
    u64 tot[C], all = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      tot[c] = ld_remote(&sh.x_sum, c);
      all += tot[c];
    }
    if (fraction >= 0.f) {
      const u64 c = ceil_mul(fraction, all);
      want = c > 0 ? c : 1;
    }
    unsigned owner = 0;
    u64 bm = before, first = before;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (bm < want && want <= bm + tot[c]) {
        owner = c;
        first = bm;
      }
      bm += tot[c];
    }
    // every CTA looks into the owner's bins itself: cheaper than a third barrier
    if (warp == 0) {
      u64 own = 0;
#pragma unroll 8
      for (int e = 0; e < PL; ++e) own += ld_remote(&sh.sums[lane * PL + e], owner);
      u64 x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x = first + x - own;
      if (lane == 0) sh.d_bin = 0;
      __syncwarp();
      if (x < want && want <= x + own)  // one lane
        for (int e = 0; e < PL; ++e) {
          const u64 v = ld_remote(&sh.sums[lane * PL + e], owner);
          if (want <= x + v) {
            sh.d_bin = (unsigned)(owner * BPC + lane * PL + e);
            sh.d_before = x;
            sh.d_inside = v;
            break;
          }
          x += v;
        }
    }
    __syncthreads();
    before = sh.d_before;
    inside = sh.d_inside;
    return (int)sh.d_bin;
  };
  // "The threshold lies in bin `bin` of a first histogram" to one key; `before` and `inside` become
  // the count or mass above that key and at it. Lists hold no element below the bin.
  auto refine = [&](bool by_mass, u64 want, int bin, u64& before, u64& inside) -> unsigned {
    // keys that can fall into the bin: its ends, moved out by more than bin_of can round
    const float width = 1.f / bin_scale, slack = 4e-6f * ((float)(bin + 1) * width + fabsf(mx));
    const float top = mx - (float)bin * width + slack, low = mx - (float)(bin + 1) * width - slack;
    unsigned hi = top < mx ? key_of(top) : key_of(mx);
    unsigned lo = bin < NB - 1 && low > -FLT_MAX ? key_of(low) : 0u;  // NaN and infinite ends: everything
    // The bin's elements, if they are few, meet in the first CTA, which finishes the search alone: a
    // round over the cluster costs it two barriers and an exchange of bins.
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int i = i0 + lane;
      const float l = i < s1 ? row[i] : 0.f;
      const bool in = i < s1 && bin_of(l) == bin;
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (!who) continue;
      unsigned at = 0;
      if (lane == 0) at = add_remote(&sh.cand, 0, __popc(who));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
      if (in && at < MAXCAND) st_remote(reinterpret_cast<float*>(sh.mass) + at, 0, l);
    }
    sync_all();
    const unsigned cands = ld_remote(&sh.cand, 0);
    if (cands <= MAXCAND) {
      if (rank == 0) {
        constexpr int PER = MAXCAND / ST;
        unsigned k[PER];
        u64 w[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int i = tid + e * ST;
          const float l = i < (int)cands ? reinterpret_cast<const float*>(sh.mass)[i] : 0.f;
          k[e] = i < (int)cands ? key_of(l) : 0u;
          w[e] = i < (int)cands ? (by_mass ? weight_fx(l, sc, sh.tab) : 1ull) : 0ull;
        }
        while (lo < hi) {  // ten bits of the key a round, with this CTA's bins alone
          const int s = max(0, 22 - __clz(hi - lo));  // (hi - lo) >> s < NB
          clear();
#pragma unroll
          for (int e = 0; e < PER; ++e)
            if (w[e] && k[e] >= lo && k[e] <= hi) {
              if (by_mass) add_mass((int)((hi - k[e]) >> s), w[e]);
              else atomicAdd(&sh.limb[0][(hi - k[e]) >> s], 1u);
            }
          __syncthreads();
          static_assert(NB == 2 * ST, "two bins a thread");
          u64 v[2], x = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int b = 2 * tid + e;
            x += v[e] = (u64)sh.limb[0][b] + ((u64)sh.limb[1][b] << 16) + ((u64)sh.limb[2][b] << 32);
          }
          u64 upto = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          if (lane == 31) sh.part[warp] = upto;
          if (tid == 0) sh.d_bin = 0;
          __syncthreads();
          u64 c = before + upto - x;
#pragma unroll
          for (int i = 0; i < SWARPS - 1; ++i) c += i < warp ? sh.part[i] : 0ull;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (c < want && want <= c + v[e]) {
              sh.d_bin = (unsigned)(2 * tid + e);
              sh.d_before = c;
              sh.d_inside = v[e];
            }
            c += v[e];
          }
          __syncthreads();
          hi -= sh.d_bin << s;
          lo = max(lo, hi - ((1u << s) - 1));
          before = sh.d_before;
          inside = sh.d_inside;
          __syncthreads();  // read before the next round writes
        }
        if (tid == 0) {
          sh.d_bin = lo;
          sh.d_before = before;
          sh.d_inside = inside;
          sh.cand = 0;
        }
      }
      sync_all();
      before = ld_remote(&sh.d_before, 0);
      inside = ld_remote(&sh.d_inside, 0);
      return ld_remote(&sh.d_bin, 0);
    }
    sync_all();  // everyone has read the count
    if (rank == 0 && tid == 0) sh.cand = 0;
    for (int it = 0; it < 5 && lo < hi; ++it) {  // ten bits of the key a round
      const int s = max(0, 22 - __clz(hi - lo));  // (hi - lo) >> s < NB
      clear();
      for (int i = s0 + lane; i < s1; i += 32) {
        const float l = row[i];
        const unsigned k = key_of(l);
        if (k >= lo && k <= hi && bin_of(l) == bin) {
          const int b = (int)((hi - k) >> s);
          if (by_mass) add_mass(b, weight_fx(l, sc, sh.tab));
          else atomicAdd(&sh.limb[0][b], 1u);
        }
      }
      publish();
      const unsigned b = (unsigned)find(want, -1.f, before, inside);
      hi -= b << s;
      lo = max(lo, hi - ((1u << s) - 1));
    }
    return lo;
  };
  // Keeps the elements that pass `keep` (all lanes call it), each warp's segment in place.
  auto squeeze = [&](auto keep) {
    int out = s0;
    for (int i0 = s0; i0 < s1; i0 += 128) {
      float l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) l[e] = i0 + 32 * e + lane < s1 ? row[i0 + 32 * e + lane] : 0.f;
      __syncwarp();  // read before lower positions are written
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool k = keep(i0 + 32 * e + lane < s1, l[e]);
        const unsigned kept = __ballot_sync(0xffffffffu, k);
        if (k) row[out + __popc(kept & ((1u << lane) - 1))] = l[e];
        out += __popc(kept);
      }
      __syncwarp();
    }
    s1 = out;
  };

  Prefix pre;
  pre.key = 0;
  pre.ties = UINT_MAX;    // everything
  unsigned tie_base = 0;  // elements at pre.key with lower ids than this warp's segment
  // Keeps what belongs to the prefix, each warp's segment in place.
  auto compact = [&]() {
    if (pre.ties != UINT_MAX) {
      unsigned t = 0;
      for (int i = s0 + lane; i < s1; i += 32) t += key_of(row[i]) == pre.key;
      t = __reduce_add_sync(0xffffffffu, t);
      if (lane == 0) sh.red_a[warp] = t;
      __syncthreads();
      unsigned all = 0;
      tie_base = 0;
      for (int w = 0; w < SWARPS; ++w) {
        if (w < warp) tie_base += sh.red_a[w];
        all += sh.red_a[w];
      }
      if (C > 1) {
        if (tid == 0) sh.x_ties = all;
        cluster_barrier();
        for (unsigned c = 0; c + 1 <= rank; ++c) tie_base += ld_remote(&sh.x_ties, c);
      }
      sync_all();
    }
    unsigned t0 = tie_base;
    squeeze([&](bool in, float l) { return pre.keeps(in, key_of(l), t0, lane); });
  };
  // Drops what lies below the threshold's bin of a first histogram, before that bin is refined.
  auto drop_below = [&](int bin) {
    squeeze([&](bool in, float l) { return in && bin_of(l) <= bin; });
  };

  int list_bin = -1;  // the lists hold the elements of the bins up to this one
  if (use_k) {
    clear();
#pragma unroll 4
    for (int i = s0 + lane; i < s1; i += 32) atomicAdd(&sh.limb[0][bin_of(row[i])], 1u);
    publish();
    u64 want = (u64)tk, before = 0, inside = 0;
    const int bin = find(want, -1.f, before, inside);
    drop_below(bin);
    pre.key = refine(false, want, bin, before, inside);
    pre.ties = want - before < inside ? (unsigned)(want - before) : UINT_MAX;
    compact();
  }
  if (use_p) {
    // elements with less than top_p of the mass before them: the last one kept is the one at
    // which the running mass reaches it, and the first of the order is always kept
    clear();
    each([&](float l, auto weight) {
      const u64 w = weight(l);
      if (w) add_mass(bin_of(l), w);
    });
    publish();
    u64 want = 0, before = 0, inside = 0;
    const int bin = find(want, tp, before, inside);
    drop_below(bin);
    Prefix pp;
    pp.key = refine(true, want, bin, before, inside);
    pp.ties = UINT_MAX;
    if (want - before < inside) {  // not all of the key's elements
      const u64 w = weight_fx(value_of(pp.key), sc, sh.tab), ties = w ? (want - before + w - 1) / w : UINT_MAX;
      if (ties * w < inside) pp.ties = (unsigned)ties;
    }
    if (pp.shorter(pre)) pre = pp;
    if (!use_k) list_bin = bin;
  }
  if (mp > 0.f) {
    // the smallest key, up to the maximum's, whose weight is min_p of the maximum's: weights grow
    // with the key, and a warp tries 32 keys a round
    unsigned lo = 0, hi = key_of(mx);
    if (mp >= 1.f) lo = hi;
    if (warp == 0) {
      const u64 least = ceil_mul(fminf(mp, 1.f), weight_fx(mx, sc, sh.tab));
      for (int shift = 27; shift > -5; shift -= 5) {
        const unsigned step = shift > 0 ? 1u << shift : 1u, off = step * (unsigned)lane;
        const unsigned cand = off < hi - lo ? lo + off : hi;
        const float x = cand < 0x007fffffu ? -INFINITY : value_of(cand);  // smaller keys are NaN patterns
        const unsigned ok = __ballot_sync(0xffffffffu, weight_fx(x, sc, sh.tab) >= least);
        const int f = ok ? __ffs(ok) - 1 : 31;
        const unsigned c0 = __shfl_sync(0xffffffffu, cand, max(f - 1, 0)), c1 = __shfl_sync(0xffffffffu, cand, f);
        if (ok && f > 0) lo = min(c0 + 1, c1);
        if (!ok) lo = min(c1 + 1, hi);
        if (ok) hi = c1;
      }
      if (lane == 0) sh.x_key = lo;
    }
    __syncthreads();
    const unsigned key = sh.x_key;
    if (key > pre.key) {
      pre.key = key;
      pre.ties = UINT_MAX;
    }
  }
  // After top-p alone nearly all that is left is kept: the passes below skip the rest instead of
  // moving everything once more.
  const bool listed = list_bin >= 0 && pre.ties == UINT_MAX;
  if ((use_p || mp > 0.f) && !listed) compact();

  // ---- the draw: running sums over the kept ids in ascending order
  u64 sum = 0;
  if (listed) each([&](float l, auto weight) { sum += key_of(l) >= pre.key ? weight(l) : 0ull; });
  else each([&](float l, auto weight) { sum += weight(l); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    sh.warp_mass[warp] = sum;
    sh.len[warp] = s1 - s0;
  }
  __syncthreads();
  u64 mine = 0;
#pragma unroll
  for (int w = 0; w < SWARPS; ++w) mine += sh.warp_mass[w];
  u64 before = 0, total = mine;
  if (C > 1) {
    if (tid == 0) sh.x_mass = mine;
    cluster_barrier();
    total = 0;
#pragma unroll
    for (unsigned c = 0; c < (unsigned)C; ++c) {
      const u64 x = ld_remote(&sh.x_mass, c);
      if (c + 1 <= rank) before += x;
      total += x;
    }
    cluster_barrier();  // the last remote read: from here on every CTA is on its own
  }
  // sums are whole numbers, so "exceeds the real number u * total" is "is at least
  // floor(u * total) + 1"
  float u = sh.set_u;
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;  // NaN and -0 too
  const u64 target = floor_mul(u, total) + 1;
  if (!(before < target && target <= before + mine)) return;
  // The id is in this CTA's slice: the warps share the segment that holds it, a chunk of 32 at a
  // time, and warp 0 picks the chunk and the element.
  int win = 0;
#pragma unroll
  for (int w = 0; w < SWARPS - 1; ++w) {
    const u64 x = sh.warp_mass[w];
    if (win == w && before + x < target) {
      before += x;
      win = w + 1;
    }
  }
  const int w0 = min(n, win * seg), w1 = w0 + sh.len[win];
  const int chunks = (w1 - w0 + 31) / 32;
  auto mass_at = [&](int i) -> u64 {
    return i < w1 && (!listed || key_of(row[i]) >= pre.key) ? weight_fx(row[i], sc, sh.tab) : 0ull;
  };
  for (int c = warp; c < chunks; c += SWARPS) {
    const int i = w0 + 32 * c + lane;
    u64 x = mass_at(i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) sh.chunk_mass[c] = x;
  }
  __syncthreads();
  auto scan = [&](u64 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  };
  const bool whole = pre.key == 0 && pre.ties == UINT_MAX;  // nothing was dropped
  if (warp == 0) {
    int c = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const u64 upto = before + scan(c0 + lane < chunks ? sh.chunk_mass[c0 + lane] : 0ull);
      const unsigned hit = __ballot_sync(0xffffffffu, upto >= target);
      if (hit) {
        c = c0 + __ffs(hit) - 1;
        if (c > c0) before = __shfl_sync(0xffffffffu, upto, c - c0 - 1);
        break;
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
    const int i = w0 + 32 * c + lane;
    const u64 upto = before + scan(mass_at(i));
    const unsigned hit = __ballot_sync(0xffffffffu, upto >= target);
    const int at = 32 * c + __ffs(hit) - 1;  // within the segment's kept elements
    if (lane == 0) {
      if (whole) p.tokens[r] = base + w0 + at;
      sh.pos = at;
    }
  }
  if (whole) return;
  // the segment was compacted: its pos-th kept element, counted in the logits again
  const int e1 = min(n, win * seg + seg), all = (e1 - w0 + 31) / 32;
  Prefix in_list = pre;
  if (listed) in_list = Prefix{1u, UINT_MAX};  // its elements have key 2, the others 0
  auto key_in = [&](int c) {
    const int i = w0 + 32 * c + lane;
    if (i >= e1) return 0u;  // below every key
    const float l = fmaxf(src[i], -INFINITY);
    return listed ? (bin_of(l) <= list_bin ? 2u : 0u) : key_of(l);
  };
  for (int c = warp; c < all; c += SWARPS) {
    const unsigned k = key_in(c);
    const unsigned gt = __ballot_sync(0xffffffffu, k > in_list.key), eq = __ballot_sync(0xffffffffu, k == in_list.key && k);
    if (lane == 0) {
      sh.chunk_gt[c] = __popc(gt);
      sh.chunk_eq[c] = __popc(eq);
    }
  }
  if (lane == 0 && warp == win) sh.red_a[0] = tie_base;  // ties before this segment
  __syncthreads();
  if (warp == 0) {
    unsigned ties = sh.red_a[0];
    int left = sh.pos;
    for (int c0 = 0; c0 < all; c0 += 32) {
      const bool in = c0 + lane < all;
      const unsigned gt = in ? sh.chunk_gt[c0 + lane] : 0u, eq = in ? sh.chunk_eq[c0 + lane] : 0u;
      const unsigned eq_to = (unsigned)scan(eq) + ties;  // ties up to and with the lane's chunk
      const unsigned kept_to = (unsigned)scan(gt + min(eq_to, in_list.ties) - min(eq_to - eq, in_list.ties));
      const unsigned hit = __ballot_sync(0xffffffffu, kept_to > (unsigned)left);
      if (hit) {
        const int who = __ffs(hit) - 1;
        const unsigned skip = who ? __shfl_sync(0xffffffffu, kept_to, who - 1) : 0u;
        unsigned t0 = who ? __shfl_sync(0xffffffffu, eq_to, who - 1) : ties;
        const int i = w0 + 32 * (c0 + who) + lane;
        unsigned kept = __ballot_sync(0xffffffffu, in_list.keeps(i < e1, key_in(c0 + who), t0, lane));
        for (left -= (int)skip; left > 0; --left) kept &= kept - 1;
        if (lane == 0) p.tokens[r] = base + w0 + 32 * (c0 + who) + __ffs(kept) - 1;
        break;
      }
      left -= (int)__shfl_sync(0xffffffffu, kept_to, 31);
      ties = __shfl_sync(0xffffffffu, eq_to, 31);
    }
  }
}

template <int C>
cudaError_t launch_rows(const SampleParams& p, int rows, size_t smem, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(sample_kernel<C>),
                                       (int)(sizeof(Share) + (size_t)kMaxSlice * 4), once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * C);
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<C>, p);
}

}  // namespace

}  // namespace skv

using namespace skv;

extern "C" int swiftkv_sample(const float* logits, int rows, int vocab, long long ld, const swiftkv_sampling* s,
                              const float* u, int32_t* tokens, swiftkv_stream stream) {
  if (rows < 0 || vocab < 1) return set_error(SWIFTKV_EINVAL, "need rows >= 0 and vocab >= 1");
  if (rows == 0) return SWIFTKV_OK;
  if (!logits || !s || !u || !tokens) return set_error(SWIFTKV_EINVAL, "null logits / settings / u / tokens");
  if (ld < vocab) return set_error(SWIFTKV_EINVAL, "row stride smaller than vocab");
  const void* const arrays[] = {logits, u, tokens, s->temperature, s->top_k, s->top_p, s->min_p};
  for (const void* a : arrays)
    if (reinterpret_cast<uintptr_t>(a) & 3) return set_error(SWIFTKV_EINVAL, "misaligned logits / u / tokens / settings");
  if (vocab > kMaxVocab) return set_error(SWIFTKV_EUNSUPPORTED, "vocab above 360448");
  if (rows > (1 << 27)) return set_error(SWIFTKV_EUNSUPPORTED, "more than 2^27 rows");
  SampleParams p;
  p.logits = logits;
  p.ld = ld;
  p.V = vocab;
  p.vec = (reinterpret_cast<uintptr_t>(logits) & 15) == 0 && ld % 4 == 0;
  p.u = u;
  p.temperature = s->temperature;
  p.top_k = s->top_k;
  p.top_p = s->top_p;
  p.min_p = s->min_p;
  p.temperature_all = s->temperature_all;
  p.top_k_all = s->top_k_all;
  p.top_p_all = s->top_p_all;
  p.min_p_all = s->min_p_all;
  p.tokens = tokens;
  // CTAs of a row's cluster, by vocabulary alone, chosen for few rows: top-p over 1 row takes 16.2 us with
  // one CTA and 16.7 with two at 8192 ids, 18.2 and 17.6 at 12288; with 2 / 4 / 8 of them 20.7 / 16.4 / 15.1 at
  // 24576, 24.4 / 18.9 / 16.8 at 32768, - / 22.0 / 18.7 at 50256. Hundreds of rows would rather have fewer (256
  // rows: 65 us with one against 84 with four at 32768, 102 with four against 156 with eight at 50256), but
  // not at 128256 (258 with four, 236 with eight).
  const int C = vocab > 32768 ? 8 : vocab > 16384 ? 4 : vocab > 8192 ? 2 : 1;
  p.slice = ((vocab + C - 1) / C + 3) & ~3;
  const size_t smem = sizeof(Share) + (size_t)p.slice * 4;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = C == 8 ? launch_rows<8>(p, rows, smem, st) : C == 4 ? launch_rows<4>(p, rows, smem, st)
                      : C == 2 ? launch_rows<2>(p, rows, smem, st) : launch_rows<1>(p, rows, smem, st);
  if (e != cudaSuccess) return set_error(SWIFTKV_ECUDA, cudaGetErrorString(e));
  return SWIFTKV_OK;
}
