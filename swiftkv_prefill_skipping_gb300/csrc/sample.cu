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
// are linear in (m - l) / T (masses as three 16-bit limbs, 32-bit shared atomics), then by
// histograms over the key range of the one bin that holds it until a single key is left.
#include <cfloat>
#include <climits>
#include <cmath>

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
constexpr int FX = 44;             // fixed-point weights: w * 2^FX
constexpr int kMaxSlice = 45056;   // floats of a row one CTA holds (176 KB)
constexpr int kMaxVocab = 8 * kMaxSlice;

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
  u64 mass[NB];                 // this CTA's bin masses
  u64 tab[TAB];
  unsigned limb[3][NB];         // 16-bit limbs of the bin masses while they are summed
  unsigned cnt[NB];             // bin counts
  u64 warp_mass[SWARPS];
  unsigned warp_cnt[SWARPS];
  float red_f[SWARPS];
  unsigned red_a[SWARPS], red_b[SWARPS];
  // exchanged between the CTAs
  float x_max;
  unsigned x_idx, x_kmin, x_kmax, x_ties;
  u64 x_mass;
  // rank 0's decisions
  int d_bin;
  u64 d_before_mass;
  unsigned d_before_cnt, d_in_cnt;
};

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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
__device__ __forceinline__ int ld_remote(const int* p, unsigned rank) {
  return (int)ld_remote(reinterpret_cast<const unsigned*>(p), rank);
}
__device__ __forceinline__ float ld_remote(const float* p, unsigned rank) {
  return __uint_as_float(ld_remote(reinterpret_cast<const unsigned*>(p), rank));
}
__device__ __forceinline__ u64 ld_remote(const u64* p, unsigned rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}

// Order-preserving map of floats to unsigned (no NaN); -0 and +0 share a key.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The row's exponent scale log2(e) / T as a pair of floats.
struct Scale {
  float m, ch, cl;
};

// round(2^FX * exp((l - m) / T)). The exponent t = (l - m) * c is kept as th + tl: l - m by a
// two-sum, the product by fused multiply-adds; |error of t| < 2^-42. th = k / 256 + r with
// |r| <= 2^-9, and 2^r - 1 = L r + (L r)^2 / 2 + ... (L = ln 2, Taylor terms up to the
// fourth), its leading term again as a pair. Scaled by 2^40 the sum fits 32 bits; the table
// entry times it is a 64-bit product, shifted into place and rounded to nearest (truncation
// would bias the sum of 10^5 small weights by 2^-28).
__device__ __forceinline__ u64 weight_fx(float l, const Scale& s, const u64* tab) {
  if (l == s.m) return 1ull << FX;
  const float dh = l - s.m;
  const float th = dh * s.ch;
  if (!(th > -(float)(FX + 1))) return 0;  // also l = -inf
  const float bb = dh - l;
  const float dl = (l - (dh - bb)) - (s.m + bb);  // l - m = dh + dl exactly
  float tl = fmaf(dh, s.ch, -th);
  tl = fmaf(dh, s.cl, tl);
  tl = fmaf(dl, s.ch, tl);
  const float magic = 12582912.f;  // 1.5 * 2^23: rounds to an integer held in the low bits
  const float kf = fmaf(th, 256.f, magic);
  const int k = __float_as_int(kf) - 0x4b400000;
  const float r = fmaf(kf - magic, -1.f / 256.f, th);
  constexpr float S40 = 1099511627776.f;
  constexpr double L = 0.69314718055994530942;
  constexpr float Lh = (float)L * S40;
  constexpr float Ll = (float)(L - (double)(float)L) * S40;
  constexpr float C2 = (float)(L * L / 2 * S40), C3 = (float)(L * L * L / 6 * S40), C4 = (float)(L * L * L * L / 24 * S40);
  const float qh = r * Lh;
  float ql = fmaf(r, Lh, -qh);
  ql = fmaf(r, Ll, ql);
  ql = fmaf(tl, Lh, ql);
  ql = fmaf(tl * r, 2.f * C2, ql);
  ql = fmaf(fmaf(fmaf(C4, r, C3), r, C2), r * r, ql);
  const int q = __float2int_rn(qh) + __float2int_rn(ql);
  const u64 t = tab[k & (TAB - 1)];                       // 2^(j / 256) * 2^44
  const int t31 = (int)((t + (1u << 13)) >> 14);          // ... * 2^30 (below 2^31)
  const long long x = (long long)t + (((long long)t31 * q) >> 26);  // 2^30 * 2^40 / 2^26 = 2^44
  const int n = -(k >> 8);                                // 0 .. FX + 1
  return (((u64)x << 1 >> n) + 1) >> 1;
}

// Per-CTA sum and count over all threads.
__device__ __forceinline__ u64 block_sum(u64 v, u64* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
#pragma unroll
  for (int i = 0; i < SWARPS; ++i) s += tmp[i];
  __syncthreads();
  return s;
}

// ceil(f * w) for a float 0 <= f < 1 (or 1): f is mant * 2^-sh exactly.
__device__ __forceinline__ u64 ceil_mul(float f, u64 w) {
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return w;
  const unsigned b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const u64 mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (e ? e : 1);  // f = mant * 2^-sh, sh >= 24
  const u64 lo = mant * w, hi = __umul64hi(mant, w);
  if (sh >= 128) return (lo | hi) != 0;
  const u64 up_lo = sh >= 64 ? ~0ull : (1ull << sh) - 1, up_hi = sh > 64 ? (sh >= 128 ? ~0ull : (1ull << (sh - 64)) - 1) : 0;
  u64 a = lo + up_lo;
  u64 c = hi + up_hi + (a < lo);
  if (sh == 64) return c;
  return sh > 64 ? c >> (sh - 64) : (a >> sh) | (c << (64 - sh));
}

// The prefix of the order that ends at (and includes `ties` ids of) key `key`.
struct Prefix {
  unsigned key, ties;
  __device__ __forceinline__ bool shorter(const Prefix& o) const { return key > o.key || (key == o.key && ties < o.ties); }
};

template <int C>
__global__ void __launch_bounds__(ST) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Share& sh = *reinterpret_cast<Share*>(smem);
  float* row = reinterpret_cast<float*>(smem + sizeof(Share));
  const unsigned rank = C > 1 ? cluster_rank() : 0;
  const int r = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int base = (int)rank * p.slice;
  const int n = max(0, min(p.slice, p.V - base));  // this CTA's ids: [base, base + n)
  const float* src = p.logits + (long long)r * p.ld + base;

  griddep_launch_dependents();
  for (int i = tid; i < TAB; i += ST) sh.tab[i] = kPow2.v[i];
  griddep_wait();
  // ---- the slice, its maximum and that one's lowest id
  float mx = -INFINITY;
  int mi = INT_MAX;
  auto take = [&](float v, int i) {
    v = v != v ? -INFINITY : v;
    if (v > mx || mi == INT_MAX) {  // ids ascend within a thread
      mx = v;
      mi = i;
    }
    return v;
  };
  if (p.vec) {
    const int n4 = n >> 2;
#pragma unroll 4
    for (int i = tid; i < n4; i += ST) {
      float4 v = __ldcs(reinterpret_cast<const float4*>(src) + i);
      v.x = take(v.x, 4 * i);
      v.y = take(v.y, 4 * i + 1);
      v.z = take(v.z, 4 * i + 2);
      v.w = take(v.w, 4 * i + 3);
      *reinterpret_cast<float4*>(row + 4 * i) = v;
    }
    for (int i = 4 * n4 + tid; i < n; i += ST) row[i] = take(src[i], i);
  } else {
#pragma unroll 4
    for (int i = tid; i < n; i += ST) row[i] = take(__ldcs(src + i), i);
  }
  unsigned gi = mi == INT_MAX ? UINT_MAX : (unsigned)(base + mi);
  auto better = [&](float v, unsigned i) {
    if (i != UINT_MAX && (gi == UINT_MAX || v > mx || (v == mx && i < gi))) {
      mx = v;
      gi = i;
    }
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v2 = __shfl_xor_sync(0xffffffffu, mx, o);
    const unsigned i2 = __shfl_xor_sync(0xffffffffu, gi, o);
    better(v2, i2);
  }
  if (lane == 0) {
    sh.red_f[warp] = mx;
    sh.red_a[warp] = gi;
  }
  __syncthreads();
  for (int w = 0; w < SWARPS; ++w) better(sh.red_f[w], sh.red_a[w]);
  if (C > 1) {
    if (tid == 0) {
      sh.x_max = mx;
      sh.x_idx = gi;
    }
    cluster_barrier();
    for (unsigned c = 0; c < (unsigned)C; ++c) better(ld_remote(&sh.x_max, c), ld_remote(&sh.x_idx, c));
  }
  const float T = p.temperature ? p.temperature[r] : p.temperature_all;
  if (!(T > 0.f) || mx == -INFINITY) {  // greedy; a row with no finite logit gives id 0
    if (rank == 0 && tid == 0) p.tokens[r] = mx == -INFINITY ? 0 : (int)gi;
    if (C > 1) cluster_barrier();  // no CTA leaves while another may read its x_max
    return;
  }
  const int tk = p.top_k ? p.top_k[r] : p.top_k_all;
  const float tp = p.top_p ? p.top_p[r] : p.top_p_all;
  const float mp = p.min_p ? p.min_p[r] : p.min_p_all;
  const bool use_k = tk > 0 && tk < p.V;
  const bool use_p = tp < 1.f;  // NaN: off
  Scale sc;
  sc.m = mx;
  {
    const double c = 1.4426950408889634074 / (double)T;
    sc.ch = (float)c;
    sc.cl = isinf(sc.ch) ? 0.f : (float)(c - (double)sc.ch);
  }
  // linear bins over the range where weights are not zero; the last bin takes the rest
  const float bin_scale = fminf(sc.ch * ((float)(NB - 1) / (float)(FX + 1)), FLT_MAX);
  auto bin_of = [&](float l) {
    const float b = (sc.m - l) * bin_scale;  // NaN (l = m = inf, or 0 * inf): bin 0
    return b >= (float)(NB - 1) ? NB - 1 : (b > 0.f ? (int)b : 0);
  };
  auto add_mass = [&](int b, u64 w) {
    atomicAdd(&sh.limb[0][b], (unsigned)(w & 0xffffu));
    atomicAdd(&sh.limb[1][b], (unsigned)((w >> 16) & 0xffffu));
    atomicAdd(&sh.limb[2][b], (unsigned)(w >> 32));
  };
  auto clear = [&]() {
    for (int b = tid; b < NB; b += ST) {
      sh.cnt[b] = 0;
      sh.limb[0][b] = sh.limb[1][b] = sh.limb[2][b] = 0;
    }
    __syncthreads();
  };
  auto publish = [&](bool mass) {  // limbs -> 64-bit masses, visible to the cluster
    __syncthreads();
    if (mass)
      for (int b = tid; b < NB; b += ST)
        sh.mass[b] = (u64)sh.limb[0][b] + ((u64)sh.limb[1][b] << 16) + ((u64)sh.limb[2][b] << 32);
    if (C > 1) cluster_barrier(); else __syncthreads();
  };
  // Rank-independent scan: every CTA sums the cluster's bins (thread t: bins 2t, 2t + 1) and
  // finds the first bin, in descending order of the logits, at which the running count or mass
  // reaches `want`. Fills sh.d_* and returns with the block synchronised.
  auto find = [&](bool by_mass, bool with_mass, u64 want, u64 before_mass, unsigned before_cnt) {
    u64 ms[2] = {0, 0};
    unsigned ct[2] = {0, 0};
    for (unsigned c = 0; c < (unsigned)C; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (with_mass) ms[e] += ld_remote(&sh.mass[2 * tid + e], c);
        ct[e] += ld_remote(&sh.cnt[2 * tid + e], c);
      }
    u64 im = ms[0] + ms[1];
    unsigned ic = ct[0] + ct[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 m2 = __shfl_up_sync(0xffffffffu, im, o);
      const unsigned c2 = __shfl_up_sync(0xffffffffu, ic, o);
      if (lane >= o) {
        im += m2;
        ic += c2;
      }
    }
    if (lane == 31) {
      sh.warp_mass[warp] = im;
      sh.warp_cnt[warp] = ic;
    }
    if (tid == 0) sh.d_bin = -1;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      im += sh.warp_mass[w];
      ic += sh.warp_cnt[w];
    }
    u64 bm = before_mass + im - ms[0] - ms[1];
    unsigned bc = before_cnt + ic - ct[0] - ct[1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // by count: the bin with bc < want <= bc + ct; by mass: bm < want <= bm + ms
      const u64 b0 = by_mass ? bm : (u64)bc, b1 = by_mass ? bm + ms[e] : (u64)(bc + ct[e]);
      if (b0 < want && want <= b1) {
        sh.d_bin = 2 * tid + e;
        sh.d_before_mass = bm;
        sh.d_before_cnt = bc;
        sh.d_in_cnt = ct[e];
      }
      bm += ms[e];
      bc += ct[e];
    }
    if (C > 1) cluster_barrier(); else __syncthreads();  // also: nobody still reads the bins
  };
  // Smallest and largest key of the cluster's elements in the open interval test `in`.
  auto key_range = [&](auto in, unsigned& lo, unsigned& hi) {
    unsigned a = UINT_MAX, b = 0;
    for (int i = tid; i < n; i += ST) {
      const float l = row[i];
      if (in(l)) {
        const unsigned k = key_of(l);
        a = min(a, k);
        b = max(b, k);
      }
    }
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    if (lane == 0) {
      sh.red_a[warp] = a;
      sh.red_b[warp] = b;
    }
    __syncthreads();
    for (int w = 0; w < SWARPS; ++w) {
      a = min(a, sh.red_a[w]);
      b = max(b, sh.red_b[w]);
    }
    if (C > 1) {
      if (tid == 0) {
        sh.x_kmin = a;
        sh.x_kmax = b;
      }
      cluster_barrier();
      for (unsigned c = 0; c < (unsigned)C; ++c) {
        a = min(a, ld_remote(&sh.x_kmin, c));
        b = max(b, ld_remote(&sh.x_kmax, c));
      }
      cluster_barrier();
    } else {
      __syncthreads();
    }
    lo = a;
    hi = b;
  };
  // Refines "the threshold lies in bin `bin` of the first histogram" to one key. On return
  // lo is that key, before_* what lies above it and in_cnt how many elements equal it.
  auto refine = [&](bool by_mass, bool with_mass, u64 want, int bin, u64& before_mass, unsigned& before_cnt,
                    unsigned& in_cnt) -> unsigned {
    unsigned lo, hi;
    key_range([&](float l) { return bin_of(l) == bin; }, lo, hi);
    for (int it = 0; it < 5 && lo != hi; ++it) {  // ten bits of the key a round
      const unsigned span = hi - lo;
      const int s = max(0, 32 - __clz(span) - 10);  // span >> s < NB
      clear();
      for (int i = tid; i < n; i += ST) {
        const unsigned k = key_of(row[i]);
        if (k >= lo && k <= hi) {
          const int b = (int)((hi - k) >> s);
          atomicAdd(&sh.cnt[b], 1u);
          if (with_mass) add_mass(b, weight_fx(row[i], sc, sh.tab));
        }
      }
      publish(with_mass);
      find(by_mass, with_mass, want, before_mass, before_cnt);
      const unsigned b = (unsigned)sh.d_bin;
      before_mass = sh.d_before_mass;
      before_cnt = sh.d_before_cnt;
      in_cnt = sh.d_in_cnt;
      const unsigned nh = hi - (b << s);
      lo = max(lo, nh - ((1u << s) - 1));
      hi = nh;
      __syncthreads();
    }
    return lo;
  };

  Prefix pre;
  pre.key = 0;
  pre.ties = UINT_MAX;  // everything
  if (use_k || use_p) {
    clear();
    for (int i = tid; i < n; i += ST) {
      const float l = row[i];
      const int b = bin_of(l);
      atomicAdd(&sh.cnt[b], 1u);
      if (use_p) {
        const u64 w = weight_fx(l, sc, sh.tab);
        if (w) add_mass(b, w);
      }
    }
    publish(use_p);
    u64 total = 0, bm;  // bm, bc, ic: mass and count before the threshold's bin, count inside it
    unsigned bc, ic;
    if (use_k) {
      find(false, use_p, (u64)tk, 0, 0);
      const int bin = sh.d_bin;
      bm = sh.d_before_mass;
      bc = sh.d_before_cnt;
      ic = sh.d_in_cnt;
      pre.key = refine(false, use_p, (u64)tk, bin, bm, bc, ic);
      pre.ties = (unsigned)tk - bc;
    }
    if (use_k && use_p) {
      // mass of the top k; the top-p search starts from a histogram of those alone
      total = bm + (u64)pre.ties * weight_fx(value_of(pre.key), sc, sh.tab);
      clear();
      for (int i = tid; i < n; i += ST) {
        const float l = row[i];
        if (key_of(l) >= pre.key) {
          const int b = bin_of(l);
          atomicAdd(&sh.cnt[b], 1u);
          add_mass(b, weight_fx(l, sc, sh.tab));
        }
      }
      publish(true);
    } else if (use_p) {
      u64 t = 0;
      for (unsigned c = 0; c < (unsigned)C; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) t += ld_remote(&sh.mass[2 * tid + e], c);
      total = block_sum(t, sh.warp_mass);
    }
    if (use_p) {
      // elements with less than top_p of the mass before them: the last one kept is the one at
      // which the running mass reaches it, and the first of the order is always kept
      const u64 c = ceil_mul(tp, total), want = c > 0 ? c : 1;
      find(true, true, want, 0, 0);
      const int bin = sh.d_bin;
      bm = sh.d_before_mass;
      bc = sh.d_before_cnt;
      ic = sh.d_in_cnt;
      Prefix pp;
      pp.key = refine(true, true, want, bin, bm, bc, ic);
      const u64 w = weight_fx(value_of(pp.key), sc, sh.tab);
      const u64 ties = w ? (want - bm + w - 1) / w : UINT_MAX;
      pp.ties = ties > UINT_MAX ? UINT_MAX : (unsigned)ties;
      if (pp.shorter(pre)) pre = pp;
    }
  }
  if (mp > 0.f) {
    // w >= min_p  <=>  l >= m + T ln(min_p)
    const double thr = (double)mx + (double)T * log((double)fminf(mp, 1.f));
    const float tf = mp >= 1.f ? mx : __double2float_ru(thr);
    // an infinite product (T = inf) leaves everything; NaN cannot arise for mx > -inf, T > 0
    const unsigned key = key_of(tf);
    if (key > pre.key) {
      pre.key = key;
      pre.ties = UINT_MAX;
    }
  }

  // ---- ids in ascending order: warp w of CTA c owns a contiguous segment
  const int seg = ((n + SWARPS - 1) / SWARPS + 31) & ~31;
  const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
  unsigned tie_base = 0;  // equal-key ids before this warp's segment
  if (pre.ties != UINT_MAX) {
    unsigned t = 0;
    for (int i = s0 + lane; i < s1; i += 32) t += key_of(row[i]) == pre.key;
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) sh.red_a[warp] = t;
    __syncthreads();
    unsigned all = 0;
    for (int w = 0; w < SWARPS; ++w) {
      if (w < warp) tie_base += sh.red_a[w];
      all += sh.red_a[w];
    }
    if (C > 1) {
      if (tid == 0) sh.x_ties = all;
      cluster_barrier();
      for (unsigned c = 0; c < rank; ++c) tie_base += ld_remote(&sh.x_ties, c);
    }
  }
  // kept weight of id i (all lanes call; t0: ties seen so far in this segment)
  auto kept = [&](int i, unsigned& t0) -> u64 {
    const bool in = i < s1;
    const float l = in ? row[i] : 0.f;
    const unsigned k = in ? key_of(l) : 0u;
    bool keep = in && k > pre.key;
    if (pre.ties == UINT_MAX) {
      keep = in && k >= pre.key;
    } else {
      const unsigned eq = __ballot_sync(0xffffffffu, in && k == pre.key);
      if (in && k == pre.key) keep = t0 + __popc(eq & ((1u << lane) - 1)) < pre.ties;
      t0 += __popc(eq);
    }
    return keep ? weight_fx(l, sc, sh.tab) : 0ull;
  };
  u64 sum = 0;
  {
    unsigned t0 = tie_base;
    for (int i = s0; i < s1; i += 32) sum += kept(i + lane, t0);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh.warp_mass[warp] = sum;
  __syncthreads();
  u64 before = 0, total = 0;
  for (int w = 0; w < SWARPS; ++w) {
    if (w < warp) before += sh.warp_mass[w];
    total += sh.warp_mass[w];
  }
  if (C > 1) {
    if (tid == 0) sh.x_mass = total;
    cluster_barrier();
    const u64 mine = total;
    total = 0;
    for (unsigned c = 0; c < (unsigned)C; ++c) {
      const u64 x = c == rank ? mine : ld_remote(&sh.x_mass, c);
      if (c < rank) before += x;
      total += x;
    }
  }
  // the first id whose running sum exceeds u * total; sums are whole, so "exceeds the real
  // number u * total" is "is at least floor(u * total) + 1"
  float u = p.u[r];
  u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
  const u64 up = ceil_mul(u, total);
  u64 target;
  {
    // ceil(u * total) equals the product exactly when the product is whole
    const unsigned b = __float_as_uint(u);
    const int e = (int)(b >> 23);
    const u64 mant = u > 0.f ? (e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu) : 0;
    const int s = 150 - (e ? e : 1);
    const u64 lo = mant * total, hi = __umul64hi(mant, total);
    bool whole;
    if (s >= 128) whole = (lo | hi) == 0;
    else if (s > 64) whole = lo == 0 && (hi & ((1ull << (s - 64)) - 1)) == 0;
    else if (s == 64) whole = lo == 0;
    else whole = (lo & ((1ull << s) - 1)) == 0;
    target = whole ? up + 1 : up;
  }
  if (before < target && target <= before + sum) {  // one warp of the cluster
    unsigned t0 = tie_base;
    u64 run = before;
    for (int i = s0; i < s1; i += 32) {
      const u64 w = kept(i + lane, t0);
      u64 inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + inc >= target);
      if (hit) {
        if (lane == 0) p.tokens[r] = base + i + __ffs(hit) - 1;
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (C > 1) cluster_barrier();  // shared memory stays until every CTA has read it
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
  if ((reinterpret_cast<uintptr_t>(logits) & 3) || (reinterpret_cast<uintptr_t>(u) & 3))
    return set_error(SWIFTKV_EINVAL, "misaligned logits / u");
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
  const int C = vocab > 32768 ? 8 : vocab > 16384 ? 4 : vocab > 8192 ? 2 : 1;
  p.slice = ((vocab + C - 1) / C + 3) & ~3;
  const size_t smem = sizeof(Share) + (size_t)p.slice * 4;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = C == 8 ? launch_rows<8>(p, rows, smem, st) : C == 4 ? launch_rows<4>(p, rows, smem, st)
                      : C == 2 ? launch_rows<2>(p, rows, smem, st) : launch_rows<1>(p, rows, smem, st);
  if (e != cudaSuccess) return set_error(SWIFTKV_ECUDA, cudaGetErrorString(e));
  return SWIFTKV_OK;
}
