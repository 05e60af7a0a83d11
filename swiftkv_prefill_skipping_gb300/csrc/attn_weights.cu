// Attention weight received by each cached key: for key j of a KV head,
//   A_j <- decay * A_j + sum over the chunk's rows i that see j and the group's query heads h of
//          exp(q_ih . k_j / sqrt(d) - lse_ih)
// with the log-sum-exp of the attention itself, so K is read once and nothing is normalised here.
// Every key has exactly one writer, and sums run in a fixed order: no atomics.
//
// weights_rows_kernel (chunks of few rows, decode): HBM-bound on K. One warp per (key unit, KV
// head) walks 16-key pages through a 4-slot cp.async ring (12 warps per SM); K is the A operand
// of mma.sync m16n8k16 and the chunk's rows x heads its columns, so a key's sum is a sum along
// the accumulator's row: one register per key and two shuffles a page.
//
// 24 rows of ~1100 keys, 40 / 8 heads x 128: 15.3 us, 3.7 TB/s (11.1 with K still in L2); FP8 13.2 us.
//
// weights_tc_kernel (longer chunks): S^T = K Q^T on tcgen05. An item is a 256-key tile of one
// (sequence, KV head); the tile stays in shared memory while 128-row query tiles of every head of
// the group stream past it, each used for both halves (at 128 keys an item the query tiles' way from L2
// was 6.7 TB/s). The transposed product gives each of the 128 threads of a warpgroup one key: it
// reads its row of S from TMEM, adds exp2(s c - lse_column) over the columns, and keeps the key's sum
// in a register for the whole item; no score leaves the SM.
//
// Each half has two accumulators, a warpgroup for each, and a warp that issues its products: one
// issuing warp for all spent 1000 cycles a tile on waits and issue where the product takes 512.
// 4 chunks of ~1960 rows after 0 - 4032 keys, 32 / 8 heads x 128: 213 us, 903 TFLOP/s (FP8 227, with the
// expansion of K; 0 - 6048 keys through a window of 1024: 138). A key's sum is off by 2e-7 of itself: four
// float32 sums and ex2.approx (2^-22) for each of thousands of weights. Bound by the epilogue: without its sums 138 us, without the exponentials alone 170 (they are one per score, 32 a
// cycle and SM, as many cycles as the product). Masks are decided for a warp's 32 keys by 32 rows:
// all seen, none, or by element, which costs twice as much (218 us when decided by tile).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "attn_common.cuh"
#include "common.cuh"
#include "pdl.cuh"
#include "rows_common.cuh"
#include "serving.h"
#include "tc_common.cuh"

namespace skv {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------- few rows

constexpr int RW = kWeightWarps;  // warps per CTA, one CTA per SM
constexpr int RSTAGES = 4;  // ring slots per warp

template <int D, bool FP8>
struct Rp {
  static constexpr int KBYTES = kPageSize * D * (FP8 ? 1 : 2);
  static constexpr int STAGE = KBYTES + 2 * kPageSize * 4;  // K, the page's scores, its scales
  static constexpr int SMEM = RW * RSTAGES * STAGE;
};

// NT: columns in groups of 8 (rows x heads of a chunk, at most 8 NT).
template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(RW * 32, 1) weights_rows_kernel(const WeightsArgs a,
                                                                  const __grid_constant__ InlineInts inl,
                                                                  const bf16* __restrict__ kpool,
                                                                  const uint8_t* __restrict__ k8,
                                                                  const float* __restrict__ kscale, int num_units,
                                                                  float scale_log2) {
  using S = Rp<D, FP8>;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int* const lists = list_base(a.lists, inl);
  const int *units = lists + a.o_units, *cu = lists + a.o_cu, *ctx = lists + a.o_ctx;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = smem + (size_t)warp * RSTAGES * S::STAGE;
  const int G = a.n_q / a.n_kv;
  const long long total = (long long)num_units * a.n_kv;
  const long long gw = (long long)warp * gridDim.x + blockIdx.x, nw = (long long)gridDim.x * RW;
  constexpr int RB = D * (FP8 ? 1 : 2), CH = RB / 16;  // bytes and 16-byte chunks of a key
  // chunks XOR-swizzled so that 8 rows of one chunk fall into 8 bank groups (rows of 64 bytes
  // come in pairs per 128)
  auto swz = [](int row, int ch) { return row * RB + ((ch ^ (RB >= 128 ? (row & 7) : ((row >> 1) & 3))) << 4); };

  struct Geo {
    int s, kvh, k0, k1, p0, npages;
  };
  auto geo = [&](long long v) {
    Geo g;
    const int u = (int)(v / a.n_kv);
    g.kvh = (int)(v - (long long)u * a.n_kv);
    g.s = units[3 * u];
    g.k0 = units[3 * u + 1];
    g.k1 = g.k0 + units[3 * u + 2];
    g.p0 = g.k0 / kPageSize;
    g.npages = (g.k1 + kPageSize - 1) / kPageSize - g.p0;
    return g;
  };
  const bool accumulate = a.decay != 0.f;
  long long lv = gw;
  int lp = 0, lslot = 0;
  Geo lg;
  if (lv < total) lg = geo(lv);
  auto issue = [&]() {
    if (lv < total) {
      unsigned char* st = ring + lslot * S::STAGE;
      const int page = a.bt[(size_t)lg.s * a.max_pages + lg.p0 + lp];
      const bool ok = page >= 0 && page < a.num_pages;
      const size_t blk = ok ? (size_t)page * a.n_kv + lg.kvh : 0;
      const unsigned char* src = (FP8 ? reinterpret_cast<const unsigned char*>(k8)
                                      : reinterpret_cast<const unsigned char*>(kpool)) + blk * S::KBYTES;
#pragma unroll
      for (int c = lane; c < kPageSize * CH; c += 32)
        cp_async16(smem_u32(st + swz(c / CH, c % CH)), src + c * 16, ok ? 16 : 0);
      if (lane < 4 && accumulate)
        cp_async16(smem_u32(st + S::KBYTES + lane * 16), a.scores + blk * kPageSize + lane * 4, ok ? 16 : 0);
      if (FP8 && lane >= 4 && lane < 8)
        cp_async16(smem_u32(st + S::KBYTES + lane * 16), kscale + blk * kPageSize + (lane - 4) * 4, ok ? 16 : 0);
      if (++lslot == RSTAGES) lslot = 0;
      if (++lp == lg.npages) {
        lp = 0;
        lv += nw;
        if (lv < total) lg = geo(lv);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < RSTAGES - 1; ++i) issue();

  const int g0 = lane >> 2, qd = lane & 3;
  uint32_t qf[NT][D / 16][2];
  float qback[NT][2];  // FP8: what undoes the power of two of a column's q
  float lse2[NT][2];
  int qpos[NT][2];
  long long cv = gw;
  int cp = 0, cslot = 0;
  Geo cg;
  if (cv < total) cg = geo(cv);
  while (cv < total) {
    issue();
    cp_async_wait<RSTAGES - 1>();
    __syncwarp();
    const unsigned char* st = ring + cslot * S::STAGE;
    if (cp == 0) {
      // the chunk's rows x heads as B columns (column c: row c / G, head c % G of the group), read
      // once per unit; columns past them weigh nothing
      const int seq0 = cu[cg.s], M = (cu[cg.s + 1] - seq0) * G, c0 = ctx[cg.s];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int cb = t * 8 + g0;
        const bool in = cb < M;
        const bf16* src = a.q + (size_t)(seq0 + (in ? cb / G : 0)) * a.ldq + (cg.kvh * G + (in ? cb % G : 0)) * D;
        if (FP8) {  // f16, dims 16 ks + 4 qd .. + 3: the order in which K's codes arrive
          float back;
          load_q_f16<D, false>(src, in, qd, qf[t], back);
#pragma unroll
          for (int e = 0; e < 2; ++e) qback[t][e] = __shfl_sync(0xffffffffu, back, (2 * qd + e) * 4);
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[t][ks][0] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 2 * qd) : 0u;
            qf[t][ks][1] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + 2 * qd) : 0u;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = t * 8 + 2 * qd + e;
          const bool on = col < M;
          lse2[t][e] = on ? a.lse[(size_t)(cg.kvh * G + col % G) * a.ldl + seq0 + col / G] * kLog2e : INFINITY;
          qpos[t][e] = on ? c0 + col / G : -1;
        }
      }
    }
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
    if (FP8) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ks += 2) {
        uint32_t r[4];  // keys 0-7 and 8-15 of chunk ks, then of chunk ks + 1
        ldmatrix_x4(smem_u32(st + swz(krow, ks + (lane >> 4))), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ka[4];
          ka[0] = f16x2_from_e4m3x2(r[2 * h] & 0xffffu);
          ka[1] = f16x2_from_e4m3x2(r[2 * h + 1] & 0xffffu);
          ka[2] = f16x2_from_e4m3x2(r[2 * h] >> 16);
          ka[3] = f16x2_from_e4m3x2(r[2 * h + 1] >> 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16_16816(s[t], ka, qf[t][ks + h]);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t ka[4];
        ldmatrix_x4(smem_u32(st + swz(krow, ks * 2 + (lane >> 4))), ka[0], ka[1], ka[2], ka[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_bf16_16816(s[t], ka, qf[t][ks]);
      }
    }
    const float* old = reinterpret_cast<const float*>(st + S::KBYTES);
    const int key0 = (cg.p0 + cp) * kPageSize;
    float sum[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key = key0 + g0 + 8 * half;
      const float c = FP8 ? scale_log2 * old[kPageSize + g0 + 8 * half] : scale_log2;
      float w = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w += attn_visible(key, qpos[t][e], a.window, a.sinks)
                   ? exp2f(fmaf(s[t][2 * half + e], FP8 ? c * qback[t][e] : c, -lse2[t][e])) : 0.f;
      w += __shfl_xor_sync(0xffffffffu, w, 1);
      w += __shfl_xor_sync(0xffffffffu, w, 2);
      sum[half] = w;
    }
    const int page = a.bt[(size_t)cg.s * a.max_pages + cg.p0 + cp];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, kStatusBadPage);
    } else if (qd == 0) {
      float* dst = a.scores + ((size_t)page * a.n_kv + cg.kvh) * kPageSize;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = g0 + 8 * half, key = key0 + row;
        if (key >= cg.k0 && key < cg.k1) dst[row] = accumulate ? fmaf(a.decay, old[row], sum[half]) : sum[half];
      }
    }
    __syncwarp();
    if (++cslot == RSTAGES) cslot = 0;
    if (++cp == cg.npages) {
      cp = 0;
      cv += nw;
      if (cv < total) cg = geo(cv);
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------- tcgen05

using namespace tc;

constexpr int BK = 128;        // keys per half of an item: an item is kWeightTile = 2 BK keys
constexpr int BQ = 128;        // query rows per tile
constexpr int QST = 4;         // query tiles in flight
constexpr int SBUF = 2;        // S accumulators of a half (128 TMEM columns each)
constexpr int TMEM_COLS = 2 * SBUF * BQ;
constexpr int EPI0 = 4;        // warp 0 loads Q, 1 and 2 issue a half's products, 3 loads K; then a warpgroup
constexpr int WT = 32 * EPI0 + 2 * SBUF * 128;  // for each accumulator

struct WCtrl {
  uint64_t k_full[2], k_empty[2], q_full[QST], q_empty[QST], s_full[2][SBUF], s_empty[2][SBUF], fin;
  uint32_t tmem_base;
  int abort;
  int pend_k[2], pend_q[QST];
  alignas(16) float lse[2 * SBUF][2][BQ];  // [warpgroup][parity], read 16 bytes at a time
  float comb[2][2][BK];                    // the second warpgroups' sums: [item parity][half]
};

template <int D>
constexpr int w_smem() {
  return 1024 + 2 * BK * D * 2 + QST * BQ * D * 2 + (int)sizeof(WCtrl);
}

// d[0 .. 1] = (x0, x1) * c + (l0, l1) and acc[0 .. 1] += (p0, p1), each one packed fp32 instruction.
__device__ __forceinline__ void fma2(float* d, uint32_t x0, uint32_t x1, float c, float l0, float l1) {
  asm("{\n .reg .b64 a, b, e, f;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 e, {%5, %6};\n"
      " fma.rn.f32x2 f, a, b, e;\n mov.b64 {%0, %1}, f;\n}\n"
      : "=f"(d[0]), "=f"(d[1])
      : "r"(x0), "r"(x1), "f"(c), "f"(l0), "f"(l1));
}
__device__ __forceinline__ void add2(float* acc, float p0, float p1) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(acc[0]), "+f"(acc[1])
      : "f"(p0), "f"(p1));
}

struct WItem {
  int s, kvh, key0, seq0, n, c0, nk, qt0, qt1;
  bool sink;
};
__device__ __forceinline__ bool w_item(long long it, const int* __restrict__ tiles, long long n_items, const WeightsArgs& a,
                                       WItem& I) {
  const int Gd = gridDim.x, c = blockIdx.x;
  const long long w = it * Gd + ((it & 1) ? (Gd - 1 - c) : c);
  if (w >= n_items) return false;
  const int t = (int)(w / a.n_kv);
  I.kvh = (int)(w - (long long)t * a.n_kv);
  I.s = tiles[2 * t];
  I.key0 = tiles[2 * t + 1] * kWeightTile;
  const int *cu = a.lists + a.o_cu, *ctx = a.lists + a.o_ctx;
  I.seq0 = cu[I.s];
  I.n = cu[I.s + 1] - I.seq0;
  I.c0 = ctx[I.s];
  I.nk = I.c0 + I.n;
  // rows that see some key of the tile
  const int lo = max(0, I.key0 - I.c0);
  long long hi = I.n;
  I.sink = a.window > 0 && I.key0 < a.sinks;
  if (a.window > 0 && !I.sink) hi = min(hi, (long long)I.key0 + kWeightTile - 1 + a.window - I.c0);
  I.qt0 = lo / BQ;
  I.qt1 = hi > lo ? (int)((hi + BQ - 1) / BQ) : I.qt0;
  return true;
}

template <int D>
__global__ void __launch_bounds__(WT, 1) weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                           const __grid_constant__ CUtensorMap tmK,
                                                           const __grid_constant__ WeightsArgs a,
                                                           const float* __restrict__ kscale,
                                                           const int* __restrict__ bt_k, int pages_k,
                                                           const int* __restrict__ tiles, long long n_items,
                                                           float scale_log2) {
  constexpr int HALVES = D / 64;
  constexpr int HALF = BK * 128;            // bytes of 128 rows x 64 dims
  constexpr int TILE = HALVES * HALF;
  constexpr uint32_t IDESC = make_idesc(BK, BQ, false, false);
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sK = smem_u32(smem), sQ = sK + 2 * TILE;
  WCtrl* ctl = reinterpret_cast<WCtrl*>(smem + (2 + QST) * TILE);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_q / a.n_kv;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ctl->k_full[i]), 1);
      mbar_init(bar(ctl->k_empty[i]), 1);
      ctl->pend_k[i] = -1;
      for (int j = 0; j < SBUF; ++j) {
        mbar_init(bar(ctl->s_full[i][j]), 1);
        mbar_init(bar(ctl->s_empty[i][j]), 128);
      }
    }
    for (int i = 0; i < QST; ++i) {
      mbar_init(bar(ctl->q_full[i]), 1);
      mbar_init(bar(ctl->q_empty[i]), 2);
      ctl->pend_q[i] = -1;
    }
    mbar_init(bar(ctl->fin), 2);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  WItem I;
  griddep_wait();  // launched as a dependent of the kernel before it

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      unsigned g = 0;  // query tiles so far (only remainders and low quotient bits are used)
      for (long long it = 0; ok && w_item(it, tiles, n_items, a, I); ++it) {
        for (int qt = I.qt0; ok && qt < I.qt1; ++qt)
          for (int h = 0; h < G; ++h, ++g) {
            const int st = (int)(g % QST);
            const uint32_t ph = (uint32_t)((g / QST) & 1);
            if (!mbar_wait_ready(bar(ctl->q_empty[st]), ph ^ 1, abort_flag)) {
              ok = false;
              break;
            }
            mbar_expect_tx(bar(ctl->q_full[st]), TILE);
            ctl->pend_q[st] = (int)ph;
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
              tma_load_2d(sQ + st * TILE + hf * HALF, &tmQ, (I.kvh * G + h) * D + hf * 64, I.seq0 + qt * BQ,
                          bar(ctl->q_full[st]));
          }
      }
    }
  } else if (warp == 3) {  // a lane a page
    bool ok = true;
    for (long long it = 0; ok && w_item(it, tiles, n_items, a, I); ++it) {
      const int key = I.key0 + lane * kPageSize;
      // pages without a key that some row sees are not read
      const bool need = lane < kWeightTile / kPageSize && key < I.nk &&
                        (key + kPageSize > window_begin(I.c0, a.window) || key < a.sinks);
      const int page = need ? bt_k[(size_t)I.s * a.max_pages + (key >> 4)] : -1;
      const int row = page >= 0 && page < pages_k ? (page * a.n_kv + I.kvh) * kPageSize
                                                  : pages_k * a.n_kv * kPageSize;  // past the end: zeros
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && mbar_wait_ready(bar(ctl->k_empty[half]), (uint32_t)(it & 1) ^ 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) {
          mbar_expect_tx(bar(ctl->k_full[half]), TILE);
          ctl->pend_k[half] = (int)(it & 1);
        }
        __syncwarp();
        const int p = lane - half * (BK / kPageSize);
        if (p >= 0 && p < BK / kPageSize) {
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf)
            tma_load_2d(sK + half * TILE + hf * HALF + p * 2048, &tmK, hf * 64, row, bar(ctl->k_full[half]));
        }
        __syncwarp();
      }
    }
  } else if (warp < EPI0) {  // the products of half w: the whole warp waits, one lane issues
    const int w = warp - 1;
    // descriptors of this half's keys and of the first Q stage; an offset in bytes adds its sixteenth
    const uint64_t k0 = sdesc(sK + w * TILE), q0 = sdesc(sQ);
    bool ok = true;
    unsigned g = 0;  // query tiles so far
    for (long long it = 0; ok && w_item(it, tiles, n_items, a, I); ++it) {
      const int tiles_here = (I.qt1 - I.qt0) * G;
      const uint32_t kph = (uint32_t)(it & 1);
      if (!(ok = __all_sync(0xffffffffu, mbar_wait_ready(bar(ctl->k_full[w]), kph, abort_flag)))) break;
      if (lane == 0) ctl->pend_k[w] = -1;
      for (int t = 0; t < tiles_here; ++t, ++g) {
        const int st = (int)(g % QST), sb = (int)(g % SBUF);
        const uint32_t b0 = bar(ctl->s_empty[w][sb]), b1 = bar(ctl->q_full[st]), p0 = (g / SBUF & 1) ^ 1, p1 = g / QST & 1;
        const bool free = mbar_test_wait(b0, p0), loaded = mbar_test_wait(b1, p1);  // both tests in flight
        ok = (free || mbar_wait(b0, p0, abort_flag)) && (loaded || mbar_wait(b1, p1, abort_flag));
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        if (elect_lane()) {
          ctl->pend_q[st] = -1;
          const uint32_t d = tmem + (w * SBUF + sb) * BQ;
          const uint64_t q = q0 + st * (TILE / 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int off = ((kk >> 2) * HALF + (kk & 3) * 32) / 16;
            tc_mma(d, k0 + off, q + off, IDESC, kk != 0);
          }
          tc_commit(bar(ctl->s_full[w][sb]));
          tc_commit(bar(ctl->q_empty[st]));
          if (t + 1 == tiles_here) tc_commit(bar(ctl->k_empty[w]));
        }
        __syncwarp();
      }
      if (tiles_here == 0 && lane == 0) mbar_arrive(bar(ctl->k_empty[w]));  // nothing sees the keys
    }
  } else {
    static_assert(SBUF == 2, "");
    // this warpgroup's half of the keys, and the parity of its tiles
    const int wg = (warp - EPI0) >> 2, half = wg >> 1, sb = wg & 1;
    const int quarter = warp & 3;  // the TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t s_addr = tmem + ((uint32_t)(quarter * 32) << 16) + wg * BQ;
    auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    unsigned g = 0;  // query tiles so far
    bool ok = true;
    for (long long it = 0; w_item(it, tiles, n_items, a, I); ++it) {
      // this thread's key: whether some row sees it (the first one's window reaches back furthest),
      // and the score's scale
      const int key0 = I.key0 + half * BK, key = key0 + r;
      const bool seen = key < I.nk && (key >= window_begin(I.c0, a.window) || key < a.sinks);
      float c = scale_log2;
      if (kscale && seen) {
        const int page = bt_k[(size_t)I.s * a.max_pages + (key >> 4)];
        c *= page >= 0 && page < pages_k ? kscale[((size_t)page * a.n_kv + I.kvh) * kPageSize + (key & 15)] : 0.f;
      }
      const int tiles_here = (I.qt1 - I.qt0) * G;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      int t = (int)((sb + g) & 1), qt = I.qt0, h = t;  // the rows and head of the next tile
      auto settle = [&]() {
        while (h >= G) {
          h -= G;
          ++qt;
        }
      };
      settle();
      auto lse_here = [&]() -> float {  // of this thread's column, negated, in log2
        const int row = qt * BQ + r;
        return qt < I.qt1 && row < I.n ? -a.lse[(size_t)(I.kvh * G + h) * a.ldl + I.seq0 + row] * kLog2e : -INFINITY;
      };
      float next = lse_here();
      for (; t < tiles_here; t += 2) {
        const unsigned turn = (g + t) >> 1;  // of this warpgroup
        float* lse = ctl->lse[wg][turn & 1];
        lse[r] = next;
        wg_sync();  // written; and everyone has left the buffer of two turns ago
        const int q0 = qt * BQ;
        h += 2;
        settle();
        next = lse_here();
        // after an expired wait the loops run on without work, so that every thread still meets
        // the same barriers
        ok = ok && mbar_wait_ready(bar(ctl->s_full[half][sb]), turn & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        // no key of the tile hidden from any row, and no row past the chunk
        const bool interior = key0 + BK - 1 <= I.c0 + q0 && q0 + BQ <= I.n &&
                              (a.window <= 0 || key0 > I.c0 + q0 + BQ - 1 - a.window || key0 + BK <= a.sinks);
        // columns of this tile whose rows see the key: [lo, hi)
        const int lo = max(0, key - I.c0 - q0);
        long long last = min(BQ, I.n - q0);
        if (a.window > 0 && key >= a.sinks) last = min(last, (long long)key + a.window - I.c0 - q0);
        const int hi = (int)max(last, 0LL);
        // two groups of 32 columns in registers; a group is loaded as soon as one has been summed,
        // so that the accumulator is free when half of it has been
        uint32_t v[2][32];
        tmem_ld32_async(s_addr, v[0]);
        tmem_ld32_async(s_addr + 32, v[1]);
#pragma unroll
        for (int cb = 0; cb < BQ; cb += 32) {
          uint32_t* x = v[(cb / 32) & 1];
          if (cb % 64 == 0) {
            tmem_wait32(v[0]);
            tmem_wait32(v[1]);
            if (cb == 64) {
              tc_fence_before();
              mbar_arrive(bar(ctl->s_empty[half][sb]));  // S has been read: the accumulator may be refilled
            }
          }
          // whether every key of the warp is seen by every row of these columns, or none by any
          const bool all = interior || __all_sync(0xffffffffu, lo <= cb && cb + 32 <= hi);
          if (all) {
            float e[32];  // two columns an instruction, all exponents before the exponentials
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse + cb + i);
              fma2(e + i, x[i], x[i + 1], c, l.x, l.y);
              fma2(e + i + 2, x[i + 2], x[i + 3], c, l.z, l.w);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) e[i] = ex2_approx(e[i]);
#pragma unroll
            for (int i = 0; i < 32; i += 2) add2(acc + (i & 3), e[i], e[i + 1]);
          } else if (__any_sync(0xffffffffu, lo < cb + 32 && cb < hi)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float e = fmaf(__uint_as_float(x[i]), c, lse[cb + i]);
              acc[i & 3] += ex2_approx(cb + i >= lo && cb + i < hi ? e : -INFINITY);
            }
          }
          if (cb < 64) tmem_ld32_async(s_addr + cb + 64, x);
        }
      }
      g += tiles_here;
      float w = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      float* other = &ctl->comb[it & 1][half][r];
      if (sb == 1) *other = w;
      asm volatile("bar.sync %0, 256;" ::"r"(5 + half) : "memory");
      if (sb == 0 && ok && seen) {
        w += *other;
        const int own = a.bt[(size_t)I.s * a.max_pages + (key >> 4)];
        if (own >= 0 && own < a.num_pages) {
          float* dst = a.scores + ((size_t)own * a.n_kv + I.kvh) * kPageSize + (key & 15);
          *dst = a.decay != 0.f ? fmaf(a.decay, *dst, w) : w;
        } else {
          atomicOr(a.status, kStatusBadPage);
        }
      }
    }
  }

  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      atomicOr(a.status, kStatusTimeout);
      for (int i = 0; i < 2 + QST; ++i) {
        const int ph = i < 2 ? ctl->pend_k[i] : ctl->pend_q[i - 2];
        if (ph < 0) continue;
        const uint32_t b = i < 2 ? bar(ctl->k_full[i]) : bar(ctl->q_full[i - 2]);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(b, (uint32_t)ph) && global_ns() - t0 < kTimeoutNs) {
        }
      }
    }
    if ((warp == 1 || warp == 2) && elect_lane()) {  // products in flight
      tc_commit(bar(ctl->fin));
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(bar(ctl->fin), 0) && global_ns() - t0 < kTimeoutNs) {
      }
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

template <int D, bool FP8, int NT>
cudaError_t rows_launch(const WeightsArgs& a, const InlineInts& inl, const bf16* k, const uint8_t* k8, const float* ks,
                        int num_units, int num_sms, cudaStream_t s) {
  constexpr int smem = Rp<D, FP8>::SMEM;
  static_assert(smem <= 227 * 1024, "rings must fit in shared memory");
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(weights_rows_kernel<D, FP8, NT>), smem, once);
  if (e != cudaSuccess) return e;
  const long long total = (long long)num_units * a.n_kv;
  const int ctas = (int)(total < num_sms ? total : num_sms);
  return launch_pdl(weights_rows_kernel<D, FP8, NT>, dim3(ctas), dim3(RW * 32), smem, s, a, inl, k, k8, ks, num_units,
                    kLog2e / sqrtf((float)D));
}

template <int D, bool FP8>
cudaError_t rows_cols(const WeightsArgs& a, const InlineInts& inl, const bf16* k, const uint8_t* k8, const float* ks,
                      int max_cols, int num_units, int num_sms, cudaStream_t s) {
  if (max_cols <= 8) return rows_launch<D, FP8, 1>(a, inl, k, k8, ks, num_units, num_sms, s);
  if (max_cols <= 16) return rows_launch<D, FP8, 2>(a, inl, k, k8, ks, num_units, num_sms, s);
  return rows_launch<D, FP8, 4>(a, inl, k, k8, ks, num_units, num_sms, s);
}

template <int D>
cudaError_t tc_launch(const WeightsArgs& a, const bf16* k, const float* ks, const int* bt_k, int pages_k,
                      const int* tiles, int num_tiles, int num_sms, cudaStream_t s) {
  CUtensorMap mq, mk;
  if (!tma_map_bf16_2d(&mq, a.q, a.T, a.n_q * D, a.ldq, 64, BQ, true) ||
      !tma_map_bf16_2d(&mk, k, pages_k * a.n_kv * kPageSize, D, D, 64, kPageSize, true))
    return cudaErrorNotSupported;
  constexpr int smem = w_smem<D>();
  static_assert(smem <= 227 * 1024, "shared memory");
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(weights_tc_kernel<D>), smem, once);
  if (e != cudaSuccess) return e;
  const long long n_items = (long long)num_tiles * a.n_kv;
  return launch_pdl(weights_tc_kernel<D>, dim3((unsigned)(n_items < num_sms ? n_items : num_sms)), dim3(WT), smem, s, mq, mk,
                    a, ks, bt_k, pages_k, tiles, n_items, kLog2e / sqrtf((float)D));
}

}  // namespace

cudaError_t launch_weights_rows(const WeightsArgs& a, const InlineInts& inl, const bf16* k, const uint8_t* k8,
                                const float* ks, int d_head, int max_cols, int num_units, int num_sms, cudaStream_t s) {
  if (max_cols > kWeightCols) return cudaErrorNotSupported;
  if (d_head == 128)
    return k8 ? rows_cols<128, true>(a, inl, k, k8, ks, max_cols, num_units, num_sms, s)
              : rows_cols<128, false>(a, inl, k, k8, ks, max_cols, num_units, num_sms, s);
  if (d_head == 64)
    return k8 ? rows_cols<64, true>(a, inl, k, k8, ks, max_cols, num_units, num_sms, s)
              : rows_cols<64, false>(a, inl, k, k8, ks, max_cols, num_units, num_sms, s);
  return cudaErrorNotSupported;
}

cudaError_t launch_weights_tc(const WeightsArgs& a, const bf16* k, const float* ks, const int* bt_k, int pages_k,
                              int d_head, const int* tiles, int num_tiles, int num_sms, cudaStream_t s) {
  if (d_head == 128) return tc_launch<128>(a, k, ks, bt_k, pages_k, tiles, num_tiles, num_sms, s);
  if (d_head == 64) return tc_launch<64>(a, k, ks, bt_k, pages_k, tiles, num_tiles, num_sms, s);
  return cudaErrorNotSupported;
}

}  // namespace skv
