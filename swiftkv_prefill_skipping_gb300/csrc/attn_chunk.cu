// Attention of prompt chunks over the paged cache on tcgen05 (swiftkv_attend's tiles): causal, with
// an optional window and sinks, the log-sum-exp of every row, d_head 64 or 128.
//
// Work item: two 128-row query tiles that share every key block. With an even number of query heads
// per KV head (head_pairs) they are the same rows of two heads of one KV head; otherwise rows
// [256 p, 256 p + 128) and the next 128 of one head (the second absent past the chunk's end). The
// blocks of an item are those of the sinks and those from its first row's window to its last row's
// position, one ascending list of which tile A needs a prefix. Persistent: one CTA per SM walks its
// share of the items, heaviest first, alternate rounds reversed.
//
// A block is 128 keys. Per tile and block: S = Q K^T (tensor memory, 128 columns), softmax, P over S
// as bf16, O += P V. Both tiles' S and O fill the 512 columns of tensor memory exactly, so a tile's
// S has one buffer, and the tiles take turns: while the softmax warps of one work (one thread per
// row), the tensor core runs the other's two products. Against 64-key blocks with two S buffers
// (attention_tc2.cu) that halves the number of hand-overs between tensor core and softmax, whose
// latency is what bounds that kernel. P is rounded once to bf16
// (at most 2^-8 of a weight and so 2^-8 of sum p |v| in the output, which is itself rounded to bf16
// with 2^-8 of its value); a second product with the remainders would add half of the tensor work.
// Row sums use the unrounded weights, in float32.
//
// 12 warps: 0 TMA, 1 and 2 the tiles' MMAs, 3 idle, 4-7 and 8-11 softmax of tile A and B with the
// registers that the first four give up. All mbarrier waits are bounded; when one expires the CTA
// flags kStatusTimeout, drains its copies and MMAs, frees tensor memory and exits.
//
// Pages without a visible key are not loaded (zeros instead), and pages of V that the chunk sees in
// part come from zero-padded copies (launch_v_tail). FP8: K and V are an expansion to bf16 codes;
// the block's 128 key and value scales travel with V, scores take the key's and P the value's.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "serving.h"
#include "tc_common.cuh"

namespace skv {

namespace {

using namespace tc;

constexpr int BQ = 128;                // query rows per tile
constexpr int BKV = 128;               // keys per block
constexpr int PAGES = BKV / kPageSize;
constexpr int ST = 2;                  // K and V stages
constexpr int THREADS = 384;
constexpr int REGS_ISSUE = 72, REGS_SOFTMAX = 216;  // 72 + 2 x 216 = 3 x 168, the registers at launch
constexpr int O_COL = 256;             // tensor memory: S_A 0, S_B 128, O_A 256, O_B 384
constexpr float kLag = 8.f;            // log2 headroom of the running maximum
constexpr float kLn2 = 0.69314718055994531f;

struct Ctrl {
  uint64_t q_full, q_empty, k_full[ST], k_empty[ST], v_full[ST], v_empty[ST];
  uint64_t s_full[2], p_full[2], pv_done[2], o_empty[2], fin[2];
  uint32_t tmem_base;
  int abort;
  int pend[1 + 2 * ST];                // phases of copies in flight: Q, K stages, V stages
  alignas(16) float scale[ST][2][BKV];  // FP8: key scales, value scales
};

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = 128 * 128;          // 128 rows x 64 dims
  static constexpr int TILE = HALVES * HALF;      // Q tile, K block or V block
  static constexpr int SMEM = 1024 + (2 + 2 * ST) * TILE + (int)sizeof(Ctrl);
  static constexpr uint32_t IDESC_S = make_idesc(BQ, BKV, false, false);  // Q (K-major) x K (K-major)
  static constexpr uint32_t IDESC_O = make_idesc(BQ, D, false, true);     // P (tensor memory) x V (MN-major)
};

struct Item {
  int s, h, hb, seq0, n, c0, nk, q0a, q0b, nblk_a, nblk_b, nblk, nsink, nwin;
  bool has_b;
  // first key of list entry j
  __device__ __forceinline__ int key0(int j) const { return (j < nsink ? j : nwin + j - nsink) * BKV; }
};

__device__ __forceinline__ bool item_at(int it, const ChunkArgs& a, Item& I) {
  const int G = gridDim.x, c = blockIdx.x;
  const long long w = (long long)it * G + ((it & 1) ? (G - 1 - c) : c);
  if (w >= a.num_items) return false;
  const int per = a.head_pairs ? a.n_q / 2 : a.n_q;
  const int tile = a.tiles[w / per], k = (int)(w % per);
  I.s = tile >> 16;
  const int qp = tile & 0xffff;
  I.seq0 = a.cu[I.s];
  I.n = a.cu[I.s + 1] - I.seq0;
  I.c0 = a.ctx[I.s];
  I.nk = I.c0 + I.n;
  if (a.head_pairs) {
    I.h = 2 * k;
    I.hb = 2 * k + 1;
    I.q0a = I.q0b = qp * BQ;
    I.has_b = true;
  } else {
    I.h = I.hb = k;
    I.q0a = qp * 2 * BQ;
    I.q0b = I.q0a + BQ;
    I.has_b = I.q0b < I.n;
  }
  const int end_a = (min(I.nk, I.c0 + I.q0a + BQ) + BKV - 1) / BKV;
  const int end_b = I.has_b ? (min(I.nk, I.c0 + I.q0b + BQ) + BKV - 1) / BKV : 0;
  const int end = I.has_b ? end_b : end_a, w0 = window_begin(I.c0 + I.q0a, a.window);
  I.nsink = w0 > 0 ? min(end, (min(a.sinks, w0) + BKV - 1) / BKV) : 0;
  I.nwin = max(I.nsink, w0 / BKV);
  auto entries = [&](int last) { return min(I.nsink, last) + max(0, last - I.nwin); };
  I.nblk_a = entries(end_a);
  I.nblk_b = entries(end_b);
  I.nblk = I.has_b ? I.nblk_b : I.nblk_a;
  return true;
}

// d[0 .. 1] = x[0 .. 1] * c + m and acc[0 .. 1] += p[0 .. 1], each one packed fp32 instruction
__device__ __forceinline__ void fma2(float* d, const float* x, float c, float m) {
  asm("{\n .reg .b64 a, b, e, f;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 e, {%5, %5};\n"
      " fma.rn.f32x2 f, a, b, e;\n mov.b64 {%0, %1}, f;\n}\n"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(x[0]), "f"(x[1]), "f"(c), "f"(m));
}
__device__ __forceinline__ void add2(float* acc, const float* p) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n add.rn.f32x2 a, a, b;\n"
      " mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(acc[0]), "+f"(acc[1])
      : "f"(p[0]), "f"(p[1]));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) attn_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                const __grid_constant__ CUtensorMap tmK,
                                                                const __grid_constant__ CUtensorMap tmV,
                                                                const __grid_constant__ CUtensorMap tmTail,
                                                                const __grid_constant__ ChunkArgs a, float scale_log2) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sQ = smem_u32(smem), sK = sQ + 2 * C::TILE, sV = sK + ST * C::TILE;
  Ctrl* ctl = reinterpret_cast<Ctrl*>(smem + (2 + 2 * ST) * C::TILE);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool fp8 = a.k_scale != nullptr;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };

  if (threadIdx.x == 0) {
    mbar_init(bar(ctl->q_full), 1);
    mbar_init(bar(ctl->q_empty), 2);
    for (int i = 0; i < ST; ++i) {
      mbar_init(bar(ctl->k_full[i]), 1);
      mbar_init(bar(ctl->v_full[i]), 1);
      mbar_init(bar(ctl->k_empty[i]), 2);
      mbar_init(bar(ctl->v_empty[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(ctl->s_full[t]), 1);
      mbar_init(bar(ctl->p_full[t]), 128);
      mbar_init(bar(ctl->pv_done[t]), 1);
      mbar_init(bar(ctl->o_empty[t]), 128);
      mbar_init(bar(ctl->fin[t]), 1);
    }
    for (int i = 0; i < 1 + 2 * ST; ++i) ctl->pend[i] = -1;
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  Item I;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
    if (warp == 0 && lane == 0) {
      const int group = a.n_q / a.n_kv, none = a.num_pages * a.n_kv * kPageSize;  // rows past the pool: zeros
      int kv_i = 0;
      bool ok = true;
      for (int it = 0; ok && item_at(it, a, I); ++it) {
        const int kvh = I.h / group;
        if (it > 0 && !mbar_wait(bar(ctl->q_empty), (uint32_t)((it - 1) & 1), abort_flag)) break;
        mbar_expect_tx(bar(ctl->q_full), (I.has_b ? 2 : 1) * C::TILE);
        ctl->pend[0] = it & 1;
        for (int t = 0; t < (I.has_b ? 2 : 1); ++t)
#pragma unroll
          for (int hf = 0; hf < C::HALVES; ++hf)
            tma_load_2d(sQ + t * C::TILE + hf * C::HALF, &tmQ, (t ? I.hb : I.h) * D + hf * 64,
                        I.seq0 + (t ? I.q0b : I.q0a), bar(ctl->q_full));
        const TailPages tail = tail_pages(I.c0, I.n, a.window, a.sinks);
        const int w0 = window_begin(I.c0 + I.q0a, a.window);
        for (int j = 0; ok && j < I.nblk; ++j, ++kv_i) {
          const int st = kv_i % ST;
          const uint32_t ph = (uint32_t)((kv_i / ST) & 1);
          const int key0 = I.key0(j);
          int row[PAGES];
#pragma unroll
          for (int p = 0; p < PAGES; ++p) {
            const int key = key0 + p * kPageSize;
            row[p] = none;
            if (key < I.nk && (key + kPageSize > w0 || key < a.sinks)) {
              const int page = a.bt[(size_t)I.s * a.max_pages + (key >> 4)];
              if (page >= 0 && page < a.num_pages) row[p] = (page * a.n_kv + kvh) * kPageSize;
              else atomicOr(a.status, kStatusBadPage);
            }
          }
          if (!(ok = mbar_wait(bar(ctl->k_empty[st]), ph ^ 1, abort_flag))) break;
          mbar_expect_tx(bar(ctl->k_full[st]), C::TILE);
          ctl->pend[1 + st] = (int)ph;
#pragma unroll
          for (int p = 0; p < PAGES; ++p)
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_2d(sK + st * C::TILE + hf * C::HALF + p * 2048, &tmK, hf * 64, row[p], bar(ctl->k_full[st]));
          if (!(ok = mbar_wait(bar(ctl->v_empty[st]), ph ^ 1, abort_flag))) break;
          mbar_expect_tx(bar(ctl->v_full[st]), C::TILE + (fp8 ? 2 * BKV * 4 : 0));
          ctl->pend[1 + ST + st] = (int)ph;
#pragma unroll
          for (int p = 0; p < PAGES; ++p) {
            const CUtensorMap* map = &tmV;
            int vrow = row[p];
            if (a.v_tail && vrow != none) {
              const int pidx = key0 / kPageSize + p;
#pragma unroll
              for (int t = 0; t < kTailSlots; ++t)
                if (pidx == tail.page[t]) {
                  map = &tmTail;
                  vrow = ((I.s * kTailSlots + t) * a.n_kv + kvh) * kPageSize;
                }
            }
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_2d(sV + st * C::TILE + hf * C::HALF + p * 2048, map, hf * 64, vrow, bar(ctl->v_full[st]));
            if (fp8) {  // page 0's scales for a page that is not loaded: its keys are masked
              const size_t sr = row[p] != none ? (size_t)row[p] : (size_t)kvh * kPageSize;
              const uint32_t dst = smem_u32(&ctl->scale[st][0][p * kPageSize]);
              bulk_load(dst, a.k_scale + sr, kPageSize * 4, bar(ctl->v_full[st]));
              bulk_load(dst + BKV * 4, a.v_scale + sr, kPageSize * 4, bar(ctl->v_full[st]));
            }
          }
        }
      }
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // tile t's MMAs; g counts its blocks over all items, oi the items that used its O
      const int t = warp - 1;
      int kv_base = 0, g = 0, oi = 0;
      bool ok = true;
      for (int it = 0; ok && item_at(it, a, I); ++it) {
        const int nb = t ? I.nblk_b : I.nblk_a;
        if (!mbar_wait(bar(ctl->q_full), (uint32_t)(it & 1), abort_flag)) break;
        ctl->pend[0] = -1;
        if (nb == 0) mbar_arrive(bar(ctl->q_empty));
        for (int j = 0; ok && j < I.nblk; ++j) {
          const int kv = kv_base + j, st = kv % ST;
          const uint32_t ph = (uint32_t)((kv / ST) & 1);
          if (!(ok = mbar_wait(bar(ctl->k_full[st]), ph, abort_flag))) break;
          ctl->pend[1 + st] = -1;
          if (j >= nb) {  // a block this tile does not read: only release it, once it has arrived
            mbar_arrive(bar(ctl->k_empty[st]));
            if (!(ok = mbar_wait(bar(ctl->v_full[st]), ph, abort_flag))) break;
            ctl->pend[1 + ST + st] = -1;
            mbar_arrive(bar(ctl->v_empty[st]));
            continue;
          }
          // the buffer holds P of the previous block until the product that reads it has completed
          if (g > 0 && !(ok = mbar_wait(bar(ctl->pv_done[t]), (uint32_t)((g - 1) & 1), abort_flag))) break;
          tc_fence_after();
          const uint32_t k = sK + st * C::TILE, q = sQ + t * C::TILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::HALF + (kk & 3) * 32;
            tc_mma(tmem + t * BKV, sdesc(q + off), sdesc(k + off), C::IDESC_S, kk != 0);
          }
          tc_commit(bar(ctl->s_full[t]));
          tc_commit(bar(ctl->k_empty[st]));
          if (j + 1 == nb) tc_commit(bar(ctl->q_empty));
          if (!(ok = mbar_wait(bar(ctl->v_full[st]), ph, abort_flag))) break;
          ctl->pend[1 + ST + st] = -1;
          if (!(ok = mbar_wait(bar(ctl->p_full[t]), (uint32_t)(g & 1), abort_flag))) break;
          // the first P V of an item overwrites O: the previous item's output must have left
          if (j == 0 && oi > 0 && !(ok = mbar_wait(bar(ctl->o_empty[t]), (uint32_t)((oi - 1) & 1), abort_flag))) break;
          tc_fence_after();
          const uint32_t v = sV + st * C::TILE;
#pragma unroll
          for (int kk = 0; kk < BKV / 16; ++kk)  // 16 keys: 8 columns of P, 2 KB of each 64-dim half of V
            tc_mma_ts(tmem + O_COL + t * 128, tmem + t * BKV + kk * 8, sdesc_sw128(v + kk * 2048, C::HALF, 1024),
                      C::IDESC_O, (j | kk) != 0);
          tc_commit(bar(ctl->pv_done[t]));
          tc_commit(bar(ctl->v_empty[st]));
          ++g;
        }
        kv_base += I.nblk;
        if (nb > 0) ++oi;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + t * BKV, o_addr = tmem + lane_off + O_COL + t * 128;
    int g = 0, kvb = 0;
    bool ok = true;
    for (int it = 0; ok && item_at(it, a, I); kvb += I.nblk, ++it) {
      const int nb = t ? I.nblk_b : I.nblk_a, q0 = t ? I.q0b : I.q0a;
      if (nb == 0) continue;
      const int qrow = q0 + r, qpos = I.c0 + qrow;
      const int first = window_begin(qpos, a.window), last = min(qpos, I.nk - 1), sinks = a.window > 0 ? a.sinks : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j, ++g) {
        // a warp leaves as one: what follows is collective
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(ctl->s_full[t]), (uint32_t)(g & 1), abort_flag)))) break;
        tc_fence_after();
        float x[BKV];
        {
          uint32_t v[BKV / 32][32];
#pragma unroll
          for (int c = 0; c < BKV / 32; ++c) tmem_ld32_async(s_addr + 32 * c, v[c]);
#pragma unroll
          for (int c = 0; c < BKV / 32; ++c) {
            tmem_wait32(v[c]);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[32 * c + i] = __uint_as_float(v[c][i]);
          }
        }
        const float* scales = nullptr;
        if (fp8) {
          const int kv = kvb + j, st = kv % ST;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(ctl->v_full[st]), (uint32_t)((kv / ST) & 1), abort_flag))))
            break;
          scales = ctl->scale[st][0];
#pragma unroll
          for (int i = 0; i < BKV; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + i);
            x[i] *= f.x;
            x[i + 1] *= f.y;
            x[i + 2] *= f.z;
            x[i + 3] *= f.w;
          }
        }
        const int key0 = I.key0(j);
        // no key of the block hidden from any row of the tile
        const bool inside = key0 + BKV - 1 <= I.c0 + q0 && key0 + BKV <= I.nk &&
                            (a.window <= 0 || key0 > I.c0 + q0 + BQ - 1 - a.window || key0 + BKV <= a.sinks);
        if (!inside) {  // the row's visible keys as bits, 32 at a time
#pragma unroll
          for (int c = 0; c < BKV / 32; ++c) {
            const int b = key0 + 32 * c;
            auto upto = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };  // the first n bits
            const uint32_t in = upto(last + 1 - b) & (~upto(first - b) | upto(sinks - b));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(in >> i & 1u)) x[32 * c + i] = -INFINITY;
          }
        }
        float mx;
        {
          float pm[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v = fmax3f(x[k], x[k + 8], x[k + 16]);
#pragma unroll
            for (int e = 24; e < BKV; e += 16) v = fmax3f(v, x[k + e], e + 8 < BKV ? x[k + e + 8] : x[k + e]);
            pm[k] = v;
          }
          mx = fmax3f(fmax3f(pm[0], pm[1], pm[2]), fmax3f(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * scale_log2;
        }
        const bool move = mx > m + kLag;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? mx : m;
          const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
          if (j > 0) {  // O holds the blocks before: S of this one was issued after their last product
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(o_addr + c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= f;
              tmem_st32(o_addr + c, v);
            }
          }
          l *= f;
          m = mn;
        }
        const float mneg = m == -INFINITY ? 0.f : -m;  // a row that has seen nothing yet: P = 0
#pragma unroll
        for (int i = 0; i < BKV; i += 2) fma2(x + i, x + i, scale_log2, mneg);
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll
        for (int i = 0; i < BKV; i += 2) {
          x[i] = ex2_approx(x[i]);
          x[i + 1] = ex2_approx(x[i + 1]);
          add2(sum + (i & 7), x + i);
        }
        l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
        if (fp8) {
#pragma unroll
          for (int i = 0; i < BKV; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + BKV + i);
            x[i] *= f.x;
            x[i + 1] *= f.y;
            x[i + 2] *= f.z;
            x[i + 3] *= f.w;
          }
        }
        uint32_t p[BKV / 2];
#pragma unroll
        for (int i = 0; i < BKV / 2; ++i) p[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        tmem_st64(s_addr, p);
        tc_fence_before();
        mbar_arrive(bar(ctl->p_full[t]));
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(ctl->pv_done[t]), (uint32_t)((g - 1) & 1), abort_flag));
      if (ok) {
        tc_fence_after();
        const float inv = 1.f / l;
        const int head = t ? I.hb : I.h;
        if (a.lse && qrow < I.n) a.lse[(size_t)head * a.ldl + I.seq0 + qrow] = (m + log2f(l)) * kLn2;
        bf16* dst = a.out + (size_t)(I.seq0 + min(qrow, I.n - 1)) * a.ldo + (size_t)head * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(o_addr + c, v);
          if (qrow < I.n) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 u;
              u.x = pack_bf16(v[e] * inv, v[e + 1] * inv);
              u.y = pack_bf16(v[e + 2] * inv, v[e + 3] * inv);
              u.z = pack_bf16(v[e + 4] * inv, v[e + 5] * inv);
              u.w = pack_bf16(v[e + 6] * inv, v[e + 7] * inv);
              *reinterpret_cast<uint4*>(dst + c + e) = u;
            }
          }
        }
        tc_fence_before();
        mbar_arrive(bar(ctl->o_empty[t]));
      }
    }
  }

  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      atomicOr(a.status, kStatusTimeout);
      for (int i = 0; i < 1 + 2 * ST; ++i) {
        const int ph = ctl->pend[i];
        if (ph < 0) continue;
        const uint32_t b = i == 0 ? bar(ctl->q_full) : i <= ST ? bar(ctl->k_full[i - 1]) : bar(ctl->v_full[i - 1 - ST]);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(b, (uint32_t)ph) && global_ns() - t0 < kTimeoutNs) {
        }
      }
    }
    if (threadIdx.x == 32 || threadIdx.x == 64) {  // MMAs each issuing thread has in flight
      const uint32_t f = bar(ctl->fin[threadIdx.x == 64]);
      tc_commit(f);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(f, 0) && global_ns() - t0 < kTimeoutNs) {
      }
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D>
cudaError_t launch_d(const ChunkArgs& a, const bf16* q, int ldq, int T, const bf16* k, const bf16* v, int num_sms,
                     cudaStream_t s) {
  using C = Cfg<D>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  CUtensorMap mq, mk, mv, mt;
  const int rows = a.num_pages * a.n_kv * kPageSize;
  if (!tma_map_bf16_2d(&mq, q, T, a.n_q * D, ldq, 64, BQ, true) ||
      !tma_map_bf16_2d(&mk, k, rows, D, D, 64, kPageSize, true) || !tma_map_bf16_2d(&mv, v, rows, D, D, 64, kPageSize, true))
    return cudaErrorNotSupported;
  mt = mv;
  if (a.v_tail &&
      !tma_map_bf16_2d(&mt, a.v_tail, a.tail_seqs * kTailSlots * a.n_kv * kPageSize, D, D, 64, kPageSize, true))
    return cudaErrorNotSupported;
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_chunk_kernel<D>), C::SMEM, once);
  if (e != cudaSuccess) return e;
  attn_chunk_kernel<D><<<(int)(a.num_items < num_sms ? a.num_items : num_sms), THREADS, C::SMEM, s>>>(
      mq, mk, mv, mt, a, 1.4426950408889634f / sqrtf((float)D));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_chunk(const ChunkArgs& a, const bf16* q, int ldq, int T, const bf16* k, const bf16* v, int d_head,
                              int num_sms, cudaStream_t s) {
  if (a.num_items <= 0) return cudaSuccess;
  if (a.head_pairs && (a.n_q / a.n_kv) % 2) return cudaErrorNotSupported;
  if (!a.k_scale != !a.v_scale) return cudaErrorNotSupported;
  if (d_head == 128) return launch_d<128>(a, q, ldq, T, k, v, num_sms, s);
  if (d_head == 64) return launch_d<64>(a, q, ldq, T, k, v, num_sms, s);
  return cudaErrorNotSupported;
}

}  // namespace skv
