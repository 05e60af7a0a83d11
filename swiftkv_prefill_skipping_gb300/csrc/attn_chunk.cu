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
// A block is 80 keys at d_head 128 and 128 keys at 64: per tile, tensor memory then holds the scores S
// of one block, the weights P of another (bf16, two a column) and O, and both tiles fill its 512
// columns almost exactly. Because P does not lie over S, S of the next block is issued as soon as
// the softmax warps have read this block's into registers, and the softmax of one block runs while the
// tensor core computes the scores of the next and O += P V of the one before. With P over S
// (128-key blocks) each of the three hand-overs between tensor core and softmax, some 500 cycles, stood
// in a tile's chain: 691 us for 4 x ~1960 rows after 0 - 6048 keys and 32 heads, 605 of them with
// the softmax left out. P is rounded once to bf16
// (at most 2^-8 of a weight and so 2^-8 of sum p |v| in the output, which is itself rounded to bf16
// with 2^-8 of its value); a second product with the remainders would add half of the tensor work.
// Row sums use the unrounded weights, in float32.
//
// 12 warps: 0 loads Q and K and 3 loads V by TMA, each with the page ids of a block read one block
// ahead; 1 and 2 issue the tiles' MMAs (the warp converged, one elected lane); 4-7 and 8-11 are the
// softmax of tile A and B, one thread per row, with the registers that the first four give up. All
// mbarrier waits are bounded; when one expires the CTA flags kStatusTimeout, drains its copies and
// MMAs, frees tensor memory and exits.
//
// The softmax computes P against the running maximum as it is. Only where a row has none yet, or where
// its sum of a block passes 2^16, does a warp look for the block's own maximum, before it computes P
// (again): seeking it in every block stood in the chain with 370 of its 2400 cycles. Exponentials, sums and
// the rounding of P go four columns at a time, and FP8 is a template parameter, so that no branch
// parts them (436 us with all three undone).
//
// 4 chunks of ~1960 rows after 0 - 6048 keys, 32 / 8 heads x 128: 361 us, 1.42 PFLOP/s (392 called without
// a pause, where the power cap lowers the clock); the same rows through a window of 1024 and 4 sinks:
// 150 us. Those scores are nearly flat; with q 16 times as large, where sums outgrow the running maximum
// more often, 454 us. FP8: 547 and 207 us, of which the expansion to bf16 is the difference. Bound by the tensor core and the hand-overs to it: 337 us
// without any softmax. S of an 80-key block reads 6.5 KB of shared memory per 16 dims, 52 cycles
// where the product takes 40, and a wider block does not fit beside P and O: with that the products
// alone take 307 us. Measured and not kept: four softmax warpgroups on alternate 64-key blocks with P
// over S (504 us, where this form took 434: S waits for the product of two blocks before); two threads a
// row, half of a block's columns each (509).
//
// Pages without a visible key are not loaded (zeros instead), and pages of V that the chunk sees in
// part come from zero-padded copies (launch_v_tail). FP8: K and V are an expansion to bf16 codes;
// the block's key and value scales travel with V, scores take the key's and P the value's (times
// kValueShift).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "pdl.cuh"
#include "serving.h"
#include "tc_common.cuh"

namespace skv {

namespace {

using namespace tc;

constexpr int BQ = 128;                // query rows per tile
constexpr int THREADS = 384;
constexpr int REGS_ISSUE = 72, REGS_SOFTMAX = 216;  // 72 + 2 x 216 = 3 x 168, the registers at launch
constexpr float kGrown = 65536.f;      // a block's row sum from which the running maximum is moved
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int BKV = D == 128 ? 80 : 128;  // keys per block
  static constexpr int PAGES = BKV / kPageSize;
  static constexpr int KST = 3, VST = 3;           // K and V stages
  static constexpr int HALVES = D / 64;
  static constexpr int Q_HALF = BQ * 128, KV_HALF = BKV * 128;  // rows x 64 dims
  static constexpr int Q_TILE = HALVES * Q_HALF, KV_TILE = HALVES * KV_HALF;
  // tensor memory columns of a tile: S, P (half as many), O
  static constexpr int COLS = 256, P_COL = BKV, O_COL = COLS - D;
  static_assert(P_COL + BKV / 2 <= O_COL && BKV % 16 == 0, "two tiles in 512 columns");
  static constexpr uint32_t IDESC_S = make_idesc(BQ, BKV, false, false);  // Q (K-major) x K (K-major)
  static constexpr uint32_t IDESC_O = make_idesc(BQ, D, false, true);     // P (tensor memory) x V (MN-major)
};

template <int D>
struct Ctrl {
  using C = Cfg<D>;
  uint64_t q_full, q_empty, k_full[C::KST], k_empty[C::KST], v_full[C::VST], v_empty[C::VST];
  uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2], o_empty[2], fin[2];
  uint32_t tmem_base;
  int abort;
  int pend[1 + C::KST + C::VST];                  // phases of copies in flight: Q, K stages, V stages
  alignas(16) float scale[C::VST][2][C::BKV];      // FP8: key scales, value scales
};
template <int D>
constexpr int smem_bytes() {
  return 1024 + 2 * Cfg<D>::Q_TILE + (Cfg<D>::KST + Cfg<D>::VST) * Cfg<D>::KV_TILE + (int)sizeof(Ctrl<D>);
}

struct Item {
  int s, h, hb, seq0, n, c0, nk, q0a, q0b, nblk_a, nblk_b, nblk, nsink, nwin;
  bool has_b;
  // block of list entry j
  __device__ __forceinline__ int block(int j) const { return j < nsink ? j : nwin + j - nsink; }
};

template <int BKV>
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

// 16 columns of this thread's tensor-memory lane; a load's registers hold values after tmem_wait16
__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                 "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_row(uint32_t addr, float* x) {
#pragma unroll
  for (int c = 0; c < N; c += 16) tmem_ld16_async(addr + c, x + c);
#pragma unroll
  for (int c = 0; c < N; c += 16) tmem_wait16(x + c);
}
// N (a multiple of 8) 32-bit columns, complete on return
template <int N>
__device__ __forceinline__ void tmem_st_row(uint32_t addr, const uint32_t* r) {
#pragma unroll
  for (int c = 0; c < N; c += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(addr + c), "r"(r[c]),
                 "r"(r[c + 1]), "r"(r[c + 2]), "r"(r[c + 3]), "r"(r[c + 4]), "r"(r[c + 5]), "r"(r[c + 6]), "r"(r[c + 7])
                 : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
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

template <int D, bool FP8>
__global__ void __launch_bounds__(THREADS, 1) attn_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                const __grid_constant__ CUtensorMap tmK,
                                                                const __grid_constant__ CUtensorMap tmV,
                                                                const __grid_constant__ CUtensorMap tmTail,
                                                                const __grid_constant__ ChunkArgs a, float scale_log2) {
  using C = Cfg<D>;
  constexpr int BKV = C::BKV, PAGES = C::PAGES, KST = C::KST, VST = C::VST;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t sQ = smem_u32(smem), sK = sQ + 2 * C::Q_TILE, sV = sK + KST * C::KV_TILE;
  Ctrl<D>* ctl = reinterpret_cast<Ctrl<D>*>(smem + 2 * C::Q_TILE + (KST + VST) * C::KV_TILE);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  // a warp leaves a wait as one: what follows is collective
  auto wait_all = [&](uint32_t b, uint32_t phase) { return __all_sync(0xffffffffu, mbar_wait_ready(b, phase, abort_flag)) != 0; };

  if (threadIdx.x == 0) {
    mbar_init(bar(ctl->q_full), 1);
    mbar_init(bar(ctl->q_empty), 2);
    for (int i = 0; i < KST; ++i) {
      mbar_init(bar(ctl->k_full[i]), 1);
      mbar_init(bar(ctl->k_empty[i]), 2);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(bar(ctl->v_full[i]), 1);
      mbar_init(bar(ctl->v_empty[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(ctl->s_full[t]), 1);
      mbar_init(bar(ctl->s_empty[t]), 128);
      mbar_init(bar(ctl->p_full[t]), 128);
      mbar_init(bar(ctl->pv_done[t]), 1);
      mbar_init(bar(ctl->o_empty[t]), 128);
      mbar_init(bar(ctl->fin[t]), 1);
    }
    for (int i = 0; i < 1 + KST + VST; ++i) ctl->pend[i] = -1;
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
  griddep_wait();  // launched as a dependent of the kernel that writes the tail copies (or the expansion)

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
    if (warp == 0 || warp == 3) {
      // warp 0: Q and K, warp 3: V and the scales. Lane p looks after page p of a block (one thread
      // doing it for all pages, at a dependent instruction every few cycles, took longer than the block)
      const bool is_v = warp == 3;
      const int group = a.n_q / a.n_kv;
      // the lane's page id in block j of item X, loaded one block ahead of its use
      auto load_page = [&](const Item& X, int j) {
        const int key = X.block(j) * BKV + lane * kPageSize;
        // not read where no row of the item sees a key of the page
        const bool need = lane < PAGES && key < X.nk && (key + kPageSize > window_begin(X.c0 + X.q0a, a.window) || key < a.sinks);
        return make_int2(need, need ? a.bt[(size_t)X.s * a.max_pages + (key >> 4)] : 0);
      };
      int kv_i = 0;
      int2 pg = make_int2(0, 0);
      bool ok = true, have = item_at<BKV>(0, a, I);
      if (have) pg = load_page(I, 0);
      for (int it = 0; ok && have; ++it) {
        Item N;
        const bool have_next = item_at<BKV>(it + 1, a, N);
        const int kvh = I.h / group;
        const TailPages tail = tail_pages(I.c0, I.n, a.window, a.sinks);
        if (!is_v) {
          // Q overwrites the previous item's, once its last S has completed
          if (it > 0 && !(ok = wait_all(bar(ctl->q_empty), (uint32_t)((it - 1) & 1)))) break;
          if (lane == 0) {
            mbar_expect_tx(bar(ctl->q_full), (I.has_b ? 2 : 1) * C::Q_TILE);
            ctl->pend[0] = it & 1;
            for (int t = 0; t < (I.has_b ? 2 : 1); ++t)
#pragma unroll
              for (int hf = 0; hf < C::HALVES; ++hf)
                tma_load_2d(sQ + t * C::Q_TILE + hf * C::Q_HALF, &tmQ, (t ? I.hb : I.h) * D + hf * 64,
                            I.seq0 + (t ? I.q0b : I.q0a), bar(ctl->q_full));
          }
        }
        for (int j = 0; j < I.nblk; ++j, ++kv_i) {
          int2 next = pg;
          if (j + 1 < I.nblk) next = load_page(I, j + 1);
          else if (have_next) next = load_page(N, 0);
          const int st = is_v ? kv_i % VST : kv_i % KST;
          const uint32_t ph = (uint32_t)((is_v ? kv_i / VST : kv_i / KST) & 1);
          const uint32_t full = is_v ? bar(ctl->v_full[st]) : bar(ctl->k_full[st]);
          // a page that is not needed, or outside the pool, reads rows past the pool's end: zeros
          const bool valid = pg.x && pg.y >= 0 && pg.y < a.num_pages;
          if (pg.x && !valid) atomicOr(a.status, kStatusBadPage);
          int row = (valid ? pg.y * a.n_kv + kvh : a.num_pages * a.n_kv) * kPageSize;
          const CUtensorMap* map = is_v ? &tmV : &tmK;
          const size_t sr = valid ? (size_t)row : (size_t)kvh * kPageSize;  // scales of a masked page: page 0's
          if (is_v && a.v_tail && valid) {
            const int pidx = I.block(j) * PAGES + lane;
#pragma unroll
            for (int t = 0; t < kTailSlots; ++t)
              if (pidx == tail.page[t]) {
                map = &tmTail;
                row = ((I.s * kTailSlots + t) * a.n_kv + kvh) * kPageSize;
              }
          }
          if (!(ok = wait_all(is_v ? bar(ctl->v_empty[st]) : bar(ctl->k_empty[st]), ph ^ 1))) break;
          if (lane == 0) {
            mbar_expect_tx(full, C::KV_TILE + (is_v && FP8 ? 2 * BKV * 4 : 0));
            ctl->pend[is_v ? 1 + KST + st : 1 + st] = (int)ph;
          }
          __syncwarp();
          if (lane < PAGES) {
            const uint32_t dst = (is_v ? sV : sK) + st * C::KV_TILE + lane * 2048;
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf) tma_load_2d(dst + hf * C::KV_HALF, map, hf * 64, row, full);
            if (is_v && FP8) {
              const uint32_t sd = smem_u32(&ctl->scale[st][0][lane * kPageSize]);
              bulk_load(sd, a.k_scale + sr, kPageSize * 4, full);
              bulk_load(sd + BKV * 4, a.v_scale + sr, kPageSize * 4, full);
            }
          }
          pg = next;
        }
        I = N;
        have = have_next;
      }
    } else {
      // tile t's MMAs, the warp waiting as one and one lane issuing; g counts its blocks over all items, oi
      // the items that used its O
      const int t = warp - 1;
      // descriptors of the tile's Q and of stage 0; an offset in bytes adds its sixteenth
      const uint64_t q = sdesc(sQ + t * C::Q_TILE), k0 = sdesc(sK), v0 = sdesc_sw128(sV, C::KV_HALF, 1024);
      const uint32_t base = tmem + t * C::COLS;
      int kv_base = 0, g = 0, oi = 0;
      bool ok = true;
      for (int it = 0; ok && item_at<BKV>(it, a, I); ++it) {
        const int nb = t ? I.nblk_b : I.nblk_a;
        if (!(ok = wait_all(bar(ctl->q_full), (uint32_t)(it & 1)))) break;
        if (lane == 0) {
          ctl->pend[0] = -1;
          if (nb == 0) mbar_arrive(bar(ctl->q_empty));
        }
        // two phases, both tests in flight
        auto wait2 = [&](uint64_t& b0, uint32_t p0, uint64_t& b1, uint32_t p1) {
          const bool r0 = mbar_test_wait(bar(b0), p0), r1 = mbar_test_wait(bar(b1), p1);
          const bool done = (r0 || mbar_wait(bar(b0), p0, abort_flag)) && (r1 || mbar_wait(bar(b1), p1, abort_flag));
          return __all_sync(0xffffffffu, done) != 0;
        };
        // S of block j of the item, the tile's block g + j: the softmax has read the one before it
        auto issue_s = [&](int j) -> bool {
          const int kv = kv_base + j, st = kv % KST, gj = g + j;
          // s_empty's phase before its first is complete from the start
          if (!wait2(ctl->k_full[st], (uint32_t)((kv / KST) & 1), ctl->s_empty[t], (uint32_t)((gj - 1) & 1))) return false;
          tc_fence_after();
          if (elect_lane()) {
            ctl->pend[1 + st] = -1;
            const uint64_t k = k0 + st * (C::KV_TILE / 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma(base, q + ((kk >> 2) * C::Q_HALF + (kk & 3) * 32) / 16,
                     k + ((kk >> 2) * C::KV_HALF + (kk & 3) * 32) / 16, C::IDESC_S, kk != 0);
            tc_commit(bar(ctl->s_full[t]));
            tc_commit(bar(ctl->k_empty[st]));
            if (j + 1 == nb) tc_commit(bar(ctl->q_empty));
          }
          __syncwarp();
          return true;
        };
        auto issue_pv = [&](int j) -> bool {
          const int kv = kv_base + j, st = kv % VST;
          if (!wait2(ctl->v_full[st], (uint32_t)((kv / VST) & 1), ctl->p_full[t], (uint32_t)((g + j) & 1))) return false;
          // the first P V of an item overwrites O: the previous item's output must have left
          if (j == 0 && oi > 0 && !wait_all(bar(ctl->o_empty[t]), (uint32_t)((oi - 1) & 1))) return false;
          tc_fence_after();
          if (elect_lane()) {
            ctl->pend[1 + KST + st] = -1;
            const uint64_t v = v0 + st * (C::KV_TILE / 16);
#pragma unroll
            for (int kk = 0; kk < BKV / 16; ++kk)  // 16 keys: 8 columns of P, 2 KB of each 64-dim half of V
              tc_mma_ts(base + C::O_COL, base + C::P_COL + kk * 8, v + kk * 128, C::IDESC_O, (j | kk) != 0);
            tc_commit(bar(ctl->pv_done[t]));
            tc_commit(bar(ctl->v_empty[st]));
          }
          __syncwarp();
          return true;
        };
        if (nb > 0) ok = issue_s(0);
        for (int j = 0; ok && j < nb; ++j) {
          if (j + 1 < nb && !(ok = issue_s(j + 1))) break;
          ok = issue_pv(j);
        }
        // blocks this tile does not read: only released, once they have arrived
        for (int j = nb; ok && j < I.nblk; ++j) {
          const int kv = kv_base + j, ks = kv % KST, vs = kv % VST;
          if (!(ok = wait2(ctl->k_full[ks], (uint32_t)((kv / KST) & 1), ctl->v_full[vs], (uint32_t)((kv / VST) & 1)))) break;
          if (lane == 0) {
            ctl->pend[1 + ks] = -1;
            mbar_arrive(bar(ctl->k_empty[ks]));
            ctl->pend[1 + KST + vs] = -1;
            mbar_arrive(bar(ctl->v_empty[vs]));
          }
        }
        kv_base += I.nblk;
        g += nb;
        if (nb > 0) ++oi;
      }
    }
  } else {
    // (216 registers; 12 to 116 bytes of them spill, at d_head 64 most)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t s_addr = tmem + ((uint32_t)(quarter * 32) << 16) + t * C::COLS;
    int g = 0, kvb = 0;
    bool ok = true;
    auto wait = [&](uint64_t& b, uint32_t phase) { return wait_all(bar(b), phase); };
    for (int it = 0; ok && item_at<BKV>(it, a, I); kvb += I.nblk, ++it) {
      const int nb = t ? I.nblk_b : I.nblk_a, q0 = t ? I.q0b : I.q0a;
      if (nb == 0) continue;
      // rows past the chunk see what its last row sees
      const int qw = q0 + quarter * 32, qrow = qw + lane, qpos = I.c0 + min(qrow, I.n - 1);
      const int first = window_begin(qpos, a.window), last = min(qpos, I.nk - 1), sinks = a.window > 0 ? a.sinks : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j, ++g) {
        if (!(ok = wait(ctl->s_full[t], (uint32_t)(g & 1)))) break;
        tc_fence_after();
        float x[BKV];
        tmem_ld_row<BKV>(s_addr, x);
        tc_fence_before();
        mbar_arrive(bar(ctl->s_empty[t]));  // S of the next block may be computed
        const float* scales = nullptr;
        if (FP8) {
          const int kv = kvb + j, st = kv % VST;
          if (!(ok = wait(ctl->v_full[st], (uint32_t)((kv / VST) & 1)))) break;
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
        const int key0 = I.block(j) * BKV;
        // no key of the block hidden from any row of the warp
        const bool inside = key0 + BKV - 1 <= I.c0 + qw && key0 + BKV <= I.nk &&
                            (a.window <= 0 || key0 > I.c0 + qw + 31 - a.window || key0 + BKV <= a.sinks);
        if (!inside) {  // the row's visible keys as bits, 16 at a time
#pragma unroll
          for (int c = 0; c < BKV / 16; ++c) {
            const int b = key0 + 16 * c;
            auto upto = [](int n) { return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1; };  // the first n bits
            const uint32_t in = upto(last + 1 - b) & (~upto(first - b) | upto(sinks - b));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!(in >> i & 1u)) x[16 * c + i] = -INFINITY;
          }
        }
        // P against the running maximum as it is. The block's own maximum is sought only for rows that have
        // none yet (the first block), or, with P computed again, where a row's sum has outgrown the old
        // one: seeking it every time costs 40 us of 400.
        uint32_t p[BKV / 2];
        float add, f = 1.f;
        bool seek = __any_sync(0xffffffffu, m == -INFINITY), any = false;
#pragma unroll 1
        while (true) {
          if (seek) {
            float pm[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float v = x[k];
#pragma unroll
              for (int e = 8; e + 8 < BKV; e += 16) v = fmax3f(v, x[k + e], x[k + e + 8]);
              pm[k] = BKV % 16 ? v : fmaxf(v, x[k + BKV - 8]);
            }
            const float mx = fmax3f(fmax3f(pm[0], pm[1], pm[2]), fmax3f(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * scale_log2;
            const bool move = mx > m;
            any = __any_sync(0xffffffffu, move);
            if (move) {
              f = m == -INFINITY ? 0.f : ex2_approx(m - mx);
              m = mx;
              l *= f;
            }
          }
          const float mneg = m == -INFINITY ? 0.f : -m;  // a row that has seen nothing yet: P = 0
          float sum[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll
          for (int i = 0; i < BKV; i += 4) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) fma2(e + k, x + i + k, scale_log2, mneg);
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = ex2_approx(e[k]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) add2(sum + ((i + k) & 7), e + k);
            if (FP8) {
              const float4 w = *reinterpret_cast<const float4*>(scales + BKV + i);
              e[0] *= w.x;
              e[1] *= w.y;
              e[2] *= w.z;
              e[3] *= w.w;
            }
            p[i / 2] = pack_bf16(e[0], e[1]);
            p[i / 2 + 1] = pack_bf16(e[2], e[3]);
          }
          add = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
          if (seek || !__any_sync(0xffffffffu, add > kGrown)) break;
          seek = true;
        }
        l += add;
        // P and O belong to the previous block's product until it has completed
        if (g > 0 && !(ok = wait(ctl->pv_done[t], (uint32_t)((g - 1) & 1)))) break;
        tc_fence_after();
        if (any && j > 0) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float v[32];
            tmem_ld32(s_addr + C::O_COL + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= f;
            tmem_st32(s_addr + C::O_COL + c, v);
          }
        }
        tmem_st_row<BKV / 2>(s_addr + C::P_COL, p);
        tc_fence_before();
        mbar_arrive(bar(ctl->p_full[t]));
      }
      if (ok) ok = wait(ctl->pv_done[t], (uint32_t)((g - 1) & 1));
      if (ok) {
        tc_fence_after();
        const float inv = (FP8 ? 1.f / kValueShift : 1.f) / l;
        const int head = t ? I.hb : I.h;
        if (a.lse && qrow < I.n) a.lse[(size_t)head * a.ldl + I.seq0 + qrow] = (m + log2f(l)) * kLn2;
        bf16* dst = a.out + (size_t)(I.seq0 + min(qrow, I.n - 1)) * a.ldo + (size_t)head * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(s_addr + C::O_COL + c, v);
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
      for (int i = 0; i < 1 + KST + VST; ++i) {
        const int ph = ctl->pend[i];
        if (ph < 0) continue;
        const uint32_t b = i == 0 ? bar(ctl->q_full) : i <= KST ? bar(ctl->k_full[i - 1]) : bar(ctl->v_full[i - 1 - KST]);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(b, (uint32_t)ph) && global_ns() - t0 < kTimeoutNs) {
        }
      }
    }
    if ((warp == 1 || warp == 2) && elect_lane()) {  // MMAs each issuing lane has in flight
      const uint32_t f = bar(ctl->fin[warp - 1]);
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

template <int D, bool FP8>
cudaError_t launch_d(const ChunkArgs& a, const bf16* q, int ldq, int T, const bf16* k, const bf16* v, int num_sms,
                     cudaStream_t s) {
  constexpr int smem = smem_bytes<D>();
  static_assert(smem <= 227 * 1024, "shared memory");
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
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_chunk_kernel<D, FP8>), smem, once);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_chunk_kernel<D, FP8>, dim3(a.num_items < num_sms ? a.num_items : num_sms), dim3(THREADS), smem,
                    s, mq, mk, mv, mt, a, 1.4426950408889634f / sqrtf((float)D));
}

}  // namespace

cudaError_t launch_attn_chunk(const ChunkArgs& a, const bf16* q, int ldq, int T, const bf16* k, const bf16* v, int d_head,
                              int num_sms, cudaStream_t s) {
  if (a.num_items <= 0) return cudaSuccess;
  if (a.head_pairs && (a.n_q / a.n_kv) % 2) return cudaErrorNotSupported;
  if (!a.k_scale != !a.v_scale) return cudaErrorNotSupported;
  if (d_head == 128)
    return a.k_scale ? launch_d<128, true>(a, q, ldq, T, k, v, num_sms, s) : launch_d<128, false>(a, q, ldq, T, k, v, num_sms, s);
  if (d_head == 64)
    return a.k_scale ? launch_d<64, true>(a, q, ldq, T, k, v, num_sms, s) : launch_d<64, false>(a, q, ldq, T, k, v, num_sms, s);
  return cudaErrorNotSupported;
}

}  // namespace skv
