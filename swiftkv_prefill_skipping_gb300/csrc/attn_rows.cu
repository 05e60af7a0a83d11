// Attention of single tokens and short chunks over the paged cache, split along the keys
// (swiftkv_attend's rows; window, sinks and the log-sum-exp included).
//
//   o = sum_j exp(z_j - m) v_j / sum_j exp(z_j - m),  z = q . k / sqrt(d),  j over the visible keys
//
// Bound by HBM on K and V: each is read once per item. An item is up to 16 columns, the rows of a
// short chunk times the query heads of one KV head, so that tokens of one sequence share the read.
// Its keys are cut into units, one warp per (unit, KV head) at a time, all warps of the GPU with
// units of about the same length. A warp walks 16-key pages through its own cp.async ring of
// XOR-swizzled tiles that runs ahead across units; nothing is synchronised wider than a warp.
//
// Both products are transposed: S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16, keys or
// dimensions as the 16 rows of A and the columns as the 8 of B. A group of 8 columns then fills an
// instruction; with the heads as rows of A (attention_split.cu) half of every instruction and half
// of the accumulators are padding, and the registers they took let more warps run (8 on a bf16 cache,
// where the rings fill shared memory, 12 on FP8) and hide one another's latency. P^T becomes a B
// operand by one movmatrix per 8 keys. The running maximum may lag behind by 2^8 before O is rescaled,
// so no reduction over the keys is needed while it holds.
//
// P enters P V as two bf16 parts (about 17 bits). FP8: K's codes enter as f16 (exact, times 2^-8) and
// the key's scale multiplies the score in float32, q as f16 under a power of two per column; V's codes enter as bf16 (exact) and the value's
// scale rides on P, P' = 2^16 p s_v, which has float32's range in bf16: keys whose value scales are any
// factor apart keep their bits. (P' in f16 against the largest scale so far lost those far below it.)
// The 2^16, undone at the end, keeps P' above bf16's subnormals for value scales down to float32's;
// scales have to stay below 2^100.
//
// A unit that covers its item writes the output, others (max, sum, unnormalised O) records that
// attn_rows_merge joins, one warp per column.
//
// 24 rows of ~1100 keys, 40 / 8 heads x 128, bf16: 27.4 us, 4.1 TB/s; 16 windows of 4096 keys and 4
// sinks, 32 / 8 heads, FP8: 39.7 us, 3.5 TB/s, and bf16 53 us, 5.0 TB/s. With one or two units a warp the
// rings' start, the last round and the merge (3 us) do not overlap anything. On FP8 no unit is full
// either (2.0 instructions a cycle and SM, 45 % of the ALU, 18 % of the tensor pipe, DRAM 51 %): 12 warps
// do not cover the chain from a page's codes to its weights and back. 167 registers; with 16 columns 60
// bytes spill. 64 rows of 3000 FP8 keys: 94 us, 4.3 TB/s. 4 rows of up to 64 keys: 7.3 us, the launches'
// latency.
#include <cfloat>

#include "common.cuh"
#include "pdl.cuh"
#include "rows_common.cuh"
#include "serving.h"

namespace skv {

namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLag = 8.f;  // log2 headroom of the running maximum

template <int D, bool FP8>
struct Rg {
  static constexpr int RB = D * (FP8 ? 1 : 2);        // bytes of a key's K or V row
  static constexpr int PAGE = kPageSize * RB;
  static constexpr int STAGE = 2 * PAGE + (FP8 ? 2 * kPageSize * 4 : 0) + 16;  // K, V, scales, validity
  static constexpr int WARPS = FP8 ? kRowsWarps8 : kRowsWarps;
  static constexpr int SLOTS = (227 * 1024) / (WARPS * STAGE) < 6 ? (227 * 1024) / (WARPS * STAGE) : 6;
  static constexpr int SMEM = WARPS * SLOTS * STAGE;
  static_assert(SLOTS >= 2 && SMEM <= 227 * 1024, "ring");
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four e4m3 codes as two f16 pairs, each value times 2^-8 (exactly: the exponent fields differ by 8
// and f16's subnormals cover e4m3's): the even and the odd bytes. Cheaper than two conversions and
// the moves that line their inputs up, and part of it runs on the multiply pipe.
constexpr float kCodeScale = 256.f;
__device__ __forceinline__ void unpack4(uint32_t r, uint32_t& even, uint32_t& odd) {
  even = ((r * 128u) & 0x3f803f80u) | ((r * 256u) & 0x80008000u);
  odd = ((r >> 1) & 0x3f803f80u) | (r & 0x80008000u);
}
// The same as two bf16 pairs with the values themselves: the shifted bits are 2^-120 of them, subnormal
// for e4m3's subnormals, and the product (which keeps subnormals) is exact.
__device__ __forceinline__ void unpack4_bf16(uint32_t r, uint32_t& even, uint32_t& odd) {
  uint32_t x[2] = {((r << 4) & 0x07f007f0u) | ((r << 8) & 0x80008000u), ((r >> 4) & 0x07f007f0u) | (r & 0x80008000u)};
  const uint32_t up = 0x7b807b80u;  // 2^120 twice
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), *reinterpret_cast<const __nv_bfloat162*>(&up));
    x[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  even = x[0];
  odd = x[1];
}

// NT: columns in groups of 8.
template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(Rg<D, FP8>::WARPS * 32, 1) attn_rows_kernel(
    const RowsArgs a, const __grid_constant__ InlineInts inl, const unsigned char* __restrict__ kpool,
    const unsigned char* __restrict__ vpool, const float* __restrict__ kscale, const float* __restrict__ vscale,
    float scale_log2) {
  using S = Rg<D, FP8>;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int* const lists = list_base(a.lists, inl);
  const int *items = lists + a.o_items, *units = lists + a.o_units, *ubeg = lists + a.o_ubeg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = smem + (size_t)warp * S::SLOTS * S::STAGE;
  const int G = a.n_q / a.n_kv;
  const long long total = (long long)a.num_units * a.n_kv;
  const long long gw = (long long)warp * gridDim.x + blockIdx.x, nw = (long long)gridDim.x * S::WARPS;
  constexpr int CH = S::RB / 16;
  // 16-byte chunks XOR-swizzled so that 8 rows of one chunk fall into 8 bank groups (64-byte rows
  // come in pairs per 128)
  auto swz = [](int row, int ch) { return row * S::RB + ((ch ^ (S::RB >= 128 ? (row & 7) : ((row >> 1) & 3))) << 4); };

  struct Geo {
    int item, kvh, k0, k1, p0, npages, seq;
  };
  auto geo = [&](long long v) {
    Geo g;
    const int u = (int)(v / a.n_kv);
    g.kvh = (int)(v - (long long)u * a.n_kv);
    g.item = units[3 * u];
    g.k0 = units[3 * u + 1];
    g.k1 = g.k0 + units[3 * u + 2];
    g.seq = items[4 * g.item + 2];
    g.p0 = g.k0 / kPageSize;
    g.npages = (g.k1 + kPageSize - 1) / kPageSize - g.p0;
    return g;
  };
  constexpr int NC = kPageSize * CH / 32;  // 16-byte chunks of a page per lane
  int at[NC];                              // their places in a slot
#pragma unroll
  for (int i = 0; i < NC; ++i) at[i] = swz((lane + 32 * i) / CH, (lane + 32 * i) % CH);
  long long lv = gw;
  int lp = 0, lslot = 0;
  Geo lg;
  if (lv < total) lg = geo(lv);
  auto issue = [&]() {
    if (lv < total) {
      unsigned char* st = ring + lslot * S::STAGE;
      const int page = a.bt[(size_t)lg.seq * a.max_pages + lg.p0 + lp];
      const bool ok = page >= 0 && page < a.num_pages;
      const size_t blk = ok ? (size_t)page * a.n_kv + lg.kvh : 0;
      const int key0 = (lg.p0 + lp) * kPageSize;
      const unsigned char *kp = kpool + blk * S::PAGE + lane * 16, *vp = vpool + blk * S::PAGE + lane * 16;
      const uint32_t to = smem_u32(st);
      if (ok && key0 >= lg.k0 && key0 + kPageSize <= lg.k1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          cp_async16(to + at[i], kp + i * 512, 16);
          cp_async16(to + S::PAGE + at[i], vp + i * 512, 16);
        }
      } else {  // rows outside the unit become zeros
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int key = key0 + (lane + 32 * i) / CH, bytes = ok && key >= lg.k0 && key < lg.k1 ? 16 : 0;
          cp_async16(to + at[i], kp + i * 512, bytes);
          cp_async16(to + S::PAGE + at[i], vp + i * 512, bytes);
        }
      }
      if (FP8 && lane < 8)  // 16 K scales, then 16 V scales
        cp_async16(smem_u32(st + 2 * S::PAGE + lane * 16), (lane < 4 ? kscale : vscale) + blk * kPageSize + (lane & 3) * 4,
                   ok ? 16 : 0);
      if (lane == 0) {
        *reinterpret_cast<int*>(st + S::STAGE - 16) = ok;
        if (!ok) atomicOr(a.status, kStatusBadPage);
      }
      if (++lslot == S::SLOTS) lslot = 0;
      if (++lp == lg.npages) {
        lp = 0;
        lv += nw;
        if (lv < total) lg = geo(lv);
      }
    }
    cp_async_commit();  // possibly empty: keeps the group count uniform
  };
#pragma unroll
  for (int i = 0; i < S::SLOTS - 1; ++i) issue();

  const int g0 = lane >> 2, qd = lane & 3;
  uint32_t qf[NT][D / 16][2];
  float o[NT][D / 16][4];           // O^T: 16 dimensions x 8 columns a tile
  float m[NT][2], l[NT][2];         // of columns 2 qd, 2 qd + 1
  float qback[NT][2];               // FP8: what undoes their q's power of two
  int qpos[NT][2];                  // their positions, -1: no such column
  int row0 = 0, cols = 0, pos_lo = 0, pos_hi = 0;
  long long cv = gw;
  int cp = 0, cslot = 0;
  Geo cg;
  if (cv < total) cg = geo(cv);
  while (cv < total) {
    issue();
    cp_async_wait<S::SLOTS - 1>();
    __syncwarp();
    const unsigned char* st = ring + cslot * S::STAGE;
    if (cp == 0) {  // a new unit: Q as B operands straight from memory, fresh softmax state
      const int* it = items + 4 * cg.item;
      row0 = it[0];
      cols = it[1] * G;
      pos_lo = it[3];
      pos_hi = it[3] + it[1] - 1;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int cb = t * 8 + g0;
        const bool in = cb < cols;
        const bf16* src = a.q + (size_t)(row0 + (in ? cb / G : 0)) * a.ldq + (cg.kvh * G + (in ? cb % G : 0)) * D;
        if (FP8) {  // f16, dims 16 ks + 4 qd + {0, 2} and {1, 3}: the order in which K's codes arrive
          float back;
          load_q_f16<D, true>(src, in, qd, qf[t], back);
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
          qpos[t][e] = col < cols ? pos_lo + col / G : -1;
          m[t][e] = -INFINITY;
          l[t][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
      }
    }

    // S^T = K Q^T: keys g0, g0 + 8 (rows) x columns 2 qd, 2 qd + 1, in two independent chains
    float s[NT][2][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][c][e] = 0.f;
    const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
    if (FP8) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ks += 2) {
        uint32_t r[4];  // keys 0-7 and 8-15 of chunk ks, then of chunk ks + 1
        ldmatrix_x4(smem_u32(st + swz(krow, ks + (lane >> 4))), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ka[4];
          unpack4(r[2 * h], ka[0], ka[2]);
          unpack4(r[2 * h + 1], ka[1], ka[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16_16816(s[t][h], ka, qf[t][ks + h]);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t ka[4];
        ldmatrix_x4(smem_u32(st + swz(krow, ks * 2 + (lane >> 4))), ka[0], ka[1], ka[2], ka[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_bf16_16816(s[t][ks & 1], ka, qf[t][ks]);
      }
    }
    const int key0 = (cg.p0 + cp) * kPageSize;
    const float* sc = reinterpret_cast<const float*>(st + 2 * S::PAGE);  // FP8: 16 key, 16 value scales
    const float c_lo = FP8 ? kCodeScale * scale_log2 * sc[g0] : scale_log2;
    const float c_hi = FP8 ? kCodeScale * scale_log2 * sc[g0 + 8] : scale_log2;
    // every key of the page visible to every column
    const bool inside = *reinterpret_cast<const int*>(st + S::STAGE - 16) && key0 >= cg.k0 && key0 + kPageSize <= cg.k1 &&
                        key0 + kPageSize - 1 <= pos_lo &&
                        (a.window <= 0 || key0 > pos_hi - a.window || key0 + kPageSize <= a.sinks);
    float z[NT][4];  // scaled scores: [0] key g0 col 0, [1] key g0 col 1, [2], [3] key g0 + 8
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[t][e] = (s[t][0][e] + s[t][1][e]) * ((e < 2 ? c_lo : c_hi) * (FP8 ? qback[t][e & 1] : 1.f));
    if (!inside) {
      const bool ok = *reinterpret_cast<const int*>(st + S::STAGE - 16);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + g0 + (e < 2 ? 0 : 8);
          if (!(ok && key >= cg.k0 && key < cg.k1 && attn_visible(key, qpos[t][e & 1], a.window, a.sinks))) z[t][e] = -INFINITY;
        }
    }
    float v_lo = 1.f, v_hi = 1.f;  // FP8: the shifted value scales of keys g0, g0 + 8 (0 outside the unit)
    if (FP8) {
      v_lo = key0 + g0 >= cg.k0 && key0 + g0 < cg.k1 ? kValueShift * sc[kPageSize + g0] : 0.f;
      v_hi = key0 + g0 + 8 >= cg.k0 && key0 + g0 + 8 < cg.k1 ? kValueShift * sc[kPageSize + g0 + 8] : 0.f;
    }
    bool move = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) move |= fmaxf(z[t][e], z[t][e + 2]) > m[t][e] + kLag;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(z[t][e], z[t][e + 2]);
#pragma unroll
          for (int o2 = 4; o2 <= 16; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
          const float mn = mx > m[t][e] + kLag ? mx : m[t][e];
          al[e] = mn == m[t][e] ? 1.f : exp2f(m[t][e] - mn);  // 0 the first time
          m[t][e] = mn;
          l[t][e] *= al[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][i][e] *= al[e & 1];
      }
    }
    // P^T as B operands: rows of 8 keys become columns by a transpose within the warp
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2_approx(z[t][e] - (m[t][e & 1] == -INFINITY ? 0.f : m[t][e & 1]));
      l[t][0] += p[0] + p[2];
      l[t][1] += p[1] + p[3];
      uint32_t h0, l0, h1, l1;
      split_pair_bf16(p[0] * v_lo, p[1] * v_lo, h0, l0);
      split_pair_bf16(p[2] * v_hi, p[3] * v_hi, h1, l1);
      ph[t][0] = transpose8(h0);
      ph[t][1] = transpose8(h1);
      pl[t][0] = transpose8(l0);
      pl[t][1] = transpose8(l1);
    }
    // O^T += V^T P^T. bf16: tile i holds dims 16 i + row. FP8: ldmatrix.trans yields two keys x two
    // neighbouring dims, so rows 0-7 are the even dims of the chunk and rows 8-15 the odd ones
    const unsigned char* vb = st + S::PAGE;
    if (FP8) {
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {
        uint32_t r[4];  // keys 0-7 and 8-15 of chunk c, then of chunk c + 1
        ldmatrix_x4_trans(smem_u32(vb + swz(krow, c + (lane >> 4))), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t va[4];
          unpack4_bf16(r[2 * h], va[0], va[1]);
          unpack4_bf16(r[2 * h + 1], va[2], va[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_bf16_16816(o[t][c + h], va, ph[t]);
            mma_bf16_16816(o[t][c + h], va, pl[t]);
          }
        }
      }
    } else {
      const int vrow = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t va[4];  // (dims 0-7, keys 0-7), (dims 8-15, keys 0-7), (dims 0-7, keys 8-15), ...
        ldmatrix_x4_trans(smem_u32(vb + swz(vrow, i * 2 + ((lane >> 3) & 1))), va[0], va[1], va[2], va[3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma_bf16_16816(o[t][i], va, ph[t]);
          mma_bf16_16816(o[t][i], va, pl[t]);
        }
      }
    }
    __syncwarp();  // the slot is refilled by a later issue()
    if (++cslot == S::SLOTS) cslot = 0;

    if (++cp == cg.npages) {
      const bool whole = ubeg[cg.item + 1] - ubeg[cg.item] == 1;
      const int u = (int)(cv / a.n_kv);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[t][e];
#pragma unroll
          for (int o2 = 4; o2 <= 16; o2 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
          const int col = t * 8 + 2 * qd + e;
          if (col >= cols) continue;
          // dims this thread holds of tile i: bf16 16 i + g0 and + 8; FP8 16 i + 2 g0 and + 1
          if (whole) {
            const int row = row0 + col / G, h = cg.kvh * G + col % G;
            const float f = (FP8 ? 1.f / kValueShift : 1.f) / sum;
            if (a.lse && g0 == 0) a.lse[(size_t)h * a.ldl + row] = (m[t][e] + log2f(sum)) * kLn2;
            bf16* dst = a.out + (size_t)row * a.ldo + (size_t)h * D;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              if (FP8) {
                *reinterpret_cast<uint32_t*>(dst + 16 * i + 2 * g0) = pack_bf16(o[t][i][e] * f, o[t][i][2 + e] * f);
              } else {
                dst[16 * i + g0] = __float2bfloat16_rn(o[t][i][e] * f);
                dst[16 * i + 8 + g0] = __float2bfloat16_rn(o[t][i][2 + e] * f);
              }
            }
          } else {
            float* pp = a.part + (((size_t)u * a.n_kv + cg.kvh) * a.max_cols + col) * (D + 4);
            if (g0 == 0) *reinterpret_cast<float2*>(pp) = make_float2(m[t][e], sum);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              if (FP8) {
                *reinterpret_cast<float2*>(pp + 4 + 16 * i + 2 * g0) = make_float2(o[t][i][e] * (1.f / kValueShift), o[t][i][2 + e] * (1.f / kValueShift));
              } else {
                pp[4 + 16 * i + g0] = o[t][i][e];
                pp[4 + 16 * i + 8 + g0] = o[t][i][2 + e];
              }
            }
          }
        }
      cp = 0;
      cv += nw;
      if (cv < total) cg = geo(cv);
    }
  }
  cp_async_wait<0>();
}

// Joins the records of an item's units, one warp per (item, KV head, column): a lane owns D / 32
// neighbouring dimensions, lanes share out the units' maxima and sums, and a batch of records is in
// flight before the first is used, so a merge of a few units takes one trip to memory.
constexpr int MERGE_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(MERGE_WARPS * 32) attn_rows_merge(const RowsArgs a, const __grid_constant__ InlineInts inl,
                                                                     int num_items) {
  griddep_launch_dependents();
  griddep_wait();
  const int* const lists = list_base(a.lists, inl);
  const int *items = lists + a.o_items, *ubeg = lists + a.o_ubeg;
  const int G = a.n_q / a.n_kv, per = a.n_kv * a.max_cols;
  const long long w = (long long)blockIdx.x * MERGE_WARPS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)num_items * per) return;
  const int b = (int)(w / per), kvh = (int)(w % per) / a.max_cols, col = (int)(w % a.max_cols);
  const int u0 = ubeg[b], ns = ubeg[b + 1] - u0;
  if (ns <= 1 || col >= items[4 * b + 1] * G) return;  // written by its only unit / no such column
  const size_t step = (size_t)per * (D + 4);
  const float* p = a.part + (((size_t)u0 * a.n_kv + kvh) * a.max_cols + col) * (D + 4);
  constexpr int E = D / 32, B = 8;
  float o[E], m = -INFINITY, den = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int i0 = 0; i0 < ns; i0 += B) {
    float v[B][E], pm = -INFINITY, pl = 0.f;
    if (lane < B && i0 + lane < ns) {
      const float2 ml = *reinterpret_cast<const float2*>(p + (i0 + lane) * step);
      pm = ml.x;
      pl = ml.y;
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 x = make_float2(0.f, 0.f);
        if (i0 + i < ns) x = *reinterpret_cast<const float2*>(p + (i0 + i) * step + 4 + lane * E + e);
        v[i][e] = x.x;
        v[i][e + 1] = x.y;
      }
    float mx = pm;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mx = fmaxf(m, __shfl_sync(0xffffffffu, mx, 0));
    // a unit in which a column sees nothing has the maximum -inf and weighs nothing
    const float keep = m == -INFINITY ? 0.f : exp2f(m - mx), wt = pm == -INFINITY ? 0.f : exp2f(pm - mx);
    m = mx;
    float l = pl * wt;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    den = den * keep + __shfl_sync(0xffffffffu, l, 0);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(v[i][e], wi, o[e]);
    }
  }
  const int row = items[4 * b] + col / G, h = kvh * G + col % G;
  const float inv = 1.f / den;
  bf16* dst = a.out + (size_t)row * a.ldo + (size_t)h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[(size_t)h * a.ldl + row] = (m + log2f(den)) * kLn2;
}

template <int D, bool FP8, int NT>
cudaError_t launch_nt(const RowsArgs& a, const InlineInts& inl, const void* k, const void* v, const float* ks, const float* vs, int num_items,
                      int num_sms, cudaStream_t s) {
  using S = Rg<D, FP8>;
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(attn_rows_kernel<D, FP8, NT>), S::SMEM, once);
  if (e != cudaSuccess) return e;
  const long long total = (long long)a.num_units * a.n_kv;
  e = launch_pdl(attn_rows_kernel<D, FP8, NT>, dim3((unsigned)(total < num_sms ? total : num_sms)), dim3(S::WARPS * 32),
                 S::SMEM, s, a, inl, static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v), ks, vs,
                 1.4426950408889634f / sqrtf((float)D));
  if (e != cudaSuccess || a.num_units == num_items) return e;
  const long long warps = (long long)num_items * a.n_kv * a.max_cols;
  return launch_pdl(attn_rows_merge<D>, dim3((unsigned)((warps + MERGE_WARPS - 1) / MERGE_WARPS)), dim3(MERGE_WARPS * 32),
                    0, s, a, inl, num_items);
}

template <int D, bool FP8>
cudaError_t launch_cols(const RowsArgs& a, const InlineInts& inl, const void* k, const void* v, const float* ks, const float* vs, int num_items,
                        int num_sms, cudaStream_t s) {
  return a.max_cols <= 8 ? launch_nt<D, FP8, 1>(a, inl, k, v, ks, vs, num_items, num_sms, s)
                         : launch_nt<D, FP8, 2>(a, inl, k, v, ks, vs, num_items, num_sms, s);
}

}  // namespace

cudaError_t launch_attn_rows(const RowsArgs& a, const InlineInts& inl, const void* k, const void* v, const float* ks, const float* vs, int d_head,
                             int num_items, int num_sms, cudaStream_t s) {
  if (a.max_cols > kRowsCols || (!ks != !vs)) return cudaErrorNotSupported;
  if (d_head == 128)
    return ks ? launch_cols<128, true>(a, inl, k, v, ks, vs, num_items, num_sms, s)
              : launch_cols<128, false>(a, inl, k, v, ks, vs, num_items, num_sms, s);
  if (d_head == 64)
    return ks ? launch_cols<64, true>(a, inl, k, v, ks, vs, num_items, num_sms, s)
              : launch_cols<64, false>(a, inl, k, v, ks, vs, num_items, num_sms, s);
  return cudaErrorNotSupported;
}

}  // namespace skv
