// New keys and values into the paged cache, with the rotation of their positions on the way
// (swiftkv_append, and the model's own calls on an int8 cache).
//
//   k' = R(pos) k, q' = R(pos) q: pairs (i, i + d/2) turned by pos theta^(-2i/d), in float32, rounded
//   to bf16 once. Cache row ctx + i of the sequence takes
//     bf16   k' and v
//     FP8    per row and head the scale s = max|x| / 448 and the e4m3 codes of x / s
//     int8   per page and head one scale and codes round(x / s) in [-127, 127]. The scale is that of the
//            new rows, max|x| / 127, or, on a page that holds earlier rows, the larger of that and what the
//            page has; where it grows the earlier rows' codes become round(code * old / new), off by half a
//            step of the new scale each time.
//
// Bound by HBM: every row is read and written once, 4 chunks of ~1960 rows with q, 32 / 8 heads x 128, 193 MB, in 33 us;
// 11703 rows of 8 caches, 767 MB, in 123; 24 tokens in 8.5, which is the launch and two trips to memory. One cache's
// codes are bound by latency: K and V of 11703 rows, 72 MB, go into FP8 or int8 in 23 us, 2.3 TB/s inside the kernel with
// 0.55 instructions a cycle and scheduler and its warps waiting for loads: a warp reads its block, turns it, finds its
// maximum and writes in series, and 2.4 rounds of warps hide little of that. Into int8 of 8 caches, 575 MB, the same
// takes 115, 5.1 TB/s. With a division for each value those were 41, 43 and 258. A lane owns 8 neighbouring dimensions and their
// partners half a head on, so a pair turns within a lane, all accesses are 16 bytes (8 for codes), and a
// head is 8 lanes (4 at d_head 64).
//   Rows (q; K and V of a bf16 or FP8 cache): a warp takes one token and steps through its heads with the
//   token's angles in registers, 2 heads in flight per lane (4 take the registers of a warp in four). Few tokens are split among several warps.
//   Pages (K and V of an int8 cache): a warp takes one (page, cache, K or V, head): its new rows stay in
//   registers between the maximum and the codes. One warp owns the block, so a repeated call repeats its bits.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "pdl.cuh"
#include "serving.h"

namespace skv {

namespace {

constexpr int AWARPS = 4;
constexpr int UNROLL = 2;  // heads in flight per lane

// The last of n entries of the ascending f with f(s) <= v (f(0) <= v), searched by the whole warp.
template <typename F>
__device__ __forceinline__ int find_last(int n, int v, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32, at = lane * step;
    const unsigned in = __ballot_sync(0xffffffffu, at < len && f(lo + at) <= v);
    const int k = (31 - __clz(in)) * step;
    lo += k;
    len = min(step, len - k);
  }
  return lo;
}

// 16 values of a lane: dims 8 j .. + 7 and their partners.
struct Piece {
  uint4 a, b;
};
__device__ __forceinline__ void turn_piece(Piece& p, const float2* cs) {
  uint32_t* a = &p.a.x;
  uint32_t* b = &p.b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0 = __uint_as_float(a[i] << 16), x1 = __uint_as_float(a[i] & 0xffff0000u);
    float y0 = __uint_as_float(b[i] << 16), y1 = __uint_as_float(b[i] & 0xffff0000u);
    rope_turn_pair(cs[2 * i], x0, y0);
    rope_turn_pair(cs[2 * i + 1], x1, y1);
    a[i] = pack_bf16(x0, x1);
    b[i] = pack_bf16(y0, y1);
  }
}
// The largest magnitude of a lane's values as a bf16's bits, in which NaN is above infinity and that above the rest.
__device__ __forceinline__ uint32_t largest(const Piece& p) {
  const uint32_t w[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ float bits_to_f32(uint32_t bf16_bits) { return __uint_as_float(bf16_bits << 16); }
__device__ __noinline__ float largest_number(uint4 a, uint4 b) {  // NaN left out
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(bits_to_f32(w[i] & 0xffffu)), fabsf(bits_to_f32(w[i] >> 16))));
  return m;
}
// The same without NaN, and with infinities as the largest finite number.
__device__ __noinline__ uint32_t largest_finite(uint4 a, uint4 b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
    m = max(m, max(lo > 0x7f80u ? 0u : min(lo, 0x7f7fu), hi > 0x7f80u ? 0u : min(hi, 0x7f7fu)));
  }
  return m;
}
__device__ __noinline__ float2 far_angle(const unsigned long long* turns, int pos, int i) {
  return rope_angle(nullptr, 0, turns, 0, pos, i);
}
template <int D, bool NEAR>
__device__ __forceinline__ void load_angles(const AppendArgs& a, int pos, int j, float2* cs) {
  if (NEAR || pos < a.rope_len) {
    const float4* t = reinterpret_cast<const float4*>(a.rope_tab + (size_t)pos * (D / 2) + 8 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = t[i];
      cs[2 * i] = make_float2(f.x, f.y);
      cs[2 * i + 1] = make_float2(f.z, f.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = far_angle(a.rope_turn, pos, 8 * j + i);
  }
}

// Two quotients x / scale rounded to float32, from the reciprocal (itself rounded): the quotient's remainder, exact
// in a fused multiply-add, corrects it (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000",
// 1990). For scales at which no remainder is subnormal. A division by itself is some five times as long.
__device__ __forceinline__ void quotients(float2& x, float scale, float recip) {
  asm("{\n .reg .b64 a, b, c, q, r;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mov.b64 c, {%3, %3};\n"
      " mul.rn.f32x2 q, a, b;\n fma.rn.f32x2 r, q, c, a;\n fma.rn.f32x2 q, r, b, q;\n mov.b64 {%0, %1}, q;\n}\n"
      : "+f"(x.x), "+f"(x.y)
      : "f"(recip), "f"(-scale));
}
__device__ __forceinline__ bool plain_scale(float scale) { return scale > 1e-20f && scale < 1e30f; }
__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// x / scale as int8 codes: with 1.5 2^23 added the integer next to a quotient (ties to even) is the sum's last byte.
__device__ __forceinline__ uint2 codes8(uint4 v, float scale, float recip) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = pair_of(w[i]);
    quotients(x, scale, recip);
    c[2 * i] = __float_as_uint(x.x + 12582912.f);
    c[2 * i + 1] = __float_as_uint(x.y + 12582912.f);
  }
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}
// The same for values and scales of any kind; NaN becomes 0.
__device__ __forceinline__ uint32_t code8_any(float x, float scale) {
  return (uint32_t)(max(-127, min(127, __float2int_rn(x / scale))) & 255);
}
__device__ __noinline__ uint2 codes8_any(uint4 v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair_of(w[i]);
    c[2 * i] = code8_any(x.x, scale);
    c[2 * i + 1] = code8_any(x.y, scale);
  }
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}
__device__ __forceinline__ uint2 rescale8(uint2 v, float ratio) {
  uint32_t out[2] = {v.x, v.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int code = (int)(out[h] << (24 - 8 * i)) >> 24;
      r |= (uint32_t)(__float2int_rn((float)code * ratio) & 255) << (8 * i);
    }
    out[h] = r;
  }
  return make_uint2(out[0], out[1]);
}

template <int D, int KIND>
__global__ void __launch_bounds__(AWARPS * 32, 8) append_kernel(const AppendArgs a, const __grid_constant__ InlineInts inl) {
  constexpr int LPV = D / 16, VPW = 32 / LPV;  // lanes of a head, heads (or rows) of a warp's step
  griddep_launch_dependents();
  griddep_wait();
  const int* const lists = list_base(a.lists, inl);
  const int *cu = lists + a.o_cu, *ctx = lists + a.o_ctx, *off = lists + a.o_off;
  const long long* const pools = a.pools ? a.pools : reinterpret_cast<const long long*>(lists + a.o_pools);
  const int lane = threadIdx.x & 31, sub = lane / LPV, j = lane % LPV;
  unsigned w = blockIdx.x * AWARPS + (threadIdx.x >> 5);  // fewer than 2^31 warps
  if (w < a.row_warps) {
    const int t = (int)(w / (unsigned)a.splits), split = (int)(w - (unsigned)(t * a.splits));
    const int s = find_last(a.P, t, [&](int i) { return cu[i]; });
    const int row = ctx[s] + t - cu[s], pos = row + (a.o_off >= 0 ? off[s] : 0);
    const int page = KIND == kKvInt8 ? 0 : a.bt[(size_t)s * a.max_pages + (row >> 4)];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && lane == 0 && split == 0) atomicOr(a.status, kStatusBadPage);
    float2 cs[8];
    if (a.rotate) load_angles<D, false>(a, pos, j, cs);
    const int nq = a.q ? a.n_q : 0, nvec = nq + (KIND == kKvInt8 ? 0 : a.caches * 2 * a.n_kv);
    // vectors in order: the query heads, then K heads and V heads of each cache
    for (int v0 = split * UNROLL * VPW; v0 < nvec; v0 += a.splits * UNROLL * VPW) {
      Piece p[UNROLL];
      int cache[UNROLL], head[UNROLL];  // head: -1 nothing, then query heads, K heads, V heads
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int vec = v0 + u * VPW + sub;
        p[u].a = p[u].b = make_uint4(0, 0, 0, 0);
        cache[u] = 0;
        head[u] = -1;
        const bf16* src = nullptr;
        if (vec < nq) {
          head[u] = vec;
          src = a.q + (size_t)t * a.ldq + (size_t)vec * D;
        } else if (vec < nvec) {
          const int r = vec - nq, c = (int)__umulhi((uint32_t)r, a.per_cache), h = r - c * 2 * a.n_kv;
          cache[u] = c;
          head[u] = a.n_q + h;
          src = h < a.n_kv ? a.k + (size_t)t * a.ldk + (size_t)c * a.k_step + (size_t)h * D
                           : a.v + (size_t)t * a.ldv + (size_t)c * a.v_step + (size_t)(h - a.n_kv) * D;
        }
        if (src) {
          p[u].a = *reinterpret_cast<const uint4*>(src + 8 * j);
          p[u].b = *reinterpret_cast<const uint4*>(src + D / 2 + 8 * j);
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const bool is_q = head[u] < a.n_q, is_v = head[u] >= a.n_q + a.n_kv;
        if (a.rotate && !is_v) turn_piece(p[u], cs);
        if (is_q) {
          if (head[u] >= 0) {
            bf16* dst = a.q_out + (size_t)t * a.ldq_out + (size_t)head[u] * D + 8 * j;
            *reinterpret_cast<uint4*>(dst) = p[u].a;
            *reinterpret_cast<uint4*>(dst + D / 2) = p[u].b;
          }
        }
        if (KIND == kKvInt8) continue;
        const int h = head[u] - a.n_q - (is_v ? a.n_kv : 0);
        const size_t at = ((size_t)page * a.n_kv + (is_q ? 0 : h)) * kPageSize + (row & 15);
        const long long* pool = pools + (is_v ? a.pool_step : 0) + cache[u];
        if (KIND == kKvBf16) {
          if (!is_q && ok) {
            bf16* dst = reinterpret_cast<bf16*>(*pool) + at * D + 8 * j;
            *reinterpret_cast<uint4*>(dst) = p[u].a;
            *reinterpret_cast<uint4*>(dst + D / 2) = p[u].b;
          }
        } else {
          // (as the model's epilogues: the largest but NaN, infinities among them)
          uint32_t most = largest(p[u]);
#pragma unroll
          for (int o = 1; o < LPV; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
          float top = bits_to_f32(most);
          if (__any_sync(0xffffffffu, most > 0x7f80u)) {
            top = largest_number(p[u].a, p[u].b);
#pragma unroll
            for (int o = 1; o < LPV; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          }
          if (!is_q && ok) {
            const float scale = top / 448.f;
            const uint32_t* x = &p[u].a.x;
            const uint32_t* y = &p[u].b.x;
            uint16_t c[8];
            if (plain_scale(scale)) {
              const float recip = 1.f / scale;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float2 f = pair_of(x[i]), g = pair_of(y[i]);
                quotients(f, scale, recip);
                quotients(g, scale, recip);
                c[i] = e4m3x2_from_f32(f.x, f.y);
                c[4 + i] = e4m3x2_from_f32(g.x, g.y);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = pair_of(x[i]), g = pair_of(y[i]);
                c[i] = scale > 0.f ? e4m3x2_from_f32(f.x / scale, f.y / scale) : (uint16_t)0;
                c[4 + i] = scale > 0.f ? e4m3x2_from_f32(g.x / scale, g.y / scale) : (uint16_t)0;
              }
            }
            uint8_t* dst = reinterpret_cast<uint8_t*>(*pool) + at * D + 8 * j;
            *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
            *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(c[4] | (uint32_t)c[5] << 16, c[6] | (uint32_t)c[7] << 16);
            if (j == 0) reinterpret_cast<float*>(pool[2 * a.pool_step])[at] = scale;
          }
        }
      }
    }
    return;
  }
  if (KIND != kKvInt8) return;
  // int8: virtual page x of sequence s, those of a sequence starting at cu[s] / 16 + 2 s: n rows touch at
  // most floor(n / 16) + 2 pages, which is no more than the distance to the next sequence's
  const unsigned rows = (a.row_warps + AWARPS - 1) / AWARPS * AWARPS;
  if (w < rows) return;  // of the last block of rows
  w -= rows;
  const unsigned per = (unsigned)(a.caches * 2 * a.n_kv);
  const int x = (int)(w / per);
  if (x >= a.pages) return;
  const int r = (int)(w - x * per), c = (int)__umulhi((uint32_t)r, a.per_cache), h2 = r - c * 2 * a.n_kv;
  const bool is_v = h2 >= a.n_kv;
  const int h = is_v ? h2 - a.n_kv : h2;
  const int s = find_last(a.P, x, [&](int i) { return (cu[i] >> 4) + 2 * i; });
  const int r0 = cu[s], n = cu[s + 1] - r0, c0 = ctx[s];
  const int pidx = (c0 >> 4) + (x - (r0 >> 4) - 2 * s), key0 = pidx << 4;
  if (n < 1 || key0 >= c0 + n) return;
  const int page = a.bt[(size_t)s * a.max_pages + pidx];
  const int first = max(0, c0 - key0), last = min(kPageSize, c0 + n - key0);  // the page's new rows
  const bf16* src = (is_v ? a.v + (size_t)c * a.v_step : a.k + (size_t)c * a.k_step) + (size_t)h * D + 8 * j;
  const long long ld = is_v ? a.ldv : a.ldk;
  src += (r0 + key0 - c0) * ld;  // of the page's first row, which may lie before the batch's
  const long long* pool = pools + (is_v ? a.pool_step : 0) + c;
  const bool turned = !is_v && a.rotate;
  const int pos0 = key0 + (a.o_off >= 0 ? off[s] : 0);
  // all 16 rows new, near and plain (most pages of a prompt): no row needs a look of its own
  auto block = [&](auto whole_) {
    constexpr bool WHOLE = decltype(whole_)::value;
    constexpr int STEPS = kPageSize / VPW;
    Piece p[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int row = i * VPW + sub;
      p[i].a = p[i].b = make_uint4(0, 0, 0, 0);
      if (WHOLE || (row >= first && row < last)) {
        const bf16* from = src + row * ld;
        p[i].a = *reinterpret_cast<const uint4*>(from);
        p[i].b = *reinterpret_cast<const uint4*>(from + D / 2);
      }
    }
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, kStatusBadPage);
      return;
    }
    float* scale_at = reinterpret_cast<float*>(pool[2 * a.pool_step]) + (size_t)page * a.n_kv + h;
    const float old = !WHOLE && first > 0 ? *scale_at : 0.f;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int row = i * VPW + sub;
      if (turned && (WHOLE || (row >= first && row < last))) {
        float2 cs[8];
        load_angles<D, WHOLE>(a, pos0 + row, j, cs);
        turn_piece(p[i], cs);
      }
      most = max(most, largest(p[i]));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    const bool finite = most < 0x7f80u;
    if (!finite) {  // an infinity counts as the largest bf16, NaN not at all
      most = 0;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) most = max(most, largest_finite(p[i].a, p[i].b));
      most = __reduce_max_sync(0xffffffffu, most);
    }
    const float scale = fmaxf(bits_to_f32(most) / 127.f, old), by = scale > 0.f ? scale : 1.f, recip = 1.f / by;
    uint8_t* dst = reinterpret_cast<uint8_t*>(*pool) + ((size_t)page * a.n_kv + h) * kPageSize * D + 8 * j;
    if (finite && plain_scale(by)) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int row = i * VPW + sub;
        if (WHOLE || (row >= first && row < last)) {
          *reinterpret_cast<uint2*>(dst + row * D) = codes8(p[i].a, by, recip);
          *reinterpret_cast<uint2*>(dst + row * D + D / 2) = codes8(p[i].b, by, recip);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int row = i * VPW + sub;
        if (WHOLE || (row >= first && row < last)) {
          *reinterpret_cast<uint2*>(dst + row * D) = codes8_any(p[i].a, by);
          *reinterpret_cast<uint2*>(dst + row * D + D / 2) = codes8_any(p[i].b, by);
        }
      }
    }
    if (!WHOLE && scale > old) {
      const float ratio = old / scale;
      for (int row = sub; row < first; row += VPW) {
        uint2* lo = reinterpret_cast<uint2*>(dst + row * D);
        uint2* hi = reinterpret_cast<uint2*>(dst + row * D + D / 2);
        *lo = rescale8(*lo, ratio);
        *hi = rescale8(*hi, ratio);
      }
    }
    if (lane == 0 && (WHOLE || first == 0 || scale > old)) *scale_at = scale;
  };
  if (first == 0 && last == kPageSize && (!turned || pos0 + kPageSize <= a.rope_len)) block(std::true_type());
  else block(std::false_type());
}

template <int D, int KIND>
cudaError_t launch_kind(const AppendArgs& a, const InlineInts& inl, cudaStream_t s) {
  const long long rows = ((long long)a.row_warps + AWARPS - 1) / AWARPS;
  const long long pages = KIND == kKvInt8 ? ((long long)a.pages * a.caches * 2 * a.n_kv + AWARPS - 1) / AWARPS : 0;
  if (rows + pages <= 0) return cudaSuccess;
  if ((rows + pages) * AWARPS >= 1LL << 31) return cudaErrorNotSupported;
  return launch_pdl(append_kernel<D, KIND>, dim3((unsigned)(rows + pages)), dim3(AWARPS * 32), 0, s, a, inl);
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, int kind, const InlineInts& inl, cudaStream_t s) {
  return kind == kKvBf16 ? launch_kind<D, kKvBf16>(a, inl, s)
         : kind == kKvFp8 ? launch_kind<D, kKvFp8>(a, inl, s) : launch_kind<D, kKvInt8>(a, inl, s);
}

}  // namespace

cudaError_t launch_append(AppendArgs a, int kind, int d_head, const InlineInts& inl, int num_sms, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (d_head != 64 && d_head != 128) return cudaErrorNotSupported;
  a.per_cache = (uint32_t)((1ULL << 32) / (2 * a.n_kv)) + 1;  // r * this >> 32 = r / (2 n_kv) for r < 2^16
  const int vecs = (a.q ? a.n_q : 0) + (kind == kKvInt8 ? 0 : a.caches * 2 * a.n_kv);
  const int steps = (vecs + UNROLL * (512 / d_head) - 1) / (UNROLL * (512 / d_head));
  // a token's heads go to several warps until every SM has 16 of them
  a.splits = (int)std::max(1LL, std::min<long long>(steps, (16LL * num_sms + a.T - 1) / a.T));
  if ((long long)a.T * a.splits >= 1LL << 31) return cudaErrorNotSupported;
  a.row_warps = steps ? (unsigned)(a.T * a.splits) : 0;
  a.pages = kind == kKvInt8 ? (a.T >> 4) + 2 * a.P : 0;
  return d_head == 128 ? launch_d<128>(a, kind, inl, s) : launch_d<64>(a, kind, inl, s);
}

}  // namespace skv
