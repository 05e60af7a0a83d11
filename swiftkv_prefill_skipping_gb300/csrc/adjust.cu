// Penalties for repeated tokens, biases and grammar masks on logits, before swiftkv_sample.
//
//   s_i: id i is in the row's history; c_i: how often in the part after the prompt
//   x = s_i ? (l_i > 0 ? l_i * (1 / rep) : l_i * rep) : l_i
//   x = x - frequency * c_i - presence * (c_i > 0) + bias_i;  x = -inf where the mask forbids i
//
// Bound by HBM: the row is read and written once. A CTA owns a slice of one row's ids and copies it through shared
// memory. While the copy arrives it walks the row's whole history and keeps what concerns its slice, one 32-bit
// word an id: count, prompt bit and place in the bias list; the words meet the logits on their way out. No CTA waits
// for another, and counts are integers: the order of the atomics changes nothing. Everything that a CTA
// reads is asked for at its start: with lengths, ids, settings and mask one after another the same took 94 us.
// Without biases, and with histories that a count of 15 bits holds, a word has 16 bits. Slices are then half as long
// again, a history is walked less often, and three CTAs of 640 threads share an SM: 50 us where 32-bit words take 62 (16-bit
// ones with 512 threads 53, with slices of 8192 55, of 16384 55, two CTAs).
//
// 256 rows of 128256 with a mask, 262 MB: 37 us without histories (7.1 TB/s), 50 with 4000 - 8064 tokens each, of which
// the walk in every slice and the arithmetic on the words are 13, in series with the copy in each CTA and overlapped across
// three an SM. Measured with 32-bit words and not kept: the touched ids on a list (118 us with one place
// asked for at a time, 94 with one for a warp), each id computed by whoever takes its word (134), slices of 4096 and
// 12288 ids, a history walked once by a cluster of 2 / 4 / 8 CTAs with atomics on one another's words (74 / 80 / 93).
// 24 rows of 152064: 12.4 us, one row 6.7 to 8.6, latency.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "swiftkv.h"

namespace skv {

namespace {

constexpr int kThreads = 512, kMaxSlice = 8192;           // ids of a CTA: 64 KB of logits and words, three CTAs an SM
constexpr int kThreadsHalf = 640, kMaxSliceHalf = 12288;  // with 16-bit words: 72 KB, three as well
constexpr int kTargetBlocks = 304;      // CTAs that fill the GPU
constexpr unsigned kCount = 0xfffff;    // how often the id was generated
constexpr unsigned kPrompt = 1u << 20;  // it is in the prompt
constexpr int kBiasShift = 21;          // 1 + its last place in the bias list
constexpr unsigned kHalfCount = 0x7fff, kHalfPrompt = 0x8000;  // the same in 16 bits
constexpr int kMaxHistory = kCount, kMaxBias = (1 << (32 - kBiasShift)) - 2;

struct AdjustParams {
  const float* logits;
  long long ld;
  float* out;
  long long ldo;
  int V, slice, slices;  // slice: ids of a CTA, a multiple of 4
  const int* tokens;
  long long ld_tokens;
  int max_tokens;
  bool tokens16;  // histories start on 16 bytes
  const int *lens, *prompt_lens;
  const float *repetition, *presence, *frequency;
  float repetition_all, presence_all, frequency_all;
  const int* bias_ids;
  const float* bias;
  int num_bias;
  const uint32_t* mask;
  long long ld_mask;
};

// VEC: rows start on 16 bytes. HALF: histories that fit 16-bit words, two of them a word of memory, and no biases.
template <bool VEC, bool HALF>
__global__ void __launch_bounds__(HALF ? kThreadsHalf : kThreads) adjust_kernel(const AdjustParams p) {
  constexpr int AT = HALF ? kThreadsHalf : kThreads;
  extern __shared__ __align__(16) unsigned char smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int row = blockIdx.x / p.slices, base = (blockIdx.x - row * p.slices) * p.slice, tid = threadIdx.x;
  const int size = min(p.slice, p.V - base);
  const float* src = p.logits + (size_t)row * p.ld + base;
  float* dst = p.out + (size_t)row * p.ldo + base;
  const bool in_place = src == dst, lists = p.tokens || p.num_bias > 0;
  unsigned* word = reinterpret_cast<unsigned*>(smem);                                // [slice] words, with lists
  const unsigned word_bytes = lists ? p.slice * (HALF ? 2 : 4) : 0;
  float* x = reinterpret_cast<float*>(smem + word_bytes);                            // [slice], not in place
  uint32_t* allow = reinterpret_cast<uint32_t*>(x + (in_place ? 0 : p.slice));       // [slice / 32], with a mask
  // Everything that the CTA reads is asked for here, the lists beyond their ends too (as far as the arrays go):
  // one trip to memory and not one after another, which took most of a CTA's time
  constexpr int B = 2;  // fours of ids in flight
  const int* ids = p.tokens ? p.tokens + (size_t)row * p.ld_tokens : nullptr;
  auto fetch = [&](int i0, int end, int4* id) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = i0 + b * 4 * AT;
      id[b] = make_int4(-1, -1, -1, -1);
      if (p.tokens16 && i + 3 < end) {
        id[b] = *reinterpret_cast<const int4*>(ids + i);
      } else {
        if (i < end) id[b].x = ids[i];
        if (i + 1 < end) id[b].y = ids[i + 1];
        if (i + 2 < end) id[b].z = ids[i + 2];
        if (i + 3 < end) id[b].w = ids[i + 3];
      }
    }
  };
  int4 id[B];
  int len = 0, prompt = 0;
  float rep = 1.f, presence = 0.f, frequency = 0.f;
  if (ids) {
    fetch(tid * 4, p.max_tokens, id);
    len = p.lens ? p.lens[row] : p.max_tokens;
    prompt = p.prompt_lens ? p.prompt_lens[row] : 0;
    rep = p.repetition ? p.repetition[row] : p.repetition_all;
    presence = p.presence ? p.presence[row] : p.presence_all;
    frequency = p.frequency ? p.frequency[row] : p.frequency_all;
  }
  const int* bias_ids = p.bias_ids + (size_t)row * p.num_bias;
  const unsigned bias_id = tid < p.num_bias ? (unsigned)bias_ids[tid] : 0xffffffffu;
  const uint32_t* mask = p.mask ? p.mask + (size_t)row * p.ld_mask + (base >> 5) : nullptr;
  if (mask)
    for (int i = tid; i * 32 < size; i += AT) cp_async4(smem_u32(allow + i), mask + i, 4);
  if (!in_place) {
    if (VEC) {
      for (int i = tid * 4; i < size; i += 4 * AT)  // the bytes past the row's end become zeros
        cp_async16(smem_u32(x + i), src + i, min(16, (size - i) * 4));
    } else {
      for (int i = tid; i < size; i += AT) cp_async4(smem_u32(x + i), src + i, 4);
    }
  }
  cp_async_commit();
  if (lists) {
    for (unsigned i = tid * 16; i < word_bytes; i += 16 * AT) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
    auto in_prompt = [&](unsigned u) {
      if (HALF) atomicOr(word + (u >> 1), kHalfPrompt << (u & 1) * 16);
      else atomicOr(word + u, kPrompt);
    };
    auto generated = [&](unsigned u) {
      if (HALF) atomicAdd(word + (u >> 1), 1u << (u & 1) * 16);
      else atomicAdd(word + u, 1u);
    };
    __syncthreads();
    // an id less base, as unsigned: ids outside the slice, negative ones among them, are at least `size`
    if (!HALF && p.num_bias > 0) {  // an id named twice takes its last entry: the words hold nothing else yet
      for (int i = tid; i < p.num_bias; i += AT) {
        const unsigned u = (i == tid ? bias_id : (unsigned)bias_ids[i]) - (unsigned)base;
        if (u < (unsigned)size) atomicMax(word + u, (unsigned)(i + 1) << kBiasShift);
      }
      __syncthreads();
    }
    if (ids) len = min(len, p.max_tokens);
    for (int i1 = 0; i1 < len; i1 += 4 * AT * B) {
      const int i0 = i1 + tid * 4;
      if (i1 > 0) fetch(i0, len, id);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        unsigned u[4] = {(unsigned)id[b].x - (unsigned)base, (unsigned)id[b].y - (unsigned)base,
                         (unsigned)id[b].z - (unsigned)base, (unsigned)id[b].w - (unsigned)base};
        // the warp's 128 neighbours: all the prompt's, all behind it (both without a look at the single one), or neither
        const int w0 = i1 + b * 4 * AT + (tid >> 5) * 128, i = i0 + b * 4 * AT;
        if (w0 + 128 <= min(prompt, len)) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (u[e] < (unsigned)size) in_prompt(u[e]);
        } else if (w0 >= prompt && w0 + 128 <= len) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (u[e] < (unsigned)size) generated(u[e]);
        } else if (w0 < len) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < len && u[e] < (unsigned)size) {
              if (i + e < prompt) in_prompt(u[e]);
              else generated(u[e]);
            }
        }
      }
    }
  }
  if (!(rep > 0.f)) rep = 1.f;
  const float* bias = p.bias + (size_t)row * p.num_bias;
  const float per = 1.f / rep;
  constexpr unsigned count = HALF ? kHalfCount : kCount, in_list = HALF ? kHalfCount | kHalfPrompt : kCount | kPrompt;
  auto adjust = [&](unsigned w, float v) {
    if (w & in_list) v *= v > 0.f ? per : rep;
    if (w & count) v = v - frequency * (float)(w & count) - presence;
    if (!HALF && w >> kBiasShift) v += bias[(w >> kBiasShift) - 1];
    return v;
  };
  cp_async_wait<0>();
  __syncthreads();
  if (VEC && !in_place) {
    for (int u = tid * 4; u < size; u += 4 * AT) {
      float4 v = *reinterpret_cast<const float4*>(x + u);
      if (lists) {
        uint4 w;
        if (HALF) {
          const uint2 h = *reinterpret_cast<const uint2*>(word + u / 2);
          w = make_uint4(h.x & 0xffff, h.x >> 16, h.y & 0xffff, h.y >> 16);
        } else {
          w = *reinterpret_cast<const uint4*>(word + u);
        }
        if (w.x) v.x = adjust(w.x, v.x);
        if (w.y) v.y = adjust(w.y, v.y);
        if (w.z) v.z = adjust(w.z, v.z);
        if (w.w) v.w = adjust(w.w, v.w);
      }
      if (mask) {
        const unsigned a = allow[u >> 5] >> (u & 31);
        if (!(a & 1)) v.x = -INFINITY;
        if (!(a & 2)) v.y = -INFINITY;
        if (!(a & 4)) v.z = -INFINITY;
        if (!(a & 8)) v.w = -INFINITY;
      }
      if (u + 3 < size) {
        *reinterpret_cast<float4*>(dst + u) = v;
      } else {
        dst[u] = v.x;
        if (u + 1 < size) dst[u + 1] = v.y;
        if (u + 2 < size) dst[u + 2] = v.z;
      }
    }
  } else {
    for (int u = tid; u < size; u += AT) {
      const unsigned w = !lists ? 0u : HALF ? reinterpret_cast<const uint16_t*>(word)[u] : word[u];
      const bool ok = !mask || (allow[u >> 5] >> (u & 31) & 1);
      if (in_place) {  // what nothing concerns is neither read nor written
        if (!ok) dst[u] = -INFINITY;
        else if (w) dst[u] = adjust(w, src[u]);
      } else {
        dst[u] = !ok ? -INFINITY : w ? adjust(w, x[u]) : x[u];
      }
    }
  }
}

template <bool VEC, bool HALF>
cudaError_t launch_vec(const AdjustParams& p, int rows, cudaStream_t s) {
  const bool lists = p.tokens || p.num_bias > 0, in_place = p.logits == p.out;
  constexpr int most = HALF ? kMaxSliceHalf * 6 + kMaxSliceHalf / 8 : kMaxSlice * 8 + kMaxSlice / 8;
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(adjust_kernel<VEC, HALF>), most, once);
  if (e != cudaSuccess) return e;
  const int smem = (lists ? p.slice * (HALF ? 2 : 4) : 0) + (in_place ? 0 : p.slice * 4) + (p.mask ? p.slice / 8 : 0);
  const long long blocks = (long long)rows * p.slices;
  if (blocks >= 1LL << 31) return cudaErrorNotSupported;
  return launch_pdl(adjust_kernel<VEC, HALF>, dim3((unsigned)blocks), dim3(HALF ? kThreadsHalf : kThreads), smem, s, p);
}

}  // namespace

}  // namespace skv

using namespace skv;

extern "C" int swiftkv_adjust_logits(const float* logits, int rows, int vocab, long long ld, const swiftkv_adjustments* a,
                                     float* out, long long ld_out, swiftkv_stream stream) {
  if (rows < 0 || vocab < 1) return set_error(SWIFTKV_EINVAL, "need rows >= 0 and vocab >= 1");
  if (rows == 0) return SWIFTKV_OK;
  if (!logits || !a || !out) return set_error(SWIFTKV_EINVAL, "null logits / adjustments / out");
  if (ld < vocab || ld_out < vocab) return set_error(SWIFTKV_EINVAL, "row stride smaller than vocab");
  if (a->max_tokens < 0 || a->num_bias < 0) return set_error(SWIFTKV_EINVAL, "negative max_tokens or num_bias");
  const bool hist = a->max_tokens > 0, bias = a->num_bias > 0;
  if (hist && !a->tokens) return set_error(SWIFTKV_EINVAL, "null tokens");
  if (bias && (!a->bias_ids || !a->bias)) return set_error(SWIFTKV_EINVAL, "null bias_ids / bias");
  if (hist && rows > 1 && a->ld_tokens < a->max_tokens)
    return set_error(SWIFTKV_EINVAL, "stride of tokens smaller than max_tokens");
  if (a->mask && rows > 1 && a->ld_mask < (vocab + 31LL) / 32)
    return set_error(SWIFTKV_EINVAL, "stride of the mask smaller than a row's words");
  const void* const arrays[] = {logits, out, a->tokens, a->lens, a->prompt_lens, a->repetition, a->presence, a->frequency,
                                a->bias_ids, a->bias, a->mask};
  for (const void* x : arrays)
    if (reinterpret_cast<uintptr_t>(x) & 3) return set_error(SWIFTKV_EINVAL, "misaligned logits / out / adjustments");
  if (a->max_tokens > kMaxHistory) return set_error(SWIFTKV_EUNSUPPORTED, "histories above 1048575 tokens");
  if (a->num_bias > kMaxBias) return set_error(SWIFTKV_EUNSUPPORTED, "more than 2046 biases a row");
  if (vocab > (1 << 30)) return set_error(SWIFTKV_EUNSUPPORTED, "vocab above 2^30");
  if (rows > (1 << 27)) return set_error(SWIFTKV_EUNSUPPORTED, "more than 2^27 rows");
  if (!(logits == out && (ld == ld_out || rows == 1)) && rows_meet(logits, 4 * ld, 4LL * vocab, out, 4 * ld_out, 4LL * vocab, rows))
    return set_error(SWIFTKV_EINVAL, "out overlaps logits without being them");
  AdjustParams p;
  p.logits = logits;
  p.ld = ld;
  p.out = out;
  p.ldo = ld_out;
  p.V = vocab;
  p.tokens = hist ? a->tokens : nullptr;
  p.ld_tokens = a->ld_tokens;
  p.max_tokens = a->max_tokens;
  p.tokens16 = (reinterpret_cast<uintptr_t>(a->tokens) & 15) == 0 && (rows == 1 || a->ld_tokens % 4 == 0);
  p.lens = a->lens;
  p.prompt_lens = a->prompt_lens;
  p.repetition = a->repetition;
  p.presence = a->presence;
  p.frequency = a->frequency;
  p.repetition_all = a->repetition_all;
  p.presence_all = a->presence_all;
  p.frequency_all = a->frequency_all;
  p.bias_ids = a->bias_ids;
  p.bias = a->bias;
  p.num_bias = a->num_bias;
  p.mask = a->mask;
  p.ld_mask = a->ld_mask;
  const bool vec = ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & 15) == 0 &&
                   (rows == 1 || (ld % 4 == 0 && ld_out % 4 == 0));
  // Short slices while there are few rows, so that every SM has work; long ones walk a history less often.
  const bool half = hist && !bias && a->max_tokens <= (int)kHalfCount;
  const long long ids = (long long)rows * vocab, want = (ids / kTargetBlocks + 1023) / 1024 * 1024;
  p.slice = (int)std::max(1024LL, std::min<long long>(half ? kMaxSliceHalf : kMaxSlice, want));
  p.slices = (vocab + p.slice - 1) / p.slice;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = vec ? (half ? launch_vec<true, true>(p, rows, s) : launch_vec<true, false>(p, rows, s))
                            : (half ? launch_vec<false, true>(p, rows, s) : launch_vec<false, false>(p, rows, s));
  if (e != cudaSuccess)
    return set_error(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, cudaGetErrorString(e));
  return SWIFTKV_OK;
}
