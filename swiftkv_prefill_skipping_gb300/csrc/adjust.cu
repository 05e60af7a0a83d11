// Penalties for repeated tokens, biases and grammar masks on logits, before swiftkv_sample.
//
//   s_i: id i is in the row's history; c_i: how often in the part after the prompt
//   x = s_i ? (l_i > 0 ? l_i / rep : l_i * rep) : l_i
//   x = x - frequency * c_i - presence * (c_i > 0) + bias_i;  x = -inf where the mask forbids i
//
// Bound by HBM: the row is read and written once. A CTA owns a slice of one row's ids and reads the
// row's whole history itself, keeping what concerns its slice: one 32-bit word an id in shared memory,
// count, prompt bit and place in the bias list. No CTA waits for another, and integer counts make the order of
// the atomics irrelevant. The slice's logits are requested before the history is walked.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "swiftkv.h"

namespace skv {

namespace {

constexpr int AT = 512;                 // threads
constexpr unsigned kCount = 0xfffff;    // how often the id was generated
constexpr unsigned kPrompt = 1u << 20;  // it is in the prompt
constexpr int kBiasShift = 21;          // 1 + its last place in the bias list
constexpr int kMaxHistory = kCount, kMaxBias = (1 << (32 - kBiasShift)) - 2;

struct AdjustParams {
  const float* logits;
  long long ld;
  float* out;
  long long ldo;
  int V, slices;
  const int* tokens;
  long long ld_tokens;
  int max_tokens;
  const int *lens, *prompt_lens;
  const float *repetition, *presence, *frequency;
  float repetition_all, presence_all, frequency_all;
  const int* bias_ids;
  const float* bias;
  int num_bias;
  const uint32_t* mask;
  long long ld_mask;
};

// N: groups of four ids a thread owns. VEC: rows start on 16 bytes; a thread's four ids are neighbours, else they
// lie AT apart.
template <int N, bool VEC>
__global__ void __launch_bounds__(AT) adjust_kernel(const AdjustParams p) {
  constexpr int SLICE = 4 * N * AT;
  extern __shared__ __align__(16) unsigned word[];
  griddep_launch_dependents();
  griddep_wait();
  const int row = blockIdx.x / p.slices, base = (blockIdx.x - row * p.slices) * SLICE, tid = threadIdx.x;
  const int size = min(SLICE, p.V - base);
  const float* src = p.logits + (size_t)row * p.ld + base;
  float* dst = p.out + (size_t)row * p.ldo + base;
  auto at = [&](int g, int e) { return VEC ? (g * AT + tid) * 4 + e : (g * 4 + e) * AT + tid; };
  const bool in_place = src == dst;
  float x[N][4];
  auto load = [&](int g) {
    if (VEC && at(g, 3) < size) {
      const float4 f = *reinterpret_cast<const float4*>(src + at(g, 0));
      x[g][0] = f.x;
      x[g][1] = f.y;
      x[g][2] = f.z;
      x[g][3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[g][e] = at(g, e) < size ? src[at(g, e)] : 0.f;
    }
  };
  // in place a group that nothing concerns is not read either
  if (!in_place)
#pragma unroll
    for (int g = 0; g < N; ++g) load(g);
  const int* ids = p.tokens ? p.tokens + (size_t)row * p.ld_tokens : nullptr;
  const int len = ids ? max(0, min(p.max_tokens, p.lens ? p.lens[row] : p.max_tokens)) : 0;
  const int prompt = p.prompt_lens ? p.prompt_lens[row] : 0;
  const bool listed = ids || p.num_bias > 0;
  if (listed) {
#pragma unroll
    for (int g = 0; g < N; ++g) reinterpret_cast<uint4*>(word)[g * AT + tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (p.num_bias > 0) {  // an id named twice takes its last entry: the words hold nothing else yet
      for (int i = tid; i < p.num_bias; i += AT) {
        const long long u = (long long)p.bias_ids[(size_t)row * p.num_bias + i] - base;
        if (u >= 0 && u < size) atomicMax(word + u, (unsigned)(i + 1) << kBiasShift);
      }
      __syncthreads();
    }
    constexpr int B = 4;
    for (int i0 = tid; i0 < len; i0 += B * AT) {
      int id[B];
#pragma unroll
      for (int b = 0; b < B; ++b) id[b] = i0 + b * AT < len ? ids[i0 + b * AT] : -1;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const long long u = (long long)id[b] - base;
        if (u < 0 || u >= size || id[b] < 0) continue;
        if (i0 + b * AT < prompt) atomicOr(word + u, kPrompt);
        else atomicAdd(word + u, 1u);
      }
    }
    __syncthreads();
  }
  float rep = p.repetition ? p.repetition[row] : p.repetition_all;
  if (!(rep > 0.f)) rep = 1.f;
  const float presence = p.presence ? p.presence[row] : p.presence_all;
  const float frequency = p.frequency ? p.frequency[row] : p.frequency_all;
  const uint32_t* mask = p.mask ? p.mask + (size_t)row * p.ld_mask : nullptr;
  const float* bias = p.bias + (size_t)row * p.num_bias;
#pragma unroll
  for (int g = 0; g < N; ++g) {
    unsigned w[4] = {0, 0, 0, 0}, allowed = 15;
    if (listed) {
      if (VEC) {
        const uint4 q = reinterpret_cast<const uint4*>(word)[g * AT + tid];
        w[0] = q.x;
        w[1] = q.y;
        w[2] = q.z;
        w[3] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = word[at(g, e)];
      }
    }
    if (mask) {
      if (VEC) {
        const int i = base + at(g, 0);
        if (at(g, 0) < size) allowed = mask[i >> 5] >> (i & 31) & 15;
      } else {
        allowed = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = base + at(g, e);
          if (at(g, e) < size) allowed |= (mask[i >> 5] >> (i & 31) & 1) << e;
        }
      }
    }
    if (in_place) {
      if (!(w[0] | w[1] | w[2] | w[3]) && allowed == 15) continue;
      load(g);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = x[g][e];
      if (w[e]) {
        const unsigned count = w[e] & kCount, place = w[e] >> kBiasShift;
        if (w[e] & (kCount | kPrompt)) v = v > 0.f ? v / rep : v * rep;
        if (count) v = v - frequency * (float)count - presence;
        if (place) v += bias[place - 1];
      }
      x[g][e] = allowed >> e & 1 ? v : -INFINITY;
    }
    if (VEC && at(g, 3) < size) {
      *reinterpret_cast<float4*>(dst + at(g, 0)) = make_float4(x[g][0], x[g][1], x[g][2], x[g][3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at(g, e) < size) dst[at(g, e)] = x[g][e];
    }
  }
}

template <int N, bool VEC>
cudaError_t launch_n(AdjustParams p, int rows, cudaStream_t s) {
  constexpr int slice = 4 * N * AT;
  static PerDeviceOnce once;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(adjust_kernel<N, VEC>), slice * 4, once);
  if (e != cudaSuccess) return e;
  p.slices = (int)(((long long)p.V + slice - 1) / slice);
  const long long blocks = (long long)rows * p.slices;
  if (blocks >= 1LL << 31) return cudaErrorNotSupported;
  return launch_pdl(adjust_kernel<N, VEC>, dim3((unsigned)blocks), dim3(AT), slice * 4, s, p);
}

template <int N>
cudaError_t launch_vec(const AdjustParams& p, bool vec, int rows, cudaStream_t s) {
  return vec ? launch_n<N, true>(p, rows, s) : launch_n<N, false>(p, rows, s);
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
  const uintptr_t i0 = reinterpret_cast<uintptr_t>(logits), i1 = i0 + ((size_t)(rows - 1) * ld + vocab) * 4;
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(out), o1 = o0 + ((size_t)(rows - 1) * ld_out + vocab) * 4;
  if (i0 < o1 && o0 < i1 && !(i0 == o0 && (ld == ld_out || rows == 1)))
    return set_error(SWIFTKV_EINVAL, "out overlaps logits without being them");
  AdjustParams p;
  p.logits = logits;
  p.ld = ld;
  p.out = out;
  p.ldo = ld_out;
  p.V = vocab;
  p.slices = 0;
  p.tokens = hist ? a->tokens : nullptr;
  p.ld_tokens = a->ld_tokens;
  p.max_tokens = a->max_tokens;
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
  const bool vec = ((i0 | o0) & 15) == 0 && (rows == 1 || (ld % 4 == 0 && ld_out % 4 == 0));
  // Short slices while there are few rows, so that every SM has work; long ones walk a history less often.
  const long long ids = (long long)rows * vocab;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = ids < (1 << 20) ? launch_vec<1>(p, vec, rows, s)
                        : ids < (1 << 22) ? launch_vec<2>(p, vec, rows, s)
                        : ids < (1 << 23) ? launch_vec<4>(p, vec, rows, s) : launch_vec<8>(p, vec, rows, s);
  if (e != cudaSuccess)
    return set_error(e == cudaErrorNotSupported ? SWIFTKV_EUNSUPPORTED : SWIFTKV_ECUDA, cudaGetErrorString(e));
  return SWIFTKV_OK;
}
