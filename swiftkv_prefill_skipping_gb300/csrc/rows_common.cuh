// Shared by the kernels that take the rows of short chunks as columns of mma.sync.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace skv {

// A column of q (held by the 4 lanes of a group, dims 16 ks + 4 qd .. + 3 each) as f16, times the power
// of two that takes its largest element to [2^14, 2^15), and the inverse power. Exact for elements down
// to 2^-31 of the largest (below, off by 2^-39 of it), whatever q's size, where f16 alone ends at 65504.
// ALTERNATE: a lane's dims in pairs {0, 2}, {1, 3} instead of {0, 1}, {2, 3}.
template <int D, bool ALTERNATE>
__device__ __forceinline__ void load_q_f16(const bf16* src, bool in, int qd, uint32_t (*qf)[2], float& back) {
  float top = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint2 w = in ? *reinterpret_cast<const uint2*>(src + ks * 16 + 4 * qd) : make_uint2(0u, 0u);
    qf[ks][0] = w.x;
    qf[ks][1] = w.y;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[ks][e]));
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int ex = max(__float_as_int(top) >> 23, 15);  // biased; both powers stay normal
  const float to = __int_as_float((268 - ex) << 23);
  back = __int_as_float((ex - 14) << 23);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[ks][0]));
    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[ks][1]));
    qf[ks][0] = ALTERNATE ? pack_f16(x.x * to, y.x * to) : pack_f16(x.x * to, x.y * to);
    qf[ks][1] = ALTERNATE ? pack_f16(x.y * to, y.y * to) : pack_f16(y.x * to, y.y * to);
  }
}

}  // namespace skv
