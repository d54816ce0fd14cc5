// lanes16.h -- a row of up to 256 logits held by 16 lanes (four rows a wave):
// reductions within a DPP row, and the rows' loads. Shared by the balance and the
// gate kernels.
#pragma once

#include "common.h"

namespace moeblk {

// butterfly over the 16 lanes of a DPP row: xor 1, xor 2, then the mirrors of 8 and
// 16 lanes (whose halves agree by then); every lane gets the same bits
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  return v + dpp<0x140>(v);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xb1>(v));
  v = fmaxf(v, dpp<0x4e>(v));
  v = fmaxf(v, dpp<0x141>(v));
  return fmaxf(v, dpp<0x140>(v));
}

// exp through the hardware's exp2: the argument's rounding is |x| 2^-24 relative
// in the result, the instruction's own error 1 ulp (that of the reciprocal below too;
// at 65536 x 256 the outputs are 0.95e-7 off the 64-bit ones in the 2-norm, torch's fp32
// form 1.0e-7)
__device__ __forceinline__ float exp_hw(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// A lane's columns of a row: 64 i + 4 j + c with j = lane % 16, i < kNI, c < 4.
template <int kNI>
struct Row {
  float v[4 * kNI];
};

// 16-byte loads and stores at any element (rows of any length)
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

template <int kNI>
__device__ __forceinline__ void load_row(const float* logits, size_t row, int E, int j,
                                         Row<kNI>& l) {
  const float* p = logits + row * E;
#pragma unroll
  for (int i = 0; i < kNI; ++i) {
    const int e = 64 * i + 4 * j;
    f32x4_t q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (e + 4 <= E) {
      q = *reinterpret_cast<const f32x4_any_t*>(p + e);
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (e + c < E) q[c] = p[e + c];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) l.v[4 * i + c] = q[c];
  }
}

}  // namespace moeblk
