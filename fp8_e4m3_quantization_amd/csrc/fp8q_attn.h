// fp8q_attn.h -- what the attention kernels share: vector types, lane exchanges, and the search
// for a workgroup's piece of work in a batch whose lengths only the device knows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q_device.h"

namespace fp8q {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

// Sequences of a call.  Every workgroup looks for its own piece among all lengths, 64 at a time, so
// that the search grows with the square of their number: one-token sequences of 40 heads take 1.5 ms
// (prompts) and 0.4 ms (steps) at 2048, 14 and 6 ms at 8192, and would take minutes at 2^20.
constexpr int kMostSeqs = 1 << 16;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// A running reference of a softmax moves only when a score exceeds it by more than this many
// powers of two: exp2 of what lies above it then reaches at most 2^8, far inside binary32, and
// the sums need no rescaling in between (any reference gives the same quotient).
constexpr float kSoftmaxSlack = 8.0f;

// A pair of values combined over lanes l and l ^ 32 (l ^ 16): the swap leaves one half's (row's)
// value in each of the two results, in every lane.
__device__ __forceinline__ float max_over_halves(float v) {
  const v2u r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const v2u r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_over_rows(float v) {
  const v2u r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_over_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  const v2u r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return sum_over_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Inclusive prefix sum over the wave: within rows of 16 lanes, then across them.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xF, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

}  // namespace fp8q
