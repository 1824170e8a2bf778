// fp8q_attn_tile.h -- the steps of attention over a tile of bf16 keys and values in LDS, for a wave
// that owns 32 query rows: lane l has row l % 32, half l / 32 of the keys of every score tile.
#pragma once
#include "fp8q_attn.h"

namespace fp8q {

constexpr int kTileKeys = 64;
constexpr int kWaveRows = 32;
constexpr float kFar = 0x1p27f;  // a reference whose rounding (2^3) still leaves weights their range

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Order of the 16-byte chunks within a row of a tile in LDS.  K is read 16 rows at a time, one
// chunk each; V (transposing read) four rows at a time, 64 bytes each: both then touch every bank
// once.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return D == 64 ? c ^ ((row >> 1) & 7) : c ^ (row & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 64 ? c ^ (((row >> 1) & 1) << 2) : c ^ ((row & 3) << 2);
}

// S^T of a tile: s[b] holds keys 32 b .. 32 b + 31.
template <int D>
__device__ __forceinline__ void tile_scores(v16f* s, const uint16_t* kt, const v8bf* qf) {
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
#pragma unroll
  for (int st = 0; st < D / 16; ++st)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r = 32 * b + col;
      const v8bf kf = __builtin_bit_cast(
          v8bf, *reinterpret_cast<const uint4*>(kt + r * D + k_chunk<D>(r, 2 * st + half) * 8));
      s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st], s[b], 0, 0, 0);
    }
}

// V^T of 16 keys (step st of the tile) and 32 values (block i), in the order of the weights.
template <int D>
__device__ __forceinline__ v4u value_frag(const uint16_t* vt, int st, int i) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int i16 = lane & 15, side = (lane >> 4) & 1;
  const int ra = 16 * st + 4 * half + (i16 >> 2), c = 4 * i + 2 * side + ((i16 & 3) >> 1);
  const int within = 4 * (i16 & 1);
  const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4s*)(vt + ra * D + v_chunk<D>(ra, c) * 8 + within)));
  const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4s*)(vt + (ra + 8) * D + v_chunk<D>(ra + 8, c) * 8 + within)));
  return v4u{lo[0], lo[1], hi[0], hi[1]};
}

// The largest of kBlocks times 32 scores of a row, before their scale.
template <int kBlocks>
__device__ __forceinline__ float largest_score(const v16f* s) {
  float top = neg_inf();
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
  return max_over_halves(top);
}

// A row's running softmax: the sum of weighted values o^T, the reference that weights are taken
// against (log2 units), this half's sum of weights, and their sum as rounded to bf16 for the product
// with the values (summed by products of ones with 16 blocks of 4x4, in which every lane has a
// column of its own, so that a NaN stays with its row; the sum comes four times).
template <int D>
struct RowSums {
  // The rare branch that goes with a fused product costs 256-wide heads registers that they do not
  // have.
  static constexpr bool kFused = D < 256;
  v16f o[D / 32];
  float ref, sum;
  v4f rounded;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    ref = neg_inf();
    sum = 0.0f;
    rounded = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // The reference for scores s, whose largest is top (log2 units).  Returns what weights subtract.
  // Where s * scale - ref is one fused product it is exact but for its last rounding, while ref is
  // rounded: by up to 2^-24 of itself, which every weight of a row shares.  Beyond kFar that could
  // leave binary32's range of exponents; there the products are rounded too, so that the largest
  // weight is 1 again.
  template <int kBlocks>
  __device__ __forceinline__ float move_to(float top, v16f* s, float scale) {
    const bool moves = top > ref + kSoftmaxSlack;
    if (__any(moves)) {
      const float f = moves ? __builtin_amdgcn_exp2f(ref - top) : 1.0f;
      ref = moves ? top : ref;
      sum *= f;
      rounded *= f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= f;
    }
    const float base = ref == neg_inf() ? 0.0f : ref;
    if (kFused && __any(__builtin_fabsf(base) > kFar)) {
      const float back = 1.0f / scale;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = (s[b][r] * scale - base) * back;
      return 0.0f;
    }
    return base;
  }
  static __device__ __forceinline__ float weight(float s, float scale, float base) {
    return __builtin_amdgcn_exp2f(kFused ? __builtin_fmaf(s, scale, -base) : s * scale - base);
  }
  // Weights of 16 keys (half `h` of a block of scores) as the second product's operand.
  __device__ __forceinline__ v8bf weights(const v16f& s, int h, float scale, float base) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float x = weight(s[8 * h + e], scale, base), y = weight(s[8 * h + e + 1], scale, base);
      sum += x + y;
      w[e / 2] = cvt_bf16x2(x, y);
    }
    const v4s ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[0], w[1]}), rounded, 0, 0, 0);
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[2], w[3]}), rounded, 0, 0, 0);
    return __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
  }
  __device__ __forceinline__ void add_values(const uint16_t* vt, int st, v8bf p) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, value_frag<D>(vt, st, i)), p,
                                                     o[i], 0, 0, 0);
  }
};

}  // namespace fp8q
