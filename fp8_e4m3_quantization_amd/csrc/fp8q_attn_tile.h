// fp8q_attn_tile.h -- the steps of attention over E4M3 keys and values in LDS, for a wave that owns 32
// query rows: lane l has row l % 32, half l / 32 of the keys of every 32.
#pragma once
#include "fp8q_attn.h"

namespace fp8q {

// The lane's number as the compiler may not know it: addresses made of it are not shared with other
// code, where they would take registers from the loops between.
__device__ __forceinline__ int own_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

constexpr int kTileKeys = 64;
constexpr int kWaveRows = 32;
constexpr float kFar = 0x1p27f;  // a reference whose rounding (2^3) still leaves weights their range

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

// Order of the 16-byte chunks within a row of codes in LDS: the place of chunk c of row r is
// c ^ key_turn(r), or value_turn(r).  Keys are read eight rows at a time, values rows 0..3 and 8..11
// of 16 (or the others) at a time: each then touches every bank once.
template <int D>
__device__ __forceinline__ int key_turn(int r) { return D == 64 ? (r >> 1) & 3 : r & 7; }
template <int D>
__device__ __forceinline__ int value_turn(int r) {
  return D == 64 ? ((r >> 1) & 1) | ((r >> 2) & 2) : (r & 3) | ((r >> 1) & 4);
}

__device__ __forceinline__ v8bf e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(v8bf, v4u{e4m3x2_to_bf16<false>(lo), e4m3x2_to_bf16<true>(lo),
                                      e4m3x2_to_bf16<false>(hi), e4m3x2_to_bf16<true>(hi)});
}

// Codes of 32 keys (block b of those in LDS), values 32 c + 16 half .. + 15.
template <int D>
__device__ __forceinline__ uint4 key_codes(const uint8_t* ks, int c, int b, int lane) {
  const int col = lane & 31, half = lane >> 5;
  return *reinterpret_cast<const uint4*>(ks + (32 * b + col) * D + ((2 * c + half) ^ key_turn<D>(col)) * 16);
}

// S^T of 32 kBlocks keys whose codes lie in LDS; the queries' fragments 2 c and 2 c + 1 hold values
// 32 c + 16 half .. + 7 and + 8 .. + 15.
template <int D, int kBlocks>
__device__ __forceinline__ void code_scores(v16f* s, const uint8_t* ks, const v8bf* qf, int lane) {
  uint4 x[D / 32][kBlocks];
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) x[c][b] = key_codes<D>(ks, c, b, lane);
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(x[c][b].x, x[c][b].y), qf[2 * c], s[b], 0, 0, 0);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(x[c][b].z, x[c][b].w), qf[2 * c + 1], s[b], 0, 0, 0);
  }
}

// Codes of V^T of 16 keys (step st of those in LDS) and 32 values (block i): keys 4h..4h+3 and
// 8+4h..8+4h+3 for lane half h, the order in which the lane holds their scores.
template <int D>
__device__ __forceinline__ v2u value_codes(const uint8_t* vs, int st, int i, int lane) {
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  const int half = lane >> 5, i16 = lane & 15, side = (lane >> 4) & 1;
  const int r = 4 * half + ((i16 >> 1) & 3) + 8 * (i16 >> 3);
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
      (lds_v2i*)(vs + (16 * st + r) * D + ((2 * i + side) ^ value_turn<D>(r)) * 16 + 8 * (i16 & 1))));
}

// NaN codes of w become 0; their bytes' top bits are added to `odd`.
__device__ __forceinline__ uint32_t without_nans(uint32_t w, uint32_t* odd) {
  const uint32_t nan = e4m3_nan_bytes(w);
  *odd |= nan;
  return w & ~((nan >> 7) * 0xFFu);
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
    const bool is_far = __builtin_fabsf(base) > kFar;
    if (kFused && __any(is_far)) {  // (rows that are not keep their bits)
      const float back = 1.0f / scale;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = is_far ? (s[b][r] * scale - base) * back : s[b][r];
      return is_far ? 0.0f : base;
    }
    return base;
  }
  static __device__ __forceinline__ float weight(float s, float scale, float base) {
    return __builtin_amdgcn_exp2f(kFused ? __builtin_fmaf(s, scale, -base) : s * scale - base);
  }
  // Weights of the scores as the second product's operands, 16 keys each; returns their sum.
  template <int kBlocks>
  static __device__ __forceinline__ float weights_of(const v16f* s, float scale, float base, v8bf* p) {
    float t = 0.0f;
#pragma unroll
    for (int st = 0; st < 2 * kBlocks; ++st) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x = weight(s[st >> 1][8 * (st & 1) + e], scale, base);
        const float y = weight(s[st >> 1][8 * (st & 1) + e + 1], scale, base);
        t += x + y;
        w[e / 2] = cvt_bf16x2(x, y);
      }
      p[st] = __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
    }
    return t;
  }
  // The weights of 32 kBlocks keys (scores of keys not seen: -infinity), against a reference that is
  // at most 2^kSoftmaxSlack below the largest of them.  Looking for the largest score only where the weights
  // come too large saves 2 % of the time, but lets references lag: the error of 64 rows over
  // 100003 positions then is 1.4 times that of weights in binary32, and 1.23 times as it is here.
  template <int kBlocks>
  __device__ __forceinline__ void weigh(v16f* s, float scale, v8bf* p) {
    const float base = move_to<kBlocks>(largest_score<kBlocks>(s) * scale, s, scale);
    sum += weights_of<kBlocks>(s, scale, base, p);
  }
  // o^T += V^T P^T over 16 keys, whose values' codes are y.  With kClean NaN codes are left out, and
  // `odd` tells of those of the keys that count (one bit for each of the lane's eight).
  template <bool kClean>
  __device__ __forceinline__ void add_values(const v2u* y, v8bf p, uint32_t counts, uint32_t* odd) {
    const v4s ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
    const v4u w = __builtin_bit_cast(v4u, p);
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[0], w[1]}), rounded, 0, 0, 0);
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[2], w[3]}), rounded, 0, 0, 0);
    uint32_t odd0 = 0, odd1 = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v2u c = y[i];
      if (kClean) c = v2u{without_nans(c[0], &odd0), without_nans(c[1], &odd1)};
      o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(c[0], c[1]), p, o[i], 0, 0, 0);
    }
    // (four bits times this product: bit k is bit 8 k + 7, and others that no NaN code sets)
    if (kClean) *odd |= (odd0 & ((counts & 15) * 0x10204080u)) | (odd1 & ((counts >> 4 & 15) * 0x10204080u));
  }
};

}  // namespace fp8q
