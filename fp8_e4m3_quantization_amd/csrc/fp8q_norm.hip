// fp8q_norm.hip -- the two steps between a layer's products: the residual's addition with the RMS
// norm before a projection, and the SiLU of the gate times the up projection before the next, each
// written as the E4M3 codes and 1x128 group scales that the products read.
//
// Mathematics, per row of k values (all in binary32):
//   norm:  h = bf16(x + residual) (without a residual: x),  y = h w / sqrt(mean(h^2) + eps)
//   silu:  y = gate / (1 + exp(-gate)) * up
// and per group of 128 of the row: s = max(max|y|, 1e-10) / 448, codes = E4M3(y / s).  h is what
// the layer keeps, so it is rounded first and normed as kept; y is not rounded before it is
// quantized.  The quotient is a binary32 division's: reciprocal and one remainder correction (see
// fp8q_math.h, which has that for binary32 dividends too).
//
// Eight lanes take a group, 16 values each, as in fp8_group_quant: two 16-byte loads of each input,
// one 16-byte store of codes, the maximum over eight lanes without LDS.
//
// What bounds them: memory for many rows (4593 x 5120 with a residual: 34.3 us, 165 MB at 4.8 TB/s, 94 % of a
// copy's rate; 4593 x 16384 of gate and up: 63.7 us, 379 MB at 5.9 TB/s, reads outweighing writes), the
// host's call for few (16 x 5120: 7.3 us, 3.8 on the GPU; 16 x 16384 of gate and up 6.4 and 4.1).  A row is a
// workgroup's, so that its squares' sum needs one barrier and its values stay in registers; a workgroup
// that goes on to further rows instead of ending took 37.9 us for the 34.6 of then.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_device.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));

constexpr int kLaneValues = 16;

__device__ __forceinline__ void unpack8(uint4 w, float* f) {
  f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                    cvt_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void store16(uint16_t* p, const uint4& v) {
  __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
}

// A lane's 16 values of a group: their codes, and the group's scale from its first lane.
__device__ __forceinline__ void put_group(const float* y, uint8_t* q, float* scale, bool first) {
  float amax = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < kLaneValues; ++i) amax = fmaxf(amax, fabsf(y[i]));
  amax = max_over_8_lanes(amax);
  // an IEEE division: y is no bf16 value, so that the shortcut for those does not hold
  const float s = fmaxf(amax, kAmaxFloor) / kE4M3Max;
  const float inv = 1.0f / s;
  // An infinite maximum: finite values over it are 0, infinite ones NaN, as by division; the
  // remainder's product must not make NaN of the former.
  const float sf = fminf(s, 3.402823466e38f);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x4<false>(div_by_scale(y[4 * i], sf, inv), div_by_scale(y[4 * i + 1], sf, inv),
                         div_by_scale(y[4 * i + 2], sf, inv), div_by_scale(y[4 * i + 3], sf, inv));
  __builtin_nontemporal_store(v4u{w[0], w[1], w[2], w[3]}, reinterpret_cast<v4u*>(q));
  if (first) *scale = s;
}

struct NormArgs {
  const uint16_t *x, *residual, *weight;
  uint16_t *sum, *kept;  // residual_out, norm_out or NULL
  uint8_t* q;
  float* scales;
  int64_t rows, xs, rs, ss, ks;
  int k;
  float eps;
};

__device__ __forceinline__ float sum_over_wave(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Sum over the workgroup; `parity` alternates from call to call, so that one barrier suffices.
__device__ __forceinline__ float sum_over_group(float v, int parity) {
  __shared__ float s_sum[2][16];
  v = sum_over_wave(v);
  const int waves = (blockDim.x + 63) >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) s_sum[parity][threadIdx.x >> 6] = v;
  __syncthreads();
  float all = 0.0f;
  for (int w = 0; w < waves; ++w) all += s_sum[parity][w];
  return all;
}

// A lane's 16 values of a row from column c on: h, stored where a residual is added.
__device__ __forceinline__ void load_sum(const NormArgs& a, int64_t row, int c, uint4* h) {
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.xs + c);
  h[0] = load16_nt(x);
  h[1] = load16_nt(x + 1);
  if (!a.residual) return;
  const uint4* r = reinterpret_cast<const uint4*>(a.residual + row * a.rs + c);
  const uint4 r0 = load16_nt(r), r1 = load16_nt(r + 1);
  float f[16], g[16];
  unpack8(h[0], f); unpack8(h[1], f + 8);
  unpack8(r0, g); unpack8(r1, g + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] += g[i];
  h[0] = pack8(f);
  h[1] = pack8(f + 8);
  store16(a.sum + row * a.ss + c, h[0]);
  store16(a.sum + row * a.ss + c + 8, h[1]);
}

__device__ __forceinline__ float sq_sum16(const uint4* h) {
  float f[16];
  unpack8(h[0], f); unpack8(h[1], f + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= f[i];
#pragma unroll
  for (int n = 8; n >= 1; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) f[i] += f[i + n];
  return f[0];
}

__device__ __forceinline__ void put_normed(const NormArgs& a, int64_t row, int c, const uint4* h,
                                           const uint4* w, float r) {
  float y[16], f[16];
  unpack8(h[0], y); unpack8(h[1], y + 8);
  unpack8(w[0], f); unpack8(w[1], f + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = y[i] * r * f[i];
  if (a.kept) {
    store16(a.kept + row * a.ks + c, pack8(y));
    store16(a.kept + row * a.ks + c + 8, pack8(y + 8));
  }
  put_group(y, a.q + row * a.k + c, a.scales + row * (a.k / 128) + c / 128, (threadIdx.x & 7) == 0);
}

__device__ __forceinline__ void load_weight(const NormArgs& a, int c, uint4* w) {
  w[0] = w[1] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  if (a.weight) {
    w[0] = *reinterpret_cast<const uint4*>(a.weight + c);
    w[1] = *reinterpret_cast<const uint4*>(a.weight + c + 8);
  }
}

// One workgroup per row, which stays in registers: kPieces times 16 values a lane.  (Two pieces leave
// the weight no registers; it comes from the L2 again.)
template <int kPieces>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
  const int step = blockDim.x * kLaneValues;
  int parity = 0;
  uint4 w[kPieces][2];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = p * step + threadIdx.x * kLaneValues;
    if (kPieces == 1 && c < a.k) load_weight(a, c, w[p]);
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    uint4 h[kPieces][2];
    float sq = 0.0f;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = p * step + threadIdx.x * kLaneValues;
      if (c < a.k) {
        load_sum(a, row, c, h[p]);
        sq += sq_sum16(h[p]);
      }
    }
    const float r = rsqrtf(sum_over_group(sq, parity) / float(a.k) + a.eps);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = p * step + threadIdx.x * kLaneValues;
      if (c < a.k) {
        if (kPieces > 1) load_weight(a, c, w[p]);
        put_normed(a, row, c, h[p], w[p], r);
      }
    }
  }
}

// Rows longer than that: read twice, the second time as stored where a residual was added.  A lane
// reads again what it wrote itself.  Columns count in 32 bits without a sign: behind the last ones of rows of
// nearly 2^31 values lies a column past 2^31.
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a) {
  const uint32_t step = blockDim.x * kLaneValues, k = a.k;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    float sq = 0.0f;
    for (uint32_t c = threadIdx.x * kLaneValues; c < k; c += step) {
      uint4 h[2];
      load_sum(a, row, c, h);
      sq += sq_sum16(h);
    }
    const float r = rsqrtf(sum_over_group(sq, parity) / float(a.k) + a.eps);
    for (uint32_t c = threadIdx.x * kLaneValues; c < k; c += step) {
      uint4 h[2], w[2];
      const uint16_t* from = a.residual ? a.sum + row * a.ss + c : a.x + row * a.xs + c;
      h[0] = *reinterpret_cast<const uint4*>(from);
      h[1] = *reinterpret_cast<const uint4*>(from + 8);
      load_weight(a, c, w);
      put_normed(a, row, c, h, w, r);
    }
  }
}

struct SiluArgs {
  const uint16_t *gate, *up;
  uint16_t* out;  // or NULL
  uint8_t* q;
  float* scales;
  int64_t gs, us, os;
  uint32_t groups;
  FastDiv per_row;  // groups of a row
};

constexpr int kSiluBlock = 512;  // (256 and 1024 threads: within 2 %)
constexpr int kSiluGroups = kSiluBlock / 8;

__global__ __launch_bounds__(kSiluBlock) void silu_kernel(const SiluArgs a) {
  const uint32_t stride = gridDim.x * kSiluGroups;
  const int sub = threadIdx.x & 7;
  for (uint32_t g = blockIdx.x * kSiluGroups + (threadIdx.x >> 3); g < a.groups; g += stride) {
    const uint32_t row = a.per_row.div(g);
    const int c = int(g - row * a.per_row.d) * 128 + sub * kLaneValues;
    const uint4* gp = reinterpret_cast<const uint4*>(a.gate + int64_t(row) * a.gs + c);
    const uint4* up = reinterpret_cast<const uint4*>(a.up + int64_t(row) * a.us + c);
    const uint4 g0 = load16_nt(gp), g1 = load16_nt(gp + 1);
    const uint4 u0 = load16_nt(up), u1 = load16_nt(up + 1);
    float y[16], u[16];
    unpack8(g0, y); unpack8(g1, y + 8);
    unpack8(u0, u); unpack8(u1, u + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // the argument is rounded once: e is off by 2 |gate| 2^-24 of itself, which codes of 2^-4 do not show
      const float e = __builtin_amdgcn_exp2f(y[i] * -kLog2e);
      y[i] = y[i] * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
    }
    if (a.out) {
      store16(a.out + int64_t(row) * a.os + c, pack8(y));
      store16(a.out + int64_t(row) * a.os + c + 8, pack8(y + 8));
    }
    put_group(y, a.q + int64_t(g) * 128 + sub * kLaneValues, a.scales + g, sub == 0);
  }
}

// What both calls check of their rows: k whole groups, fewer than 2^31 groups, strides.
bool rows_ok(int64_t m, int32_t k) {
  return m >= 0 && k > 0 && k % 128 == 0 && m <= ((int64_t(1) << 31) - 1) / (k / 128);
}
bool stride_ok(int64_t stride, int32_t k) { return stride >= k && stride <= (int64_t(1) << 40); }

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int fp8_rms_norm_group_quant(const uint16_t* x, const uint16_t* residual,
                                        const uint16_t* weight, float eps, uint16_t* residual_out,
                                        uint16_t* norm_out, uint8_t* q, float* scales, int64_t m,
                                        int32_t k, int64_t x_stride, int64_t residual_stride,
                                        int64_t residual_out_stride, int64_t norm_out_stride,
                                        hipStream_t stream) {
  if (!rows_ok(m, k) || !(eps >= 0.0f && eps <= 1.0f) || !stride_ok(x_stride, k)) return FP8Q_EINVAL;
  if (residual && (!stride_ok(residual_stride, k) || !stride_ok(residual_out_stride, k)))
    return FP8Q_EINVAL;
  if ((norm_out && !stride_ok(norm_out_stride, k)) || (residual_out && !residual)) return FP8Q_EINVAL;
  if (m == 0) return FP8Q_OK;
  if (!x || !q || !scales || (residual && !residual_out)) return FP8Q_ENULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(residual_out, 16) || !aligned(norm_out, 16) || !aligned(q, 16) ||
      !aligned(scales, 4) || x_stride % 8 ||
      (residual && (residual_stride % 8 || residual_out_stride % 8)) ||
      (norm_out && norm_out_stride % 8))
    return FP8Q_EALIGN;
  NormArgs a = {};
  a.x = x, a.residual = residual, a.weight = weight, a.sum = residual_out, a.kept = norm_out;
  a.q = q, a.scales = scales, a.rows = m, a.xs = x_stride, a.rs = residual_stride;
  a.ss = residual_out_stride, a.ks = norm_out_stride, a.k = k, a.eps = eps;
  // Up to 8192 columns one piece a lane, beyond that two: three workgroups a compute unit instead of
  // two of 1024 threads (517 rows of 16384, without a residual, bf16 rows kept: 12.0 us, 13.8 with one).
  const int lanes = (k / kLaneValues + 63) / 64 * 64, halves = (k / 2 / kLaneValues + 63) / 64 * 64;
  const int threads = lanes <= 512 ? lanes : halves <= 1024 ? halves : 1024;
  const unsigned blocks = unsigned(clamp_grid(m));
  auto kern = lanes <= 512 ? norm_kernel<1> : halves <= 1024 ? norm_kernel<2> : norm_long_kernel;
  launch(kern, dim3(blocks), dim3(unsigned(threads)), 0, stream, a);
  return launch_status();
}

extern "C" int fp8_silu_mul_group_quant(const uint16_t* gate, const uint16_t* up, uint16_t* out,
                                        uint8_t* q, float* scales, int64_t m, int32_t k,
                                        int64_t gate_stride, int64_t up_stride, int64_t out_stride,
                                        hipStream_t stream) {
  if (!rows_ok(m, k) || !stride_ok(gate_stride, k) || !stride_ok(up_stride, k) ||
      (out && !stride_ok(out_stride, k)))
    return FP8Q_EINVAL;
  if (m == 0) return FP8Q_OK;
  if (!gate || !up || !q || !scales) return FP8Q_ENULL;
  if (!aligned(gate, 16) || !aligned(up, 16) || !aligned(out, 16) || !aligned(q, 16) ||
      !aligned(scales, 4) || gate_stride % 8 || up_stride % 8 || (out && out_stride % 8))
    return FP8Q_EALIGN;
  SiluArgs a = {};
  a.gate = gate, a.up = up, a.out = out, a.q = q, a.scales = scales;
  a.gs = gate_stride, a.us = up_stride, a.os = out_stride;
  a.per_row = FastDiv(uint32_t(k / 128));
  a.groups = uint32_t(m * (k / 128));
  const int64_t blocks = clamp_grid((int64_t(a.groups) + kSiluGroups - 1) / kSiluGroups);
  launch(silu_kernel, dim3(unsigned(blocks)), dim3(kSiluBlock), 0, stream, a);
  return launch_status();
}
