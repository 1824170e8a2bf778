// fp8q_rope.hip -- the step between the QKV projection and the paged cache: RMS norm of each
// query and key head, rotary positions, and the E4M3 write of K and V, in one pass.
//
// Mathematics, per head row x of D values at position p (all in binary32):
//   n_i = x_i * w_i / sqrt(mean(x^2) + eps)          (w absent: n = x)
//   (y_a, y_b) = (n_a c - n_b s, n_b c + n_a s)      for each pair (a, b) of the first R values
//   with c, s the table's cosine and sine of the pair at p; pairs are (i, i + R/2), or (2i, 2i+1)
//   interleaved; values R..D-1 pass.
// y is rounded once, to bf16.  The cache's K codes are made of that bf16 value, not of the
// binary32 one: a calibration window stages bf16 rows and replays them, and the live write has
// to leave the bytes the replay would.
//
// Bound: memory.  Each input is read once and each output written once: 4593 tokens of 40 + 4 + 4
// 128-wide heads, 110.6 MB, in 26.5 us (4.2 TB/s, 80 % of a plain copy's rate; the vector ALUs are
// busy 72 % of that time).  16 tokens: 4.7 us, a chain of three loads behind a launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_device.h"
#include "fp8q_kv_internal.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

struct RopeArgs {
  const uint16_t *q, *k, *v;   // rows of qs / ks / vs elements
  const uint16_t *qw, *kw;     // [D] or NULL
  const int64_t* positions;    // NULL: no rotation
  const float* cos_sin;        // [npos, rot]: rot/2 cosines, then rot/2 sines
  const int64_t* slots;        // NULL: no cache write
  uint16_t *q_out, *k_out;     // k_out may be NULL
  uint8_t *k_cache, *v_cache;
  int64_t npos, tokens, qs, ks, vs, qos, kos, nslots, cs;
  int rot, hq, hkv, d, bs;
  float eps, k_scale, k_inv, v_scale, v_inv;
};

// p[i] for an index that is the same in the whole wave, through the scalar cache: the lists of
// positions and slots are only read.
__device__ __forceinline__ int64_t uniform_at(const int64_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int64_t* constant_i64;
  return ((constant_i64)p)[i];
}

// Where token t's row lies in the pools (elements from their start), or -1: no such slot.
__device__ __forceinline__ int64_t pool_row(const RopeArgs& a, int64_t t) {
  if (!a.slots) return -1;
  const int64_t slot = uniform_at(a.slots, t);
  if (slot < 0 || slot >= a.nslots) return -1;
  const int64_t e = int64_t(a.hkv) * a.d;
  if (a.nslots <= 0x7FFFFFFF) {  // 32-bit division
    const uint32_t b = uint32_t(slot) / uint32_t(a.bs);
    return int64_t(b) * a.cs + int64_t(uint32_t(slot) - b * uint32_t(a.bs)) * e;
  }
  return slot / a.bs * a.cs + slot % a.bs * e;
}

__device__ __forceinline__ float sq_sum8(uint4 w) {
  const float a = bf16_lo(w.x), b = bf16_hi(w.x), c = bf16_lo(w.y), d = bf16_hi(w.y);
  const float e = bf16_lo(w.z), f = bf16_hi(w.z), g = bf16_lo(w.w), h = bf16_hi(w.w);
  return ((a * a + b * b) + (c * c + d * d)) + ((e * e + f * f) + (g * g + h * h));
}

__device__ __forceinline__ void unpack8(uint4 w, float* f) {
  f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

// 16-byte store with the non-temporal hint: what is written here is not read again here.
__device__ __forceinline__ void store16_nt(uint4 v, uint16_t* p) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
}

// Sum over each aligned group of 2^kLanesLog2 lanes, in every lane of it.
template <int kLanesLog2>
__device__ __forceinline__ float sum_over_lanes(float v) {
  v += dpp<0xB1>(v);                           // lane ^ 1
  v += dpp<0x4E>(v);                           // lane ^ 2
  if constexpr (kLanesLog2 >= 3) v += dpp<0x141>(v);  // mirror within 8 lanes
  if constexpr (kLanesLog2 >= 4) v += dpp<0x140>(v);  // mirror within 16
  if constexpr (kLanesLog2 >= 5) v += __shfl_xor(v, 16);
  if constexpr (kLanesLog2 >= 6) v += __shfl_xor(v, 32);
  return v;
}

// One workgroup per token.  L = D/8 lanes (a power of two) take a head, 8 values each, so a
// lane loads its head chunk in one 16-byte load, a head's mean square is a reduction over
// L neighbouring lanes, and the pair partner of a lane's chunk in the half layout is the chunk
// of the lane rot/16 away, exchanged as bf16 (four words) and normed by both lanes.  A lane keeps
// its cosines, sines and weights for every head of the token, and issues the loads of up to four
// heads before the table's, whose address waits for the position.
constexpr int kRopeAhead = 4;

template <int kLanesLog2, bool kInterleaved>
__global__ __launch_bounds__(1024) void rope_vec_kernel(const RopeArgs a) {
  constexpr int kLanes = 1 << kLanesLog2;
  constexpr int kD = 8 * kLanes;
  const int c = threadIdx.x & (kLanes - 1);
  const int g = threadIdx.x >> kLanesLog2;
  const int ng = blockDim.x >> kLanesLog2;
  const int heads = a.hq + a.hkv + (a.slots ? a.hkv : 0);
  const bool turns = 8 * c < a.rot;
  const int reach = a.rot >> 4;                       // lanes between a pair's chunks
  const bool second = !kInterleaved && c >= reach;    // this chunk holds the pairs' b
  const int partner = turns ? (second ? c - reach : c + reach) : c;
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int64_t pos = a.rot ? uniform_at(a.positions, t) : 0;
    uint4 x[kRopeAhead];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        const int h = h0 + u * ng;
        if (h >= heads) continue;
        const uint16_t* src = h < a.hq ? a.q + t * a.qs + int64_t(h) * kD
                            : h < a.hq + a.hkv ? a.k + t * a.ks + int64_t(h - a.hq) * kD
                                               : a.v + t * a.vs + int64_t(h - a.hq - a.hkv) * kD;
        x[u] = load16_nt(reinterpret_cast<const uint4*>(src) + c);
      }
    };
    load(g);
    uint4 qw = ones, kw = ones, qwp = ones, kwp = ones;
    if (a.qw) {
      qw = reinterpret_cast<const uint4*>(a.qw)[c];
      if constexpr (!kInterleaved) qwp = reinterpret_cast<const uint4*>(a.qw)[partner];
    }
    if (a.kw) {
      kw = reinterpret_cast<const uint4*>(a.kw)[c];
      if constexpr (!kInterleaved) kwp = reinterpret_cast<const uint4*>(a.kw)[partner];
    }
    if (a.rot && (pos < 0 || pos >= a.npos)) continue;
    const int64_t row = pool_row(a, t);
    float cs[8] = {}, sn[8] = {};
    if (turns) {
      const int f0 = kInterleaved ? 4 * c : 8 * (second ? c - reach : c);
      const float* p = a.cos_sin + pos * a.rot + f0;
      const float* ps = p + (a.rot >> 1);
#pragma unroll
      for (int i = 0; i < (kInterleaved ? 4 : 8); i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(p + i);
        const float4 w = *reinterpret_cast<const float4*>(ps + i);
        cs[i] = u.x; cs[i + 1] = u.y; cs[i + 2] = u.z; cs[i + 3] = u.w;
        sn[i] = w.x; sn[i + 1] = w.y; sn[i + 2] = w.z; sn[i + 3] = w.w;
      }
    }
    if constexpr (!kInterleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = second ? sn[i] : -sn[i];
    }
    for (int h0 = g; h0 < heads; h0 += kRopeAhead * ng) {
      if (h0 != g) load(h0);
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        const int h = h0 + u * ng;
        if (h >= heads) continue;
        if (h >= a.hq + a.hkv) {
          if (row >= 0)
            *reinterpret_cast<uint2*>(a.v_cache + row + int64_t(h - a.hq - a.hkv) * kD + 8 * c) =
                quant8<false>(x[u], a.v_scale, a.v_inv);
          continue;
        }
        const bool isq = h < a.hq;
        float r = 1.0f;
        if (isq ? a.qw != nullptr : a.kw != nullptr)
          r = rsqrtf(sum_over_lanes<kLanesLog2>(sq_sum8(x[u])) * (1.0f / float(kD)) + a.eps);
        float n[8], w[8], y[8];
        unpack8(x[u], n);
        unpack8(isq ? qw : kw, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = n[i] * r * w[i];
        if constexpr (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            y[i] = turns ? n[i] * cs[i / 2] - n[i + 1] * sn[i / 2] : n[i];
            y[i + 1] = turns ? n[i + 1] * cs[i / 2] + n[i] * sn[i / 2] : n[i + 1];
          }
        } else {
          float o[8], wp[8];
          const uint4 other = make_uint4(__shfl(x[u].x, partner, kLanes), __shfl(x[u].y, partner, kLanes),
                                         __shfl(x[u].z, partner, kLanes), __shfl(x[u].w, partner, kLanes));
          unpack8(other, o);
          unpack8(isq ? qwp : kwp, wp);
          // beyond the rotated part the value itself comes out: a product with 0 would turn an
          // infinity into NaN
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = turns ? n[i] * cs[i] + (o[i] * r * wp[i]) * sn[i] : n[i];
        }
        const uint4 out = make_uint4(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]),
                                     cvt_bf16x2(y[4], y[5]), cvt_bf16x2(y[6], y[7]));
        if (isq) {
          store16_nt(out, a.q_out + t * a.qos + int64_t(h) * kD + 8 * c);
        } else {
          const int64_t at = int64_t(h - a.hq) * kD + 8 * c;
          if (a.k_out) *reinterpret_cast<uint4*>(a.k_out + t * a.kos + at) = out;
          if (row >= 0)
            *reinterpret_cast<uint2*>(a.k_cache + row + at) =
                quant8<false>(out, a.k_scale, a.k_inv);
        }
      }
    }
  }
}

__device__ __forceinline__ uint8_t e4m3_of(uint16_t x, float s, float inv) {
  const float v = clip448(div_by_scale_clipped(bf16_to_f32(x), s, inv));
  return uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false) & 0xFF);
}

// Any head width, rotated part, stride and alignment: one wave per head row.  A lane reads and
// writes both values of a pair, so an output may lie on its input.
constexpr int kRopeRows = 4;
__global__ __launch_bounds__(64 * kRopeRows) void rope_scalar_kernel(const RopeArgs a,
                                                                     int interleaved) {
  const int heads = a.hq + a.hkv + (a.slots ? a.hkv : 0);
  const int lane = threadIdx.x, half = a.rot / 2;
  const int64_t items = a.tokens * heads;
  for (int64_t it = int64_t(blockIdx.x) * kRopeRows + threadIdx.y; it < items;
       it += int64_t(gridDim.x) * kRopeRows) {
    const int64_t t = it / heads;
    const int h = int(it - t * heads);
    const int64_t pos = a.rot ? a.positions[t] : 0;
    if (a.rot && (pos < 0 || pos >= a.npos)) continue;
    const int64_t row = pool_row(a, t);
    if (h >= a.hq + a.hkv) {
      const int64_t at = int64_t(h - a.hq - a.hkv) * a.d;
      if (row >= 0)
        for (int i = lane; i < a.d; i += 64)
          a.v_cache[row + at + i] = e4m3_of(a.v[t * a.vs + at + i], a.v_scale, a.v_inv);
      continue;
    }
    const bool isq = h < a.hq;
    const int64_t at = int64_t(isq ? h : h - a.hq) * a.d;
    const uint16_t* x = (isq ? a.q + t * a.qs : a.k + t * a.ks) + at;
    uint16_t* out = isq ? a.q_out + t * a.qos + at : a.k_out ? a.k_out + t * a.kos + at : nullptr;
    const uint16_t* w = isq ? a.qw : a.kw;
    float r = 1.0f;
    if (w) {
      float sq = 0.0f;
      for (int i = lane; i < a.d; i += 64) {
        const float f = bf16_to_f32(x[i]);
        sq += f * f;
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) sq += __shfl_xor(sq, o);
      r = rsqrtf(sq / float(a.d) + a.eps);
    }
    auto normed = [&](int i) {
      const float f = bf16_to_f32(x[i]);
      return w ? f * r * bf16_to_f32(w[i]) : f;
    };
    auto put = [&](int i, float y) {
      const uint16_t b = uint16_t(cvt_bf16x2(y, 0.0f));
      if (out) out[i] = b;
      if (!isq && row >= 0) a.k_cache[row + at + i] = e4m3_of(b, a.k_scale, a.k_inv);
    };
    for (int i = lane; i < half; i += 64) {
      const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : i + half;
      const float na = normed(ia), nb = normed(ib);
      const float co = a.cos_sin[pos * a.rot + i], si = a.cos_sin[pos * a.rot + half + i];
      put(ia, na * co - nb * si);
      put(ib, nb * co + na * si);
    }
    for (int i = a.rot + lane; i < a.d; i += 64) put(i, normed(i));
  }
}

int rope_check(int32_t tokens, int32_t hq, int32_t hkv, int32_t d, int32_t rot, float eps,
               int64_t npos, int64_t qs, int64_t ks, int64_t qos, int64_t kos, bool k_out) {
  if (tokens < 0 || hq <= 0 || hkv <= 0 || d <= 0 || d > 65536) return FP8Q_EINVAL;
  if (hq > (1 << 20) || hkv > (1 << 20)) return FP8Q_EINVAL;
  if (rot < 0 || rot > d || rot % 2 != 0) return FP8Q_EINVAL;
  if (rot > 0 && (npos <= 0 || npos > (int64_t(1) << 40))) return FP8Q_EINVAL;
  if (!(eps >= 0.0f && eps <= 1.0f)) return FP8Q_EINVAL;
  const int64_t eq = int64_t(hq) * d, ek = int64_t(hkv) * d, most = int64_t(1) << 30;
  if (qs < eq || ks < ek || qos < eq || (k_out && kos < ek)) return FP8Q_EINVAL;
  if (qs > most || ks > most || qos > most || (k_out && kos > most)) return FP8Q_EINVAL;
  return FP8Q_OK;
}

int rope_run(const RopeArgs& a, int interleaved, hipStream_t stream) {
  const int lanes = a.d / 8;
  const bool pow2 = a.d % 8 == 0 && lanes >= 1 && lanes <= 64 && (lanes & (lanes - 1)) == 0;
  const bool write = a.slots != nullptr;
  const bool vec = pow2 && lanes >= 4 && a.rot % (interleaved ? 8 : 16) == 0 && a.qs % 8 == 0 &&
                   a.ks % 8 == 0 && a.qos % 8 == 0 && (!a.k_out || a.kos % 8 == 0) &&
                   aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.q_out, 16) &&
                   aligned(a.k_out, 16) && aligned(a.qw, 16) && aligned(a.kw, 16) &&
                   aligned(a.cos_sin, 16) &&
                   (!write || (a.vs % 8 == 0 && a.cs % 8 == 0 && aligned(a.v, 16) &&
                               aligned(a.k_cache, 8) && aligned(a.v_cache, 8)));
  const int64_t heads = a.hq + a.hkv + (write ? a.hkv : 0);
  if (!vec) {
    const int64_t blocks = clamp_grid((a.tokens * heads + kRopeRows - 1) / kRopeRows);
    launch(rope_scalar_kernel, dim3(unsigned(blocks)), dim3(64, kRopeRows), 0, stream, a,
           interleaved);
    return launch_status();
  }
  // Few tokens: a lane group for every head of the token, in one pass.  Many: about six heads a
  // group, so that its cosines and weights serve them all, and as many workgroups as a CU holds,
  // which go on to further tokens.  4593 tokens of 48 128-wide heads: 26.7 us with 128 threads, 29.8 with 256,
  // 38 with 512; 9000 tokens of 24 64-wide heads: 13.8 us with 64 threads, 16.4 with 128.
  const int64_t all = (heads * lanes + 63) / 64 * 64;
  const bool few = a.tokens <= 2 * num_cus();
  int64_t threads = few ? all : (heads * lanes / 6 + 63) / 64 * 64;
  threads = threads < 64 ? 64 : threads > 1024 ? 1024 : threads;
  const int64_t most = few ? a.tokens : 2048 / threads * num_cus();
  const unsigned blocks = unsigned(a.tokens < most ? a.tokens : most);
  void (*kern)(RopeArgs) = nullptr;
  switch (lanes) {
    case 4: kern = interleaved ? rope_vec_kernel<2, true> : rope_vec_kernel<2, false>; break;
    case 8: kern = interleaved ? rope_vec_kernel<3, true> : rope_vec_kernel<3, false>; break;
    case 16: kern = interleaved ? rope_vec_kernel<4, true> : rope_vec_kernel<4, false>; break;
    case 32: kern = interleaved ? rope_vec_kernel<5, true> : rope_vec_kernel<5, false>; break;
    default: kern = interleaved ? rope_vec_kernel<6, true> : rope_vec_kernel<6, false>; break;
  }
  launch(kern, dim3(blocks), dim3(unsigned(threads)), 0, stream, a);
  return launch_status();
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int qk_norm_rope(const uint16_t* q, const uint16_t* k, const uint16_t* q_weight,
                            const uint16_t* k_weight, float eps, const int64_t* positions,
                            const float* cos_sin, int64_t num_positions, int32_t rot_dim,
                            int32_t interleaved, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int64_t q_stride,
                            int64_t key_stride, uint16_t* q_out, uint16_t* k_out,
                            int64_t q_out_stride, int64_t k_out_stride, hipStream_t stream) {
  const int rc = rope_check(num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, eps,
                            num_positions, q_stride, key_stride, q_out_stride, k_out_stride, true);
  if (rc != FP8Q_OK) return rc;
  if (num_tokens == 0) return FP8Q_OK;
  if (!q || !k || !q_out || !k_out || (rot_dim > 0 && (!positions || !cos_sin))) return FP8Q_ENULL;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(q_out, 2) || !aligned(k_out, 2) ||
      !aligned(q_weight, 2) || !aligned(k_weight, 2) || !aligned(positions, 8) ||
      !aligned(cos_sin, 4))
    return FP8Q_EALIGN;
  RopeArgs a = {};
  a.q = q, a.k = k, a.qw = q_weight, a.kw = k_weight, a.positions = positions;
  a.cos_sin = cos_sin, a.q_out = q_out, a.k_out = k_out, a.npos = num_positions;
  a.tokens = num_tokens, a.qs = q_stride, a.ks = key_stride, a.qos = q_out_stride;
  a.kos = k_out_stride, a.rot = rot_dim, a.hq = num_q_heads, a.hkv = num_kv_heads;
  a.d = head_dim, a.bs = 1, a.eps = eps;
  return rope_run(a, interleaved != 0, stream);
}

extern "C" int fp8_qk_norm_rope_kv_write(
    const uint16_t* q, const uint16_t* k, const uint16_t* v, const uint16_t* q_weight,
    const uint16_t* k_weight, float eps, const int64_t* positions, const float* cos_sin,
    int64_t num_positions, int32_t rot_dim, int32_t interleaved, uint8_t* k_cache,
    uint8_t* v_cache, const int64_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks, float k_scale,
    float v_scale, int64_t q_stride, int64_t key_stride, int64_t value_stride,
    int64_t cache_stride, uint16_t* q_out, uint16_t* k_out, int64_t q_out_stride,
    int64_t k_out_stride, hipStream_t stream) {
  int rc = rope_check(num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, eps,
                      num_positions, q_stride, key_stride, q_out_stride, k_out_stride,
                      k_out != nullptr);
  if (rc != FP8Q_OK) return rc;
  rc = kv_write_check(num_tokens, num_kv_heads, head_dim, block_size, num_blocks, k_scale,
                      v_scale, key_stride, value_stride, cache_stride);
  if (rc != FP8Q_OK || value_stride > (int64_t(1) << 30)) return FP8Q_EINVAL;
  if (num_tokens == 0) return FP8Q_OK;
  if (!q || !k || !v || !q_out || !k_cache || !v_cache || !slot_mapping ||
      (rot_dim > 0 && (!positions || !cos_sin)))
    return FP8Q_ENULL;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(q_out, 2) ||
      !aligned(k_out, 2) || !aligned(q_weight, 2) || !aligned(k_weight, 2) ||
      !aligned(positions, 8) || !aligned(slot_mapping, 8) || !aligned(cos_sin, 4))
    return FP8Q_EALIGN;
  RopeArgs a = {};
  a.q = q, a.k = k, a.v = v, a.qw = q_weight, a.kw = k_weight, a.positions = positions;
  a.cos_sin = cos_sin, a.slots = slot_mapping, a.q_out = q_out, a.k_out = k_out;
  a.k_cache = k_cache, a.v_cache = v_cache, a.npos = num_positions, a.tokens = num_tokens;
  a.qs = q_stride, a.ks = key_stride, a.vs = value_stride, a.qos = q_out_stride;
  a.kos = k_out_stride, a.nslots = num_blocks * block_size, a.cs = cache_stride;
  a.rot = rot_dim, a.hq = num_q_heads, a.hkv = num_kv_heads, a.d = head_dim, a.bs = block_size;
  // reciprocals on the host: IEEE binary32 division, RN(1/scale)
  a.eps = eps, a.k_scale = k_scale, a.k_inv = 1.0f / k_scale;
  a.v_scale = v_scale, a.v_inv = 1.0f / v_scale;
  return rope_run(a, interleaved != 0, stream);
}
