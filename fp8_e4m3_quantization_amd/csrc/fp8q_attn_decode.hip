// fp8q_attn_decode.hip -- attention of single query tokens over the paged E4M3 KV cache.
//
// Mathematics, per sequence and query head, over its cached positions j < len (K_j, V_j the E4M3
// values at the position's slot of the head's KV head):
//   s_j = softmax_scale * k_scale * q . K_j
//   out = v_scale * sum_j exp(s_j - r) V_j / sum_j exp(s_j - r),  lse = r + log sum_j exp(s_j - r)
// for any reference r.  Sequences with no position get zeros and lse = -infinity.
//
// Bound: memory; each cached byte is read once, for all the query heads of its KV head.  The
// heads' queries (up to 16 a wave) are the columns of 16x16x32 bf16 MFMAs: S^T = K Q^T over
// tiles of 32 positions, O^T += V^T P^T.  E4M3 values are exact in bf16.  K and V go from memory
// straight to registers.  A lane of row group g (lanes 16 g ..) ends with the scores of positions
// 4g..4g+3 and 16+4g..16+4g+3 of the tile, which are taken as its 8 of the 32 summed by the
// second product as they lie; it loads V at the same 8 positions, bytes D/16 (l % 16) onwards,
// so that both operands agree without an exchange.  P is rounded to bf16 for that product (at
// most 2^-9 of each weight, under the output's own rounding).
//
// The positions of all sequences are cut into chunks of one length, chosen on the device so that
// the workgroups are about as many as the device runs at once, whatever the lengths.  The four
// waves of a workgroup take the tiles of its chunk in turn and add up in LDS; where a sequence
// has several chunks each leaves its sums in the workspace, and the workgroup that comes last
// adds them in the order of the chunks, so that results do not depend on who that is.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_attn.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kDecWaves = 4;
constexpr int kDecTile = 32;                        // positions a wave takes at a time
constexpr int kDecStep = kDecTile * kDecWaves;      // a chunk is a multiple of this
constexpr int kDecRows = 16;                        // query heads of a workgroup
constexpr int kDecPerCu = 2;                        // workgroups per CU the chunks are cut for

struct DecodeArgs {
  const uint16_t* q;
  const uint8_t *kc, *vc;
  const int32_t *tables, *lens;
  uint16_t* out;
  float* lse;
  uint32_t* counts;  // [seqs * heads of work], zero between calls
  float* parts;      // [units * heads of work][rows][D + 2]
  int64_t ts, qs, os, cs, nblocks;
  int seqs, width, hq, hkv, group, bs;
  int row_tiles;     // ceil(group / 16)
  int units;         // chunks the grid has room for
  int target;        // chunks wanted per head of work
  float scale_log2, v_scale;
};

__device__ __forceinline__ int64_t seq_len(const DecodeArgs& a, int s) {
  const int64_t n = s < a.seqs ? a.lens[s] : 0, most = int64_t(a.width) * a.bs;
  return n < 0 ? 0 : n > most ? most : n;
}

// Values of the workspace are written and read at device scope, where every XCD sees them.
__device__ __forceinline__ void put(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Two E4M3 codes (low or high half of w) as two bf16, exact.
template <bool kHigh>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t w) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, kHigh);
  return __builtin_bit_cast(uint32_t, r);
}

template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  }
}

template <int D>
__global__ __launch_bounds__(64 * kDecWaves, D == 256 ? 1 : 2) void decode_kernel(const DecodeArgs a) {
  constexpr int kSteps = D / 32;      // MFMAs of a 16-position score tile
  constexpr int kPieces = D / 64;     // 16-byte K loads of a lane and position
  constexpr int kOut = D / 16;        // MFMAs of the second product; bytes of V of a lane
  constexpr int kVw = D / 64;         // dwords of them
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads = a.hkv * a.row_tiles;
  const int hw = blockIdx.x % heads;               // head of work: KV head and row tile
  int unit = blockIdx.x / heads;
  const int kvh = hw / a.row_tiles;
  const int row0 = (hw % a.row_tiles) * kDecRows;  // first query head of the group taken here
  const int rows = min(kDecRows, a.group - row0);

  // Chunk length, and this unit's sequence and chunk.
  int64_t all = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    int64_t n = seq_len(a, s0 + lane);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    all += n;
  }
  const int64_t want = (all + a.target - 1) / a.target;
  const int64_t chunk = max((want + kDecStep - 1) / kDecStep, int64_t(1)) * kDecStep;
  int seq = -1, part = 0, parts = 0;
  int64_t len = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const int64_t n = seq_len(a, s0 + lane);
    const int c = s0 + lane < a.seqs ? int(max((n + chunk - 1) / chunk, int64_t(1))) : 0;
    const int upto = wave_prefix(c), here = __shfl(upto, 63);
    if (unit < here) {
      const int j = __builtin_ctzll(__ballot(upto > unit));
      seq = s0 + j;
      parts = __shfl(c, j);
      part = unit - (__shfl(upto, j) - parts);
      len = __shfl(n, j);
      break;
    }
    unit -= here;
  }
  if (seq < 0) return;
  const int64_t begin = part * chunk, end = min(begin + chunk, len);

  // Queries: column l % 16 is the query head; the order of the D values follows K's loads.
  v8bf qf[kSteps];
  {
    const uint16_t* src = a.q + seq * a.qs + int64_t(kvh * a.group + row0 + min(col, rows - 1)) * D;
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
      qf[c] = __builtin_bit_cast(
          v8bf, *reinterpret_cast<const uint4*>(src + 64 * (c >> 1) + 16 * g + 8 * (c & 1)));
  }

  __shared__ int64_t s_row[kDecWaves][kDecTile];
  __shared__ float s_o[kDecWaves][kDecRows][D];
  __shared__ float s_ref[kDecWaves][kDecRows], s_sum[kDecWaves][kDecRows];
  const int64_t e = int64_t(a.hkv) * D;

  v4f o[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float ref = neg_inf(), sum = 0.0f;

  for (int64_t p0 = begin + wave * kDecTile; p0 < end; p0 += kDecStep) {
    // where the tile's positions lie in the pools; -1: none (behind the end, a bad block)
    if (lane < kDecTile) {
      const int64_t pos = p0 + lane;
      int64_t at = -1;
      if (pos < end) {
        const int64_t b = pos / a.bs;
        const int64_t id = a.tables[seq * a.ts + b];
        if (id >= 0 && id < a.nblocks) at = id * a.cs + (pos - b * a.bs) * e + int64_t(kvh) * D;
      }
      s_row[wave][lane] = at;
    }
    __builtin_amdgcn_wave_barrier();
    uint4 kx[2][kPieces];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t at = max(s_row[wave][16 * b + col], int64_t(0));
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        kx[b][c] = *reinterpret_cast<const uint4*>(a.kc + at + 64 * c + 16 * g);
    }
    uint32_t vx[8][kVw];
    bool ok[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = s_row[wave][16 * (j >> 2) + 4 * g + (j & 3)];
      ok[j] = at >= 0;
      load_bytes<kOut>(a.vc + max(at, int64_t(0)) + kOut * col, vx[j]);
    }
    __builtin_amdgcn_wave_barrier();

    float sc[8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const uint4 x = kx[b][c >> 1];
        const uint32_t lo = (c & 1) ? x.z : x.x, hi = (c & 1) ? x.w : x.y;
        const v4u w = {e4m3x2_to_bf16<false>(lo), e4m3x2_to_bf16<true>(lo),
                       e4m3x2_to_bf16<false>(hi), e4m3x2_to_bf16<true>(hi)};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), qf[c], acc, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sc[4 * b + r] = ok[4 * b + r] ? acc[r] * a.scale_log2 : neg_inf();
    }
    float top = sc[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, sc[j]);
    top = max_over_rows(top);
    const bool moves = top > ref + kSoftmaxSlack;
    if (__any(moves)) {
      const float f = moves ? __builtin_amdgcn_exp2f(ref - top) : 1.0f;
      ref = moves ? top : ref;
      sum *= f;
#pragma unroll
      for (int i = 0; i < kOut; ++i) o[i] *= f;
    }
    const float base = ref == neg_inf() ? 0.0f : ref;
    uint32_t pw[4];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float x = __builtin_amdgcn_exp2f(sc[j] - base), y = __builtin_amdgcn_exp2f(sc[j + 1] - base);
      sum += x + y;
      pw[j / 2] = cvt_bf16x2(x, y);
    }
    const v8bf pf = __builtin_bit_cast(v8bf, v4u{pw[0], pw[1], pw[2], pw[3]});
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int w = 0; w < kVw; ++w) vx[j][w] = ok[j] ? vx[j][w] : 0u;
#pragma unroll
    for (int i = 0; i < kOut; i += 2) {  // values i and i + 1 of each lane's D/16
      uint32_t pair[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        pair[j] = (i & 2) ? e4m3x2_to_bf16<true>(vx[j][i / 4]) : e4m3x2_to_bf16<false>(vx[j][i / 4]);
      v4u even, odd;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        even[j] = __builtin_amdgcn_perm(pair[2 * j + 1], pair[2 * j], 0x05040100u);
        odd[j] = __builtin_amdgcn_perm(pair[2 * j + 1], pair[2 * j], 0x07060302u);
      }
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, even), pf, o[i], 0, 0, 0);
      o[i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, odd), pf, o[i + 1], 0, 0, 0);
    }
  }

  // o[i][r] is value kOut (4g + r) + i of query column l % 16.
  sum = sum_over_rows(sum);
#pragma unroll
  for (int i = 0; i < kOut; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) s_o[wave][col][kOut * (4 * g + r) + i] = o[i][r];
  if (g == 0) {
    s_ref[wave][col] = ref;
    s_sum[wave][col] = sum;
  }
  __syncthreads();

  // The workgroup's sums: thread -> (row, 4 values) of the chunk.
  auto finish = [&](int r, int d, float ref_all, float total, float4 v) {
    const float inv = total == 0.0f ? 0.0f : a.v_scale / total;
    const int64_t h = int64_t(kvh) * a.group + row0 + r;
    *reinterpret_cast<uint2*>(a.out + seq * a.os + h * D + d) =
        make_uint2(cvt_bf16x2(v.x * inv, v.y * inv), cvt_bf16x2(v.z * inv, v.w * inv));
    if (a.lse && d == 0)
      a.lse[int64_t(seq) * a.hq + h] =
          total == 0.0f ? neg_inf() : (ref_all + __builtin_amdgcn_logf(total)) * kLn2;
  };
  const int64_t stride = int64_t(kDecRows) * (D + 2);
  const int64_t first = (int64_t(blockIdx.x / heads) - part) * heads + hw;  // part 0's place
  float* mine = a.parts + (first + int64_t(part) * heads) * stride;
  for (int it = threadIdx.x; it < rows * (D / 4); it += 64 * kDecWaves) {
    const int r = it / (D / 4), d = it % (D / 4) * 4;
    float m = s_ref[0][r];
#pragma unroll
    for (int w = 1; w < kDecWaves; ++w) m = fmaxf(m, s_ref[w][r]);
    float total = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kDecWaves; ++w) {
      const float f = s_ref[w][r] == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(s_ref[w][r] - m);
      total += s_sum[w][r] * f;
      const float4 x = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
      v.x += x.x * f; v.y += x.y * f; v.z += x.z * f; v.w += x.w * f;
    }
    if (parts == 1) {
      finish(r, d, m, total, v);
    } else {
      float* p = mine + r * (D + 2);
      put(p + d, v.x); put(p + d + 1, v.y); put(p + d + 2, v.z); put(p + d + 3, v.w);
      if (d == 0) { put(p + D, m); put(p + D + 1, total); }
    }
  }
  if (parts == 1) return;

  __shared__ int s_last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are where all see them
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(a.counts + int64_t(seq) * heads + hw, 1u, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) == uint32_t(parts - 1);
  __syncthreads();
  if (!s_last) return;
  if (threadIdx.x == 0)
    __hip_atomic_store(a.counts + int64_t(seq) * heads + hw, 0u, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  for (int it = threadIdx.x; it < rows * (D / 4); it += 64 * kDecWaves) {
    const int r = it / (D / 4), d = it % (D / 4) * 4;
    const float* p = a.parts + first * stride + r * (D + 2);
    float m = neg_inf(), total = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < parts; ++c, p += heads * stride) {
      const float pm = get(p + D), pt = get(p + D + 1);
      const float4 x = make_float4(get(p + d), get(p + d + 1), get(p + d + 2), get(p + d + 3));
      const float to = fmaxf(m, pm);
      const float f = m == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(m - to);
      const float h = pm == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(pm - to);
      total = total * f + pt * h;
      v.x = v.x * f + x.x * h; v.y = v.y * f + x.y * h;
      v.z = v.z * f + x.z * h; v.w = v.w * f + x.w * h;
      m = to;
    }
    finish(r, d, m, total, v);
  }
}

constexpr int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int decode_shape(int32_t seqs, int32_t hq, int32_t hkv, int32_t d) {
  if (seqs < 0 || seqs > (1 << 20) || hq <= 0 || hkv <= 0 || hq % hkv != 0 || hq > 65536)
    return FP8Q_EINVAL;
  if (d != 64 && d != 128 && d != 256) return FP8Q_EINVAL;
  return FP8Q_OK;
}

// Workgroups wanted per head of work, and the workspace that leaves room for.
int decode_target(int heads) {
  const int t = kDecPerCu * num_cus() / heads;
  return t < 1 ? 1 : t;
}
uint64_t counts_bytes(int64_t seqs, int64_t heads) { return uint64_t(round_up(seqs * heads * 4, 256)); }
uint64_t decode_workspace(int32_t seqs, int32_t hq, int32_t hkv, int32_t d) {
  if (seqs == 0) return 0;
  const int64_t heads = int64_t(hkv) * ((hq / hkv + kDecRows - 1) / kDecRows);
  const int64_t units = int64_t(decode_target(int(heads))) + seqs;
  return counts_bytes(seqs, heads) + uint64_t(units) * heads * kDecRows * (d + 2) * 4;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int fp8_attn_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim,
                                              uint64_t* bytes) {
  if (!bytes) return FP8Q_ENULL;
  *bytes = 0;
  const int rc = decode_shape(num_seqs, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
  *bytes = decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim);
  return FP8Q_OK;
}

extern "C" int fp8_attn_decode(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               uint16_t* out, float* lse, int32_t num_seqs, int32_t max_blocks,
                               int64_t table_stride, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               float k_scale, float v_scale, float softmax_scale, int64_t q_stride,
                               int64_t out_stride, int64_t cache_stride, void* workspace,
                               uint64_t workspace_bytes, hipStream_t stream) {
  const int rc = decode_shape(num_seqs, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
  if (max_blocks < 0 || block_size <= 0 || num_blocks <= 0 || table_stride < max_blocks)
    return FP8Q_EINVAL;
  if (int64_t(max_blocks) * block_size > (int64_t(1) << 30)) return FP8Q_EINVAL;
  const int64_t eq = int64_t(num_q_heads) * head_dim, ek = int64_t(num_kv_heads) * head_dim;
  if (q_stride < eq || out_stride < eq || q_stride > (int64_t(1) << 30) ||
      out_stride > (int64_t(1) << 30) || table_stride > (int64_t(1) << 40))
    return FP8Q_EINVAL;
  if (cache_stride < int64_t(block_size) * ek || num_blocks > (int64_t(1) << 62) / cache_stride)
    return FP8Q_EINVAL;
  if (!(k_scale >= 0x1p-64f && k_scale <= 0x1p64f) || !(v_scale >= 0x1p-64f && v_scale <= 0x1p64f) ||
      !(softmax_scale > 0.0f && softmax_scale <= 0x1p32f))
    return FP8Q_EINVAL;
  if (num_seqs == 0) return FP8Q_OK;
  if (!q || !k_cache || !v_cache || !out || !context_lens || !workspace ||
      (max_blocks > 0 && !block_tables))
    return FP8Q_ENULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256) || q_stride % 8 || out_stride % 8 || cache_stride % 16)
    return FP8Q_EALIGN;
  if (workspace_bytes < decode_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim))
    return FP8Q_EINVAL;
  DecodeArgs a = {};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.tables = block_tables, a.lens = context_lens;
  a.out = out, a.lse = lse, a.ts = table_stride, a.qs = q_stride, a.os = out_stride;
  a.cs = cache_stride, a.nblocks = num_blocks, a.seqs = num_seqs, a.width = max_blocks;
  a.hq = num_q_heads, a.hkv = num_kv_heads, a.group = num_q_heads / num_kv_heads;
  a.bs = block_size, a.row_tiles = (a.group + kDecRows - 1) / kDecRows;
  const int heads = a.hkv * a.row_tiles;
  a.target = decode_target(heads);
  a.units = a.target + num_seqs;
  a.counts = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + counts_bytes(num_seqs, heads));
  a.scale_log2 = softmax_scale * k_scale * kLog2e;
  a.v_scale = v_scale;
  const int64_t blocks = int64_t(a.units) * heads;
  if (blocks > 0x7FFFFFFF) return FP8Q_EINVAL;
  auto kern = head_dim == 64 ? decode_kernel<64> : head_dim == 128 ? decode_kernel<128> : decode_kernel<256>;
  launch(kern, dim3(unsigned(blocks)), dim3(64 * kDecWaves), 0, stream, a);
  return launch_status();
}
