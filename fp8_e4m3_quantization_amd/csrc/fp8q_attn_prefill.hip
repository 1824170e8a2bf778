// fp8q_attn_prefill.hip -- attention over whole prompts: bf16 queries, keys and values of packed
// sequences of different lengths, grouped heads, causal from the end of each sequence.
//
// Mathematics, query i of a sequence of Lq queries and Lk keys, scores s_ij = scale q_i . k_j
// over the keys j it sees (all of them, or causal j <= i + Lk - Lq):
//   out_i = sum_j exp(s_ij - r) v_j / sum_j exp(s_ij - r),   lse_i = r + log sum_j exp(s_ij - r)
// for any reference r; one pass over the keys with a running r near the largest score so far.
// A query that sees no key gets zeros and lse = -infinity.
//
// A wave owns 32 queries and walks the keys in tiles of 64.  It computes S^T = K Q^T (32x32x16
// bf16 MFMA), so that a lane holds scores of one query (column l % 32): the softmax needs no
// exchange but one between lanes l and l ^ 32.  The lane's 16 scores of a 32-key tile are then
// the B operand of O^T += V^T P^T as they lie, when the keys of each 16-key step are taken in the
// order 4h..4h+3, 8+4h..8+4h+3 for lane half h; V^T comes from LDS in that order through the
// transposing 8-byte LDS read.  P is rounded to bf16 for that product (at most 2^-9 of each
// weight, under the output's own rounding); the sum of weights is of the unrounded ones.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_attn.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kTileKeys = 64;
constexpr int kWaveRows = 32;
constexpr int kOrderedSeqs = 256;  // batches up to this size run their longest tiles first

struct PrefillArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;  // [tq, hq] or NULL
  const int32_t *cu_q, *cu_k;
  int64_t qs, ks, vs, os;
  int seqs, tq, tk, hq, hkv, causal;
  float scale_log2;  // softmax scale * log2(e)
};

// Start and length of sequence s among `total` rows, whatever the list holds.
__device__ __forceinline__ void seq_span(const int32_t* cu, int s, int total, int* start, int* len) {
  const int a = min(max(cu[s], 0), total);
  *start = a;
  *len = min(max(cu[s + 1], a), total) - a;
}

// The sequence and row tile (of `rows` queries) of work item `rank`, or false.  Tiles are ranked
// by descending index within their sequence (under a causal mask a later tile has more keys), so
// that the longest run first and the short ones fill the last round.
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int rows, int rank, int* seq,
                                          int* tile) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int s) {
    int st, n = 0;
    if (s < a.seqs) seq_span(a.cu_q, s, a.tq, &st, &n);
    return (n + rows - 1) / rows;
  };
  if (a.seqs > kOrderedSeqs) {  // in sequence order
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
      const int n = tiles_of(s0 + lane);
      const int upto = wave_prefix(n);
      const int all = __shfl(upto, 63);
      if (rank < all) {
        const int j = __builtin_ctzll(__ballot(upto > rank));
        *seq = s0 + j;
        *tile = rank - (__shfl(upto, j) - __shfl(n, j));
        return true;
      }
      rank -= all;
    }
    return false;
  }
  int n[kOrderedSeqs / 64];
  int most = 0;
#pragma unroll
  for (int c = 0; c < kOrderedSeqs / 64; ++c) {
    n[c] = c * 64 < a.seqs ? tiles_of(c * 64 + lane) : 0;
    most = max(most, n[c]);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) most = max(most, __shfl_xor(most, o));
  // S(L) = number of tiles with index >= L; find the largest L with S(L) > rank, 64 candidates
  // at a time (one per lane)
  int lo = 0, hi = most;  // S(lo) > rank is wanted, S(hi) = 0
  auto at_least = [&](int level) {
    int sum = 0;
#pragma unroll
    for (int c = 0; c < kOrderedSeqs / 64; ++c) {
      const int live = min(a.seqs - c * 64, 64);
      for (int j = 0; j < live; ++j) sum += max(__builtin_amdgcn_readlane(n[c], j) - level, 0);
    }
    return sum;
  };
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int level = lo + lane * step;
    const uint64_t more = __ballot(level < hi && at_least(level) > rank);
    if (more == 0) return false;  // only when no tile has this rank
    const int j = 63 - __builtin_clzll(more);
    hi = min(hi, lo + (j + 1) * step);
    lo = lo + j * step;
    if (step <= 1) break;
  }
  rank -= at_least(lo + 1);  // among the sequences that have a tile `lo`
#pragma unroll
  for (int c = 0; c < kOrderedSeqs / 64; ++c) {
    const uint64_t has = __ballot(n[c] > lo);
    const int all = __popcll(has);
    if (rank < all) {
      const int before = __popcll(has & ((uint64_t(1) << lane) - 1));
      const uint64_t it = __ballot(n[c] > lo && before == rank);
      *seq = c * 64 + __builtin_ctzll(it);
      *tile = lo;
      return true;
    }
    rank -= all;
  }
  return false;
}

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

typedef __attribute__((address_space(3))) void lds_void;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Bits set where one of the two bf16 in w is an infinity or NaN (exponent all ones).
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

template <int D, int kWaves>
__device__ __forceinline__ void prefill_tile(const PrefillArgs& a) {
  constexpr int kRows = kWaveRows * kWaves;
  constexpr int kChunks = D / 8;                              // 16-byte chunks of a row
  constexpr int kCopies = kTileKeys * kChunks / (64 * kWaves);  // 1 KB copies per wave and tile
  __shared__ __attribute__((aligned(16))) uint16_t k0[kTileKeys * D], k1[kTileKeys * D];
  __shared__ __attribute__((aligned(16))) uint16_t v0[kTileKeys * D], v1[kTileKeys * D];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // heads: workgroups go to the 8 XCDs in turn; where the heads divide, each XCD takes
  // neighbouring heads (which share keys and values in its L2)
  int head, rank;
  if (a.hq % 8 == 0) {
    const int per = a.hq / 8, i = blockIdx.x / 8;
    head = (blockIdx.x % 8) * per + i % per;
    rank = i / per;
  } else {
    head = blockIdx.x % a.hq;
    rank = blockIdx.x / a.hq;
  }
  int seq, tile;
  if (!find_tile(a, kRows, rank, &seq, &tile)) return;
  seq = __builtin_amdgcn_readfirstlane(seq);
  tile = __builtin_amdgcn_readfirstlane(tile);
  int q0, lq, kv0, lk;
  seq_span(a.cu_q, seq, a.tq, &q0, &lq);
  seq_span(a.cu_k, seq, a.tk, &kv0, &lk);
  const int kvh = head / (a.hq / a.hkv);
  const int first = tile * kRows;                    // the workgroup's first query
  const int mine = first + wave * kWaveRows;         // this wave's
  // keys [0, seen(i)) are seen by query i
  auto seen = [&](int i) { return a.causal ? min(max(i + lk - lq + 1, 0), lk) : lk; };
  const int last = min(first + kRows, lq) - 1;
  const int tiles = (seen(last) + kTileKeys - 1) / kTileKeys;
  const int row = mine + col;                        // this lane's query
  const int limit = row < lq ? seen(row) : 0;
  const int wave_limit = mine < lq ? seen(min(mine + kWaveRows, lq) - 1) : 0;
  const int all_see = seen(first);                   // every query of the workgroup sees these

  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(q0 + min(row, lq - 1)) * a.qs + int64_t(head) * D + 8 * half;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 16 * s));
  }

  const uint16_t* kbase = a.k + int64_t(kv0) * a.ks + int64_t(kvh) * D;
  const uint16_t* vbase = a.v + int64_t(kv0) * a.vs + int64_t(kvh) * D;
  // The copy j of a wave fills 1 KB of the tile; the lane's place in it fixes the row and, by
  // the chunk order, the chunk that it fetches.  Rows behind the last key fetch the last key.
  auto copy_tile = [&](int t, uint16_t* dk, uint16_t* dv) {
    const int left = lk - t * kTileKeys;  // > 0
    const int span = min(left, kTileKeys);
    const __amdgpu_buffer_rsrc_t rk = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(kbase + int64_t(t) * kTileKeys * a.ks), 0,
        int(((span - 1) * a.ks + D) * 2), 0x00020000);
    const __amdgpu_buffer_rsrc_t rv = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(vbase + int64_t(t) * kTileKeys * a.vs), 0,
        int(((span - 1) * a.vs + D) * 2), 0x00020000);
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int at = (wave + kWaves * j) * 64 + lane;
      const int r = at / kChunks, c = at % kChunks;
      const int from = min(r, span - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rk, (lds_void*)(dk + (wave + kWaves * j) * 512), 16,
          int(from * a.ks * 2) + k_chunk<D>(r, c) * 16, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rv, (lds_void*)(dv + (wave + kWaves * j) * 512), 16,
          int(from * a.vs * 2) + v_chunk<D>(r, c) * 16, 0, 0, 0);
    }
  };

  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  float ref = neg_inf(), sum = 0.0f;  // reference (log2 units) and this half's weights

  // S^T of tile t, softmax, O^T: kMasked tiles hold keys that some query does not see
  auto compute = [&](int t, const uint16_t* kt, const uint16_t* vt, auto masked, bool odd_values) {
    constexpr bool kMasked = decltype(masked)::value;
    v16f s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) {
        const int r = 32 * b + col;
        const v8bf kf = __builtin_bit_cast(
            v8bf, *reinterpret_cast<const uint4*>(kt + r * D + k_chunk<D>(r, 2 * st + half) * 8));
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st], s[b], 0, 0, 0);
      }
    }
    float top = neg_inf();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (kMasked) {
          const int key = t * kTileKeys + 32 * b + 8 * (r >> 2) + 4 * half + (r & 3);
          s[b][r] = key < limit ? s[b][r] : neg_inf();
        }
        top = fmaxf(top, s[b][r]);
      }
    top = max_over_halves(top) * a.scale_log2;
    if (__any(top > ref + kSoftmaxSlack)) {
      const bool moves = top > ref + kSoftmaxSlack;
      const float f = moves ? __builtin_amdgcn_exp2f(ref - top) : 1.0f;
      ref = moves ? top : ref;
      sum *= f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= f;
    }
    const float base = ref == neg_inf() ? 0.0f : ref;
    v8bf p[4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; r += 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r + e], a.scale_log2, -base));
          const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r + e + 1], a.scale_log2, -base));
          sum += x + y;
          w[e / 2] = cvt_bf16x2(x, y);
        }
        p[2 * b + r / 8] = __builtin_bit_cast(v8bf, make_uint4(w[0], w[1], w[2], w[3]));
      }
    const int i16 = lane & 15, side = (lane >> 4) & 1;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        const int ra = 16 * st + 4 * half + (i16 >> 2), c = 4 * i + 2 * side + ((i16 & 3) >> 1);
        const int byte8 = 4 * (i16 & 1);  // elements into the chunk
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s*)(vt + ra * D + v_chunk<D>(ra, c) * 8 + byte8));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s*)(vt + (ra + 8) * D + v_chunk<D>(ra + 8, c) * 8 + byte8));
        v2u l2 = __builtin_bit_cast(v2u, lo), h2 = __builtin_bit_cast(v2u, hi);
        v4u w = {l2[0], l2[1], h2[0], h2[1]};
        if (kMasked && odd_values) {  // a masked weight of 0 times an infinity is not 0
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t bad = non_finite(w[e]);
            w[e] &= ~((bad >> 15) * 0xFFFFu);
          }
        }
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), p[st], o[i], 0, 0, 0);
      }
    if (kMasked && odd_values) {  // the infinities and NaNs that this lane's query does see
      for (int j = 0; j < kTileKeys; ++j)
        if (t * kTileKeys + j < limit) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int e = 32 * i + 8 * (r >> 2) + 4 * half + (r & 3);
              const uint32_t x = vt[j * D + v_chunk<D>(j, e >> 3) * 8 + (e & 7)];
              if (non_finite(x)) o[i][r] += __uint_as_float(x << 16);
            }
        }
    }
  };
  auto odd_in = [&](const uint16_t* vt) {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const uint4 x = *reinterpret_cast<const uint4*>(vt + ((wave + kWaves * j) * 64 + lane) * 8);
      any |= non_finite(x.x) | non_finite(x.y) | non_finite(x.z) | non_finite(x.w);
    }
    return __syncthreads_or(any != 0) != 0;
  };
  auto turn = [&](int t, const uint16_t* kt, const uint16_t* vt, uint16_t* kn, uint16_t* vn) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's copies of tile t landed
    __syncthreads();                     // every wave's have, and the other buffers are free
    if (t + 1 < tiles) copy_tile(t + 1, kn, vn);
    if ((t + 1) * kTileKeys > all_see) {
      const bool odd = odd_in(vt);
      if (t * kTileKeys < wave_limit) compute(t, kt, vt, std::true_type{}, odd);
    } else {
      compute(t, kt, vt, std::false_type{}, false);
    }
  };
  if (tiles > 0) copy_tile(0, k0, v0);
  for (int t = 0; t < tiles; t += 2) {
    turn(t, k0, v0, k1, v1);
    if (t + 1 < tiles) turn(t + 1, k1, v1, k0, v0);
  }

  const float total = sum_over_halves(sum);
  if (row >= lq) return;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* dst = a.out + int64_t(q0 + row) * a.os + int64_t(head) * D + 4 * half;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<uint2*>(dst + 32 * i + 2 * r) =
          make_uint2(cvt_bf16x2(o[i][r] * inv, o[i][r + 1] * inv),
                     cvt_bf16x2(o[i][r + 2] * inv, o[i][r + 3] * inv));
  if (a.lse && half == 0)
    a.lse[int64_t(q0 + row) * a.hq + head] =
        total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
}

template <int D, int kWaves>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void prefill_kernel(const PrefillArgs a) {
  prefill_tile<D, kWaves>(a);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int attn_prefill(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, uint16_t* out,
                            float* lse, int32_t num_seqs, int32_t total_q, int32_t total_k,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            float softmax_scale, int32_t causal, int64_t q_stride,
                            int64_t key_stride, int64_t value_stride, int64_t out_stride,
                            hipStream_t stream) {
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || total_q > (1 << 30) || total_k > (1 << 30) ||
      num_seqs > (1 << 24))
    return FP8Q_EINVAL;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      num_q_heads > 65536)
    return FP8Q_EINVAL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP8Q_EINVAL;
  if (!(softmax_scale > 0.0f && softmax_scale <= 0x1p64f)) return FP8Q_EINVAL;
  const int64_t eq = int64_t(num_q_heads) * head_dim, ek = int64_t(num_kv_heads) * head_dim;
  const int64_t most = int64_t(1) << 23;  // a tile's 64 rows stay within 32-bit byte offsets
  if (q_stride < eq || out_stride < eq || key_stride < ek || value_stride < ek ||
      q_stride > most || out_stride > most || key_stride > most || value_stride > most)
    return FP8Q_EINVAL;
  if (num_seqs == 0 || total_q == 0) return FP8Q_OK;
  if (!q || !out || !cu_seqlens_q || !cu_seqlens_k || (total_k > 0 && (!k || !v))) return FP8Q_ENULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) ||
      q_stride % 8 || key_stride % 8 || value_stride % 8 || out_stride % 8)
    return FP8Q_EALIGN;
  PrefillArgs a = {};
  a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse, a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k, a.qs = q_stride, a.ks = key_stride, a.vs = value_stride;
  a.os = out_stride, a.seqs = num_seqs, a.tq = total_q, a.tk = total_k, a.hq = num_q_heads;
  a.hkv = num_kv_heads, a.causal = causal != 0, a.scale_log2 = softmax_scale * kLog2e;
  constexpr int kWaves = 4;
  // tiles of whole sequences never exceed this many
  const int64_t tiles = int64_t(total_q) / (kWaveRows * kWaves) + num_seqs;
  const int64_t blocks = tiles * num_q_heads;
  if (blocks > 0x7FFFFFFF) return FP8Q_EINVAL;
  auto kern = head_dim == 64 ? prefill_kernel<64, kWaves>
            : head_dim == 128 ? prefill_kernel<128, kWaves> : prefill_kernel<256, kWaves>;
  launch(kern, dim3(unsigned(blocks)), dim3(64 * kWaves), 0, stream, a);
  return launch_status();
}
