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
// transposing 8-byte LDS read.  P is rounded to bf16 for that product (by up to 2^-8 of each
// weight, as much as the output's own rounding); out's denominator is the sum of the rounded
// weights, so that a weight that outweighs all others loses nothing by its rounding; lse is of the
// unrounded ones.
//
// Bound: matrix cores and vector ALUs alike (a score costs as long in its exponential as in its
// products at 128-wide heads), two waves of a SIMD overlapping them: 4593 queries of 40 heads,
// 4 KV heads, 128 wide, causal (217 GFLOP) take 227 us, 0.95 PFLOP/s, call after call (the first
// dozens of calls up to 275: the clock falls to 1.75 GHz under that load before it settles); matrix
// cores are busy 57 % and vector ALUs 51 % of the time, LDS 28 %.  Without the sum of the rounded
// weights it is 7 us less; of those 217, the products and copies alone take 166, with the softmax 190.
// 128 queries a workgroup: 32 a wave, since o, two tiles of scores and q fill the registers of two
// waves a SIMD (64 a wave, alone on its SIMD: 320 us).  64-wide heads: three waves a SIMD, two prompts
// of 2500 in 72 us, vector ALUs busy 70 %, matrix cores 43 %.
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
constexpr int kPrefillWaves = 4;
constexpr int kPrefillRows = kWaveRows * kPrefillWaves;  // queries of a workgroup
constexpr float kFar = 0x1p27f;    // a reference whose rounding (2^3) still leaves weights their range
constexpr int kOrderedSeqs = 256;  // batches up to this size run their longest tiles first

struct PrefillArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;  // [tq, hq] or NULL
  const int32_t *cu_q, *cu_k;
  int64_t qs, ks, vs, os;
  int seqs, tq, tk, hq, hkv, causal;
  int items;         // work items there is room for
  int most_parts;    // parts of a tile's keys; 1: not split
  float scale_log2;  // softmax scale * log2(e)
  float* sums;       // [parts][hq][tq][D] where split
  float4* stats;     // [parts][hq][tq]: reference (log2 units), sums of the weights and of the
                     // rounded ones
};

// Parts that `tiles` tiles of keys are split into: no part is short.
constexpr int kPartTiles = 4;
__device__ __forceinline__ int parts_of(const PrefillArgs& a, int tiles) {
  return max(min(a.most_parts, tiles / kPartTiles), 1);
}

// The place of a query row's sums of one part and head.
__device__ __forceinline__ int64_t sums_at(const PrefillArgs& a, int part, int head, int q_row) {
  return (int64_t(part) * a.hq + head) * a.tq + q_row;
}

// Start and length of sequence s among `total` rows, whatever the list holds.
__device__ __forceinline__ void seq_span(const int32_t* cu, int s, int total, int* start, int* len) {
  const int a = min(max(cu[s], 0), total);
  *start = a;
  *len = min(max(cu[s + 1], a), total) - a;
}

// The sequence and row tile (of `rows` queries) of work item `rank`, or false.  Tiles are ranked
// by descending index within their sequence (under a causal mask a later tile has more keys), so
// that the longest run first and the short ones fill the last round.  `first`: the length of
// sequence `lane`, of the first 64.
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int rows, int rank, int first,
                                          int* seq, int* tile) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int s) {
    int st, n = s < 64 ? first : 0;
    if (s >= 64 && s < a.seqs) seq_span(a.cu_q, s, a.tq, &st, &n);
    return (n + rows - 1) / rows;
  };
  if (a.seqs == 1) {
    *seq = 0;
    *tile = __builtin_amdgcn_readlane(tiles_of(lane), 0) - 1 - rank;
    return *tile >= 0;
  }
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
#pragma unroll
  for (int c = 0; c < kOrderedSeqs / 64; ++c) n[c] = c * 64 < a.seqs ? tiles_of(c * 64 + lane) : 0;
  // S(L) = number of tiles with index >= L; find the largest L with S(L) > rank, 64 candidates
  // at a time (one per lane)
  int lo = 0, hi = (a.tq + rows - 1) / rows;  // S(lo) > rank is wanted, S(hi) = 0
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

// A work item: a tile of queries of one head.  Workgroups go to the 8 XCDs in turn; where the
// heads divide, each XCD takes neighbouring heads, which share keys and values in its L2.
struct Item {
  int head, seq, tile, q0, lq, kv0, lk;
  // keys [0, seen(i)) are seen by query i
  __device__ __forceinline__ int seen(const PrefillArgs& a, int i) const {
    return a.causal ? min(max(i + lk - lq + 1, 0), lk) : lk;
  }
  // tiles of keys that some query of the tile sees
  __device__ __forceinline__ int key_tiles(const PrefillArgs& a) const {
    const int last = min((tile + 1) * kPrefillRows, lq) - 1;
    return __builtin_amdgcn_readfirstlane((seen(a, last) + kTileKeys - 1) / kTileKeys);
  }
};
__device__ __forceinline__ bool find_item(const PrefillArgs& a, int index, Item* it) {
  if (index >= a.items) return false;
  int rank;
  if (a.hq % 8 == 0) {
    const int per = a.hq / 8, i = index / 8;
    it->head = (index % 8) * per + i % per;
    rank = i / per;
  } else {
    it->head = index % a.hq;
    rank = index / a.hq;
  }
  // where the first 64 sequences lie, one to a lane: read at once, before the search
  const int lane = threadIdx.x & 63;
  int q0 = 0, lq = 0, kv0 = 0, lk = 0, seq, tile;
  if (lane < a.seqs) {
    seq_span(a.cu_q, lane, a.tq, &q0, &lq);
    seq_span(a.cu_k, lane, a.tk, &kv0, &lk);
  }
  if (!find_tile(a, kPrefillRows, rank, lq, &seq, &tile)) return false;
  it->seq = __builtin_amdgcn_readfirstlane(seq);
  it->tile = __builtin_amdgcn_readfirstlane(tile);
  if (it->seq < 64) {
    it->q0 = __builtin_amdgcn_readlane(q0, it->seq);
    it->lq = __builtin_amdgcn_readlane(lq, it->seq);
    it->kv0 = __builtin_amdgcn_readlane(kv0, it->seq);
    it->lk = __builtin_amdgcn_readlane(lk, it->seq);
  } else {
    seq_span(a.cu_q, it->seq, a.tq, &it->q0, &it->lq);
    seq_span(a.cu_k, it->seq, a.tk, &it->kv0, &it->lk);
  }
  return true;
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

// Two bf16, infinities and NaNs replaced by the largest finite value of their sign: as integers
// the positive ones lie above 0x7F7F, the negative ones (unsigned) above 0xFF7F.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  typedef short v2s __attribute__((ext_vector_type(2)));
  typedef unsigned short v2us __attribute__((ext_vector_type(2)));
  const v2us below = __builtin_elementwise_min(__builtin_bit_cast(v2us, w), v2us{0xFF7F, 0xFF7F});
  const v2s x = __builtin_elementwise_min(__builtin_bit_cast(v2s, below), v2s{0x7F7F, 0x7F7F});
  return __builtin_bit_cast(uint32_t, x);
}

// The order of a turn of the pipeline below: the score products with the previous tile's weights
// between them, each K read two steps ahead of its product, then the value products.
template <int D>
__device__ __forceinline__ void pair_up() {
  constexpr int kMfma = 0x008, kVector = 0x002, kLdsRead = 0x100;
  __builtin_amdgcn_sched_group_barrier(kLdsRead, 6, 0);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kVector, 6, 0);
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kVector, 6, 0);
    __builtin_amdgcn_sched_group_barrier(kLdsRead, 2, 0);
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kLdsRead, 2, 0);
    __builtin_amdgcn_sched_group_barrier(kVector, 2, 0);
  }
}

template <int D>
__device__ __forceinline__ void prefill_tile(const PrefillArgs& a) {
  constexpr int kWaves = kPrefillWaves;
  constexpr int kChunks = D / 8;                              // 16-byte chunks of a row
  constexpr int kCopies = kTileKeys * kChunks / (64 * kWaves);  // 1 KB copies per wave and tile
  __shared__ __attribute__((aligned(16))) uint16_t k0[kTileKeys * D], k1[kTileKeys * D];
  __shared__ __attribute__((aligned(16))) uint16_t v0[kTileKeys * D], v1[kTileKeys * D];
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // (an item's parts lie 8 apart, on one XCD, where the heads are spread over them)
  const int index = a.most_parts == 1 ? blockIdx.x
                    : blockIdx.x / (8 * a.most_parts) * 8 + blockIdx.x % 8;
  const int part = a.most_parts == 1 ? 0 : blockIdx.x / 8 % a.most_parts;
  Item it;
  if (!find_item(a, index, &it)) return;
  const int head = it.head, q0 = it.q0, lq = it.lq, kvh = head / (a.hq / a.hkv);
  const int first = it.tile * kPrefillRows;          // the workgroup's first query
  const int mine = first + wave * kWaveRows;         // this wave's
  const int row = mine + col;                        // this lane's
  const int all_tiles = it.key_tiles(a), parts = parts_of(a, all_tiles);
  if (part >= parts) return;
  // this part's keys: rows kv0 .. kv0 + lk - 1 of k and v, in `tiles` tiles
  const int from_tile = all_tiles * part / parts, from = from_tile * kTileKeys;
  const int tiles = all_tiles * (part + 1) / parts - from_tile;
  const int kv0 = it.kv0 + from, lk = min(it.lk - from, tiles * kTileKeys);
  auto seen = [&](int i) { return min(max(it.seen(a, i) - from, 0), lk); };
  const int limit = row < lq ? seen(row) : 0;
  // this wave's tiles: those that some of its queries see; those that all of them see whole
  const int my_tiles = __builtin_amdgcn_readfirstlane(
      mine < lq ? (seen(min(mine + kWaveRows, lq) - 1) + kTileKeys - 1) / kTileKeys : 0);
  const int my_whole = __builtin_amdgcn_readfirstlane(mine < lq ? seen(mine) / kTileKeys : 0);

  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(q0 + min(row, lq - 1)) * a.qs + int64_t(head) * D + 8 * half;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 16 * s));
  }

  // Copies of tiles, in order: copy j of a wave fills 1 KB of the tile; the lane's place in it fixes
  // the row and, by the chunk order, the chunk that it fetches.  Rows behind the last key fetch
  // the last key.
  struct Source {
    const uint16_t* at;  // the next tile's first row
    int64_t tile;        // values from tile to tile
    int step;            // bytes from row to row
    int left;            // rows from the next tile on
    int off[kCopies];
  };
  auto source = [&](const uint16_t* p, int64_t stride, auto chunk_of) {
    Source c;
    c.at = p + int64_t(kv0) * stride + int64_t(kvh) * D;
    c.tile = kTileKeys * stride;
    c.step = int(stride) * 2;
    c.left = lk;
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int at = (wave + kWaves * j) * 64 + lane, r = at / kChunks;
      c.off[j] = r * c.step + chunk_of(r, at % kChunks) * 16;
    }
    return c;
  };
  Source ksrc = source(a.k, a.ks, [](int r, int c) { return k_chunk<D>(r, c); });
  Source vsrc = source(a.v, a.vs, [](int r, int c) { return v_chunk<D>(r, c); });
  auto copy_next = [&](Source& c, uint16_t* to) {
    if (c.left <= 0) return;
    const __amdgpu_buffer_rsrc_t from =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(c.at), 0, 0x7FFFFFFF, 0x00020000);
    int w = wave;
    asm volatile("" : "+s"(w));  // addresses in LDS are made here, not kept over the loop
    if (c.left >= kTileKeys) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)(to + (w + kWaves * j) * 512), 16,
                                                 c.off[j], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int behind = max(((wave + kWaves * j) * 64 + lane) / kChunks - c.left + 1, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)(to + (w + kWaves * j) * 512), 16,
                                                 c.off[j] - behind * c.step, 0, 0, 0);
      }
    }
    c.at += c.tile;
    c.left -= kTileKeys;
  };

  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  uint32_t odd = 0;       // not 0: values of the last tiles were held to finite ones
  int first_held = 0;     // the first key of those tiles
  // Fused, a weight's argument is one instruction instead of two: 4593 rows of 64-wide heads 140 us,
  // not 146, of 128-wide 243, not 246.  The rare branch that goes with it costs 256-wide heads
  // registers that they do not have (2300 rows: 114 us, not 104).
  constexpr bool kFused = D < 256;
  const float scale = a.scale_log2;
  float ref = neg_inf(), sum = 0.0f;  // reference (log2 units) and this half's weights
  // These, rounded as the second product takes them: summed by products of ones with 16 blocks of
  // 4x4, in which every lane has a column of its own, so that a NaN stays with its query (the sum
  // comes four times).  Against no second sum: 4593 rows of 128-wide heads 222 -> 229 us, two prompts
  // of 2500 of 64-wide ones 69 -> 74; with dot products on the vector ALUs 231 and 74.
  v4f rounded = {0.0f, 0.0f, 0.0f, 0.0f};
  float base = 0.0f;                  // weights of the current scores: exp2(s * scale - base)

  // S^T of a tile.
  auto products = [&](v16f* s, const uint16_t* kt) {
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
  };
  auto largest = [&](const v16f* s) {
    float top = neg_inf();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
    return max_over_halves(top) * scale;
  };
  // The reference for the scores s, whose largest (log2 units) is top.  Where s * scale - ref is
  // one fused product it is exact but for its last rounding, while ref is rounded: by up to 2^-24
  // of itself, which every weight of a query shares.  Beyond kFar that could leave binary32's range
  // of exponents; there the products are rounded too, so that the largest weight is 1 again.
  auto move_to = [&](float top, v16f* s) {
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
    base = ref == neg_inf() ? 0.0f : ref;
    if (kFused && __any(__builtin_fabsf(base) > kFar)) {
      const float back = 1.0f / scale;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = (s[b][r] * scale - base) * back;
      base = 0.0f;
    }
  };
  auto weight = [&](float s) {
    return __builtin_amdgcn_exp2f(kFused ? __builtin_fmaf(s, scale, -base) : s * scale - base);
  };
  // Weights of 16 keys (step st of the tile) as the second product's operand.
  auto weights = [&](const v16f* s, int st) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int r = 8 * (st & 1) + e;
      const float x = weight(s[st >> 1][r]), y = weight(s[st >> 1][r + 1]);
      sum += x + y;
      w[e / 2] = cvt_bf16x2(x, y);
    }
    const v8bf p = __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
    const v4s ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[0], w[1]}), rounded, 0, 0, 0);
    rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[2], w[3]}), rounded, 0, 0, 0);
    return p;
  };
  // V^T of 16 keys (step st of the tile) and 32 values, in the order of the weights.
  auto v_frag = [&](const uint16_t* vt, int st, int i) {
    const int i16 = lane & 15, side = (lane >> 4) & 1;
    const int ra = 16 * st + 4 * half + (i16 >> 2), c = 4 * i + 2 * side + ((i16 & 3) >> 1);
    const int within = 4 * (i16 & 1);
    const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4s*)(vt + ra * D + v_chunk<D>(ra, c) * 8 + within)));
    const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4s*)(vt + (ra + 8) * D + v_chunk<D>(ra + 8, c) * 8 + within)));
    return v4u{lo[0], lo[1], hi[0], hi[1]};
  };
  // O^T += V^T P^T over 16 keys.  With kEdge, infinities and NaNs are held to the largest finite
  // values, so that a weight of 0 gives 0; returns a word that is not 0 where there were any.
  auto add_values = [&](const uint16_t* vt, int st, v8bf p, auto edge) {
    constexpr bool kEdge = decltype(edge)::value;
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v4u w = v_frag(vt, st, i);
      if (kEdge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = finite2(w[e]);
          odd |= x ^ w[e];
          w[e] = x;
        }
        asm volatile("" : "+v"(odd));  // taken up here: the values as read need not be kept
      }
      o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w), p, o[i], 0, 0, 0);
    }
    return odd;
  };
  auto landed = [&]() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's copies landed
    __syncthreads();                     // every wave's have, and the other buffers are free
  };
  // Every wave passes one barrier a tile, and at it starts the copies of the next tile's values and
  // of the keys after those.
  auto next_tile = [&](uint16_t* k_free, uint16_t* v_free) {
    landed();
    copy_next(ksrc, k_free);
    copy_next(vsrc, v_free);
  };
  auto mask = [&](int t, v16f* s) {
    const int left = limit - t * kTileKeys - 4 * half;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = 32 * b + 8 * (r >> 2) + (r & 3) < left ? s[b][r] : neg_inf();
        if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few conditions alive at a time
      }
  };
  // The scores of tile t, which may be seen in part.
  auto scores = [&](int t, v16f* s, const uint16_t* kt) {
    products(s, kt);
    if (t >= my_whole) {
      mask(t, s);
    }
    move_to(largest(s), s);
  };
  // One turn of the pipeline, for a tile t that the wave sees whole: the scores of tile t + 1 (matrix
  // cores) beside the weights of tile t (vector ALUs), then tile t's values (matrix cores) beside
  // the largest of the new scores.  `part`: std::false_type where tile t + 1 is seen whole too, else
  // t + 1, whose scores are masked behind the products (in between, the registers do not suffice).
  auto turn = [&](const v16f* s, v16f* next, const uint16_t* kn, const uint16_t* vt,
                  uint16_t* k_free, uint16_t* v_free, auto part) {
    next_tile(k_free, v_free);
    products(next, kn);
    v8bf p[4];
#pragma unroll
    for (int st = 0; st < 4; ++st) p[st] = weights(s, st);
#pragma unroll
    for (int st = 0; st < 4; ++st) add_values(vt, st, p[st], std::false_type{});
    if constexpr (std::is_same<decltype(part), std::false_type>::value) {
      const float top = largest(next);
      if constexpr (D == 128) pair_up<D>();
      move_to(top, next);
    } else {
      if constexpr (D == 128) pair_up<D>();
      __builtin_amdgcn_sched_barrier(0);
      mask(part, next);
      move_to(largest(next), next);
    }
  };
  if (tiles > 0) {
    v16f sa[2];
    copy_next(ksrc, k0);
    copy_next(vsrc, v0);
    copy_next(ksrc, k1);
    landed();
    if (my_tiles > 0) scores(0, sa, k0);
    int t = 0;
    for (; t + 2 < my_whole; t += 2) {
      v16f sb[2];
      turn(sa, sb, k1, v0, k0, v1, std::false_type{});
      turn(sb, sa, k0, v1, k1, v0, std::false_type{});
    }
    if (t < my_whole && t + 1 < my_tiles) {
      v16f sb[2];
      turn(sa, sb, k1, v0, k0, v1, ++t);
      if (t < my_whole && t + 1 < my_tiles) {
        turn(sb, sa, k0, v1, k1, v0, ++t);
      } else {
        sa[0] = sb[0];
        sa[1] = sb[1];
      }
    }
    first_held = t * kTileKeys;
    for (; t < my_tiles; ++t) {  // the last tiles, among them those that are seen in part
      uint16_t *kt = t & 1 ? k1 : k0, *vt = t & 1 ? v1 : v0;
      next_tile(kt, t & 1 ? v0 : v1);
#pragma unroll
      for (int st = 0; st < 4; ++st) odd |= add_values(vt, st, weights(sa, st), std::true_type{});
      if (t + 1 < my_tiles) scores(t + 1, sa, t & 1 ? k0 : k1);
    }
    for (; t < tiles; ++t) next_tile(t & 1 ? k1 : k0, t & 1 ? v0 : v1);
  }

  const float total = sum_over_halves(sum), of_rounded = sum_over_halves(rounded[0]);
  // An infinity or a NaN of a value that a query sees reaches its output however small its weight.  In
  // the tiles seen whole it left the sum infinite or NaN (a weight of 0 makes an infinity NaN), in the
  // last ones it was held to a finite value: where there was any, the wave looks through its keys once
  // more, 32 columns at a time, and such values' own sum takes the output's place (rare: one infinity
  // early in 16384 tokens of 40 heads, 8.1 ms instead of 2.9; with a walk for each output 118).
  float most = 0.0f;  // NaN where one is (compared as an integer: the compiler takes this for a number)
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) most = __builtin_elementwise_maximum(most, __builtin_fabsf(o[i][r]));
  const bool fine = __all((__float_as_uint(most) & 0x7FFFFFFFu) < 0x7F800000u);
  if (!fine || __any(odd != 0)) {
    const int upto = min(my_tiles * kTileKeys, lk), sees = total == total ? limit : 0;  // (else all NaN)
    const uint16_t* const base = a.v + int64_t(kv0) * a.vs + int64_t(kvh) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v16f bad;
#pragma unroll
      for (int r = 0; r < 16; ++r) bad[r] = 0.0f;
      for (int j0 = fine ? first_held : 0; j0 < upto; j0 += 64) {  // a lane reads 8 values of 4 keys
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[u] = *reinterpret_cast<const uint4*>(base + min(j0 + 16 * u + (lane >> 2), upto - 1) * a.vs + 32 * i + 8 * (lane & 3));
        bool found = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          auto finite = [](uint32_t w) { return w == finite2(w); };
          uint64_t where = __ballot(!(finite(x[u].x) && finite(x[u].y) && finite(x[u].z) && finite(x[u].w)));
          while (where) {
            const int at = __builtin_ctzll(where) >> 2, j = j0 + 16 * u + at;
            where &= ~(uint64_t(15) << (4 * at));
            found = true;
            const uint16_t* src = base + min(j, upto - 1) * a.vs + 32 * i + 4 * half;
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const uint2 y = *reinterpret_cast<const uint2*>(src + 2 * r);
              const float f[4] = {bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y)};
#pragma unroll
              for (int e = 0; e < 4; ++e) bad[r + e] += j >= sees || __builtin_isfinite(f[e]) ? 0.0f : f[e];
            }
          }
        }
        if (!found) continue;
        bool done = true;  // what is NaN stays so
#pragma unroll
        for (int r = 0; r < 16; ++r) done &= bad[r] != bad[r];
        if (__all(done || sees <= j0 + 64)) break;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = bad[r] == 0.0f ? o[i][r] : bad[r];
    }
  }
  if (parts > 1) {
    if (row >= lq) return;
    const int64_t at = sums_at(a, part, head, q0 + row);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(a.sums + at * D + 32 * i + 2 * r + 4 * half) =
            make_float4(o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]);
    if (half == 0) a.stats[at] = make_float4(ref, total, of_rounded, 0.0f);
    return;
  }
  if (a.lse && half == 0 && row < lq)
    a.lse[int64_t(q0 + row) * a.hq + head] =
        total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
  // A lane holds every other four values of a row: through LDS, whole rows are stored at once (a
  // batch of eight prompts of up to 2048: 107 us, 112 with 8-byte stores to 32 rows each; alone, 37
  // queries: 6.3 us, not 6.1).  The keys' buffers are free: behind the last barrier no wave reads keys.
  const float inv = total == 0.0f ? 0.0f : 1.0f / of_rounded;
  uint16_t* const rows = (wave < kWaves / 2 ? k0 : k1) + wave % (kWaves / 2) * kWaveRows * D;
  constexpr int kTurn = kChunks < 16 ? kChunks - 1 : 15;  // rows' chunks are turned by these bits
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<uint2*>(rows + col * D + ((4 * i + r / 4) ^ (col & kTurn)) * 8 + 4 * half) =
          make_uint2(cvt_bf16x2(o[i][r] * inv, o[i][r + 1] * inv),
                     cvt_bf16x2(o[i][r + 2] * inv, o[i][r + 3] * inv));
  asm volatile("" ::: "memory");  // the wave's own writes, read by other lanes below
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < kWaveRows * kChunks / 64; ++j) {
    const int r = (64 * j + lane) / kChunks, c = lane % kChunks;
    const uint4 x = *reinterpret_cast<const uint4*>(rows + r * D + (c ^ (r & kTurn)) * 8);
    if (mine + r < lq)
      *reinterpret_cast<uint4*>(a.out + int64_t(q0 + mine + r) * a.os + int64_t(head) * D + 8 * c) = x;
  }
}

template <int D>
__global__ __launch_bounds__(64 * kPrefillWaves, D == 256 ? 1 : D == 128 ? 2 : 3) void prefill_kernel(const PrefillArgs a) {
  prefill_tile<D>(a);
}

// Adds up the parts of a work item's queries in order: D/4 lanes to a query.
constexpr int kPrefillJoinThreads = 256;
constexpr int join_rows(int d) { return kPrefillJoinThreads / (d / 4); }
template <int D>
__global__ __launch_bounds__(kPrefillJoinThreads) void prefill_join_kernel(const PrefillArgs a) {
  constexpr int kLanes = D / 4, kSplits = kPrefillRows / join_rows(D);
  const int index = blockIdx.x / kSplits;
  const int r = blockIdx.x % kSplits * join_rows(D) + int(threadIdx.x) / kLanes;
  const int d = threadIdx.x % kLanes * 4;
  Item it;
  if (!find_item(a, index, &it)) return;
  const int parts = parts_of(a, it.key_tiles(a)), row = it.tile * kPrefillRows + r;
  if (parts > 1 && row < it.lq) {
    float ref = neg_inf(), total = 0.0f, rounded = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const int64_t at = sums_at(a, p, it.head, it.q0 + row);
      const float4 x = *reinterpret_cast<const float4*>(a.sums + at * D + d);
      const float4 st = a.stats[at];
      const float to = fmaxf(ref, st.x);
      const float f = ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ref - to);
      const float h = st.x == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(st.x - to);
      ref = to;
      total = total * f + st.y * h;
      rounded = rounded * f + st.z * h;
      v.x = v.x * f + x.x * h; v.y = v.y * f + x.y * h;
      v.z = v.z * f + x.z * h; v.w = v.w * f + x.w * h;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / rounded;
    float y[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    // a part that is infinite or NaN counts whatever its weight, which may be 0 (rare)
    if (!__builtin_isfinite(v.x + v.y + v.z + v.w)) {
      float bad[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int p = 0; p < parts; ++p) {
        const float* x = a.sums + sums_at(a, p, it.head, it.q0 + row) * D + d;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad[e] += __builtin_isfinite(x[e]) ? 0.0f : x[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = bad[e] == 0.0f ? y[e] : bad[e];
    }
    *reinterpret_cast<uint2*>(a.out + int64_t(it.q0 + row) * a.os + int64_t(it.head) * D + d) =
        make_uint2(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]));
    if (a.lse && d == 0)
      a.lse[int64_t(it.q0 + row) * a.hq + it.head] =
          total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
  }
}

// Work items of a call (an upper bound: tiles of whole sequences), and the parts that their keys
// are split into: the number with the least estimated time.  A workgroup alone on its CU takes
// about 1 us a tile of 64 keys (128-wide heads), two on one CU about 2; joining parts costs a
// launch (4 us) and the way of their sums through memory, there and back at 5 TB/s.  As the lengths
// are known only in the mean here, a split has to promise a fifth of the time.  512 queries of 40 heads
// over 8704 keys: 144 us in one part, 105 in three; 23 queries over 2794 keys, 10 heads: 44 us in
// one, 17 in eleven.  The sums take at most kMostSums: more parts than fit there were estimated to
// gain 5 % in the mean and a third at most, on calls of milliseconds.
constexpr uint64_t kMostSums = uint64_t(256) << 20;
struct PrefillPlan {
  int64_t items;
  int parts;
  uint64_t sums_bytes, bytes;
};
PrefillPlan prefill_plan(int32_t seqs, int32_t total_q, int32_t total_k, int32_t hq, int32_t d) {
  PrefillPlan p = {};
  p.items = (int64_t(total_q) + int64_t(seqs) * (kPrefillRows - 1)) / kPrefillRows * hq;
  p.parts = 1;
  const int64_t cus = num_cus();
  const double tile_us = d == 256 ? 2.0 : d == 128 ? 1.0 : 0.7;
  const double mean = double(total_k) / seqs / kTileKeys;  // tiles of a sequence
  const double all = double(total_k) / kTileKeys;
  const double longest = seqs == 1 ? mean : (2 * mean < all ? 2 * mean : all);
  // under a causal mask prompts without a history see half of their keys in the mean
  const bool history = total_k > 2 * int64_t(total_q);
  const double spread = double(p.items) * mean * (history ? 1.0 : 0.5) / cus * tile_us;
  const uint64_t part_rows = uint64_t(total_q) * hq, part_bytes = part_rows * (d * 4 + 16);
  double best = 0.0;
  for (int n = 1; n <= 64 && n * kPartTiles <= longest + 1; ++n) {
    const int64_t groups = p.items * n;
    if (n > 1 && (n * part_bytes > kMostSums || (!history && groups > cus))) break;
    const int64_t rounds = groups <= cus ? 1 : 2 * ((groups + 2 * cus - 1) / (2 * cus));
    const double path = longest / n * tile_us * rounds;
    double us = path > spread ? path : spread;
    if (n > 1) us += 4.0 + double(total_q) * hq * n * d * 8 / 5e6;
    if (n == 1 || us < best * (p.parts == 1 ? 0.8 : 1.0)) {
      best = us;
      p.parts = n;
    }
  }
  if (p.parts == 1) return p;
  p.sums_bytes = p.parts * part_rows * d * 4;
  p.bytes = p.parts * part_bytes;
  return p;
}

int prefill_shape(int32_t seqs, int32_t total_q, int32_t total_k, int32_t hq, int32_t hkv, int32_t d) {
  if (seqs < 0 || total_q < 0 || total_k < 0 || total_q > (1 << 30) || total_k > (1 << 30) ||
      seqs > kMostSeqs)
    return FP8Q_EINVAL;
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0 || hq > 65536) return FP8Q_EINVAL;
  if (d != 64 && d != 128 && d != 256) return FP8Q_EINVAL;
  return FP8Q_OK;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int attn_prefill_workspace_size(int32_t num_seqs, int32_t total_q, int32_t total_k,
                                           int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, uint64_t* bytes) {
  if (!bytes) return FP8Q_ENULL;
  *bytes = 0;
  const int rc = prefill_shape(num_seqs, total_q, total_k, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
  if (num_seqs > 0 && total_q > 0)
    *bytes = prefill_plan(num_seqs, total_q, total_k, num_q_heads, head_dim).bytes;
  return FP8Q_OK;
}

extern "C" int attn_prefill(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, uint16_t* out,
                            float* lse, int32_t num_seqs, int32_t total_q, int32_t total_k,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            float softmax_scale, int32_t causal, int64_t q_stride,
                            int64_t key_stride, int64_t value_stride, int64_t out_stride,
                            void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  const int rc = prefill_shape(num_seqs, total_q, total_k, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
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
  const PrefillPlan p = prefill_plan(num_seqs, total_q, total_k, num_q_heads, head_dim);
  if (p.bytes > 0) {
    if (!workspace) return FP8Q_ENULL;
    if (!aligned(workspace, 256)) return FP8Q_EALIGN;
    if (workspace_bytes < p.bytes) return FP8Q_EINVAL;
  }
  PrefillArgs a = {};
  a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse, a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k, a.qs = q_stride, a.ks = key_stride, a.vs = value_stride;
  a.os = out_stride, a.seqs = num_seqs, a.tq = total_q, a.tk = total_k, a.hq = num_q_heads;
  a.hkv = num_kv_heads, a.causal = causal != 0, a.scale_log2 = softmax_scale * kLog2e;
  a.most_parts = p.parts, a.items = int(p.items);
  a.sums = static_cast<float*>(workspace);
  a.stats = p.bytes ? reinterpret_cast<float4*>(static_cast<uint8_t*>(workspace) + p.sums_bytes) : nullptr;
  // parts of an item lie 8 workgroups apart: whole eights of items
  const int64_t blocks = p.parts == 1 ? p.items : (p.items + 7) / 8 * 8 * p.parts;
  const int64_t joins = p.items * (kPrefillRows / join_rows(head_dim));
  if (p.items > 0x7FFFFFFF || blocks > 0x7FFFFFFF || joins > 0x7FFFFFFF) return FP8Q_EINVAL;
  auto kern = head_dim == 64 ? prefill_kernel<64> : head_dim == 128 ? prefill_kernel<128> : prefill_kernel<256>;
  launch(kern, dim3(unsigned(blocks)), dim3(64 * kPrefillWaves), 0, stream, a);
  if (launch_status() != FP8Q_OK || p.parts == 1) return launch_status();
  auto join = head_dim == 64 ? prefill_join_kernel<64>
              : head_dim == 128 ? prefill_join_kernel<128> : prefill_join_kernel<256>;
  launch(join, dim3(unsigned(joins)), dim3(kPrefillJoinThreads), 0, stream, a);
  return launch_status();
}
