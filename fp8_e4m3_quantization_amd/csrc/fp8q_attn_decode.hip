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
// so that both operands agree without an exchange.  P is rounded to bf16 for that product (by
// up to 2^-8 of each weight, as much as the output's own rounding); out's denominator is the sum of
// the rounded weights (one more row of the product, of ones), so that a weight that outweighs all
// others loses nothing by its rounding; lse is of the unrounded ones.
//
// The histories of all sequences, laid end to end, are cut into equal shares, one for each CU,
// whatever the lengths.  A workgroup's waves take the KV heads of its share side by side (a
// token's heads lie side by side in the pools) and, with fewer heads than waves, its tiles in
// turn.  A sequence that lies in several shares leaves their sums in the workspace, and a second
// kernel adds them in the sequence's order: results do not depend on the order of workgroups.  Where
// the table has room for kWholeMost positions at most, every sequence is a share of its own.
// One workgroup a CU: more read no faster.  Measured: 64 sequences of 500 to 8100 positions, 8 KV
// heads of 128 (525 MB): 95 us and 6 for the join, 5.5 TB/s; 2 of 131072 and 100003, 4 KV heads:
// 46 us and 7, 5.2 TB/s (a plain read stream: 5.9-6.2).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_attn.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kDecTile = 32;                        // positions a wave takes at a time
constexpr int kDecRows = 16;                        // query heads of a workgroup
constexpr int kDecPerCu = 1;                        // workgroups on a CU at once
// No history is cut where the table has room for at most this many positions a sequence (the host
// does not know the lengths).  The same histories behind a wider table take the second kernel too: one
// of 777 positions, 40 heads: 10.5 us with a table of 784, 12.1 with one of 32768; 128 of 300, 32
// heads, 8 KV heads: 17.1 and 26.2.
constexpr int kWholeMost = 1024;
constexpr int kJoinAtOnce = 8;                      // parts whose sums a thread has in flight

struct DecodeArgs {
  const uint16_t* q;
  const uint8_t *kc, *vc;
  const int32_t *tables, *lens;
  uint16_t* out;
  float* lse;
  float* parts;      // [2 * shares][heads of work][rows_most][D]: sums of weighted values
  float4* stats;     // [2 * shares][heads of work][rows_most]: Sums' values
  int64_t ts, qs, os, cs, nblocks;
  int seqs, width, hq, hkv, group, bs;
  int row_tiles;     // ceil(group / 16)
  int heads;         // heads of work: KV heads times row tiles
  int together;      // heads of work of a workgroup: a power of two, at most its waves
  int shares;        // places for shares of a head; 0: one share for each sequence
  int rows_most;     // min(group, 16)
  float scale_log2, v_scale;
};

__device__ __forceinline__ int seq_len(const DecodeArgs& a, int s) {
  const int n = s < a.seqs ? a.lens[s] : 0;
  return min(max(n, 0), a.width * a.bs);
}

// Sums of weights against a reference, and how two of them add up: by factors f and h, which
// hold for their weighted values too.
struct Sums {
  float ref, total, rounded;  // reference (log2 units), sums of the weights and of the rounded ones
  __device__ __forceinline__ Sums(float r, float t, float s) : ref(r), total(t), rounded(s) {}
  __device__ __forceinline__ explicit Sums(float4 x) : ref(x.x), total(x.y), rounded(x.z) {}
  __device__ __forceinline__ float4 packed() const { return make_float4(ref, total, rounded, 0.0f); }
  __device__ __forceinline__ void add(const Sums& b, float* f, float* h) {
    const float to = fmaxf(ref, b.ref);
    *f = ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ref - to);
    *h = b.ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(b.ref - to);
    ref = to;
    total = total * *f + b.total * *h;
    rounded = rounded * *f + b.rounded * *h;
  }
};

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

// Where one sequence lies among the shares.  Steps are whole tiles of every wave that works on a
// head; an empty sequence has one, which writes its zeros.
struct SeqPlace {
  int len, start, end;       // positions; its steps among all
  int first_share, parts;    // the share of its first step; how many shares it lies in
  // A share's place for sums is 2 u where the sequence began in an earlier share, else 2 u + 1.
  __device__ __forceinline__ int place(int part) const {
    return 2 * (first_share + part) + (part == 0);
  }
};
struct Cut {
  int step;  // positions
  int each;  // steps of a share
  int all;   // steps of all sequences
  __device__ __forceinline__ int steps_of(int n) const { return max((n + step - 1) / step, 1); }
  __device__ __forceinline__ int steps_at(const DecodeArgs& a, int s) const {
    return s < a.seqs ? steps_of(seq_len(a, s)) : 0;
  }
  __device__ __forceinline__ SeqPlace seq_at(int len, int start) const {
    SeqPlace p;
    p.len = len;
    p.start = start;
    p.end = start + steps_of(p.len);
    p.first_share = start / each;
    p.parts = (p.end - 1) / each - p.first_share + 1;
    return p;
  }
};
// What a lane keeps of sequence `lane` (of the first 64) for the searches that follow.
struct FirstSeqs {
  int len, steps, upto;  // length, steps, steps up to and with it
};
__device__ __forceinline__ int len_of(const DecodeArgs& a, const FirstSeqs& f, int s) {
  return s < 64 ? __builtin_amdgcn_readlane(f.len, s) : __builtin_amdgcn_readfirstlane(seq_len(a, s));
}
__device__ __forceinline__ Cut cut_up(const DecodeArgs& a, int waves, FirstSeqs* f) {
  Cut c;
  const int lane = threadIdx.x & 63;
  c.step = kDecTile * (waves / a.together);
  f->len = lane < a.seqs ? seq_len(a, lane) : 0;
  f->steps = lane < a.seqs ? c.steps_of(f->len) : 0;
  f->upto = wave_prefix(f->steps);
  c.all = __builtin_amdgcn_readlane(f->upto, 63);
  for (int s0 = 64; s0 < a.seqs; s0 += 64)
    c.all += __builtin_amdgcn_readlane(wave_prefix(c.steps_at(a, s0 + lane)), 63);
  c.each = max((c.all + a.shares - 1) / a.shares, 1);
  return c;
}

// Stores N values (4 or more) of query head `head`, from d on; the first lane of a row its lse.
template <int D, int N>
__device__ __forceinline__ void finish(const DecodeArgs& a, int seq, int head, int d, const Sums& s,
                                       const float* v) {
  const float inv = s.total == 0.0f ? 0.0f : a.v_scale / s.rounded;
  uint16_t* to = a.out + seq * a.os + int64_t(head) * D + d;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<uint2*>(to + i) = make_uint2(cvt_bf16x2(v[i] * inv, v[i + 1] * inv),
                                                   cvt_bf16x2(v[i + 2] * inv, v[i + 3] * inv));
  if (a.lse && d == 0)
    a.lse[int64_t(seq) * a.hq + head] =
        s.total == 0.0f ? neg_inf() : (s.ref + __builtin_amdgcn_logf(s.total)) * kLn2;
}

// Waves of a workgroup: 256-wide heads need twice the registers.
constexpr int waves_of(int d) { return d == 256 ? 4 : 8; }

template <int D, int kDecWaves = waves_of(D)>
__global__ __launch_bounds__(64 * kDecWaves, D == 256 ? 1 : 2) void decode_kernel(const DecodeArgs a) {
  constexpr int kSteps = D / 32;      // MFMAs of a 16-position score tile
  constexpr int kPieces = D / 64;     // 16-byte K loads of a lane and position
  constexpr int kOut = D / 16;        // MFMAs of the second product; bytes of V of a lane
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the 8 XCDs in turn: where a share has several, they stay on one.
  const int sets = a.heads / a.together;
  const int share = blockIdx.x / (8 * sets) * 8 + blockIdx.x % 8;
  const int hw0 = blockIdx.x / 8 % sets * a.together;  // first head of work here
  if (a.shares == 0 && share >= a.seqs) return;
  const int turn = wave / a.together, turns = kDecWaves / a.together;
  const int hw = hw0 + wave % a.together;          // this wave's
  const int kvh = hw / a.row_tiles;
  auto rows_of = [&](int h) { return min(kDecRows, a.group - h % a.row_tiles * kDecRows); };
  auto head_of = [&](int h) { return h / a.row_tiles * a.group + h % a.row_tiles * kDecRows; };
  const int rows = rows_of(hw);

  FirstSeqs firsts = {};
  Cut cut;
  int step = 0, seq_start = 0, seq = 0, share_end = 0;
  if (a.shares == 0) {  // this sequence, whole
    cut.step = kDecTile * turns;
    cut.each = 1 << 30;
    seq = share;
    firsts.len = seq_len(a, min(lane, a.seqs - 1));
  } else {
    cut = cut_up(a, kDecWaves, &firsts);
    step = share * cut.each;
    if (step >= cut.all) return;
    share_end = min(step + cut.each, cut.all);
  }
  for (int s0 = 0; a.shares > 0 && s0 < a.seqs; s0 += 64) {
    const int n = s0 == 0 ? firsts.steps : cut.steps_at(a, s0 + lane);
    const int upto = s0 == 0 ? firsts.upto : wave_prefix(n), here = __builtin_amdgcn_readlane(upto, 63);
    if (step < seq_start + here) {
      const int j = __builtin_ctzll(__ballot(upto > step - seq_start));
      seq = s0 + j;
      seq_start += __builtin_amdgcn_readlane(upto, j) - __builtin_amdgcn_readlane(n, j);
      break;
    }
    seq_start += here;
  }

  __shared__ int64_t s_row[kDecWaves][kDecTile];
  __shared__ __attribute__((aligned(16))) v4f s_o[kDecWaves][kOut][64];
  __shared__ __attribute__((aligned(16))) float4 s_stats[kDecWaves][64];
  const int64_t e = int64_t(a.hkv) * D;

  while (true) {  // over the share's pieces of sequences
  const SeqPlace sp = cut.seq_at(len_of(a, firsts, seq), seq_start);
  const int piece_end = a.shares == 0 ? sp.end : min(sp.end, share_end);
  const int begin = (step - seq_start) * cut.step;
  const int end = min((piece_end - seq_start) * cut.step, sp.len);
  const int part = a.shares == 0 ? 0 : share - sp.first_share;
  const int32_t* table = a.tables + seq * a.ts;

  // A tile's K and V: lane (g, col) holds K of positions col and 16 + col, and kOut bytes of V
  // of the 8 positions whose scores it will hold.  The registers of K are free for the next tile's
  // once the scores are made, those of V once the products with the weights are, so that each
  // loads during the other's half of the work.
  uint4 kx[2][kPieces];
  uint32_t vx[8][kOut / 4];
  bool ok[8];
  // The block number of lane l's position p0 + l (l < 32), one tile ahead of the loads that it
  // addresses; -1: no such position.
  auto block_of = [&](int p0) {
    const int pos = p0 + lane;
    return lane < kDecTile && pos < end ? table[uint32_t(pos) / uint32_t(a.bs)] : -1;
  };
  auto load_k = [&](int p0, int id) {
    if (lane < kDecTile) {
      const uint32_t pos = uint32_t(p0 + lane);
      const bool good = id >= 0 && id < a.nblocks;
      s_row[wave][lane] = good ? id * a.cs + int64_t(pos % uint32_t(a.bs)) * e + int64_t(kvh) * D : -1;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t at = max(s_row[wave][16 * b + col], int64_t(0));
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        kx[b][c] = *reinterpret_cast<const uint4*>(a.kc + at + 64 * c + 16 * g);
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = s_row[wave][16 * (j >> 2) + 4 * g + (j & 3)];
      ok[j] = at >= 0;
      load_bytes<kOut>(a.vc + max(at, int64_t(0)) + kOut * col, vx[j]);
    }
    __builtin_amdgcn_wave_barrier();
  };

  v8bf qf[kSteps];
  v4f o[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v4f ones_row = {0.0f, 0.0f, 0.0f, 0.0f};  // sums of the rounded weights, the same in each row
  float ref = neg_inf(), sum = 0.0f;
  float sc[8];
  auto scores = [&]() {
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
  };
  auto weigh = [&]() {
    float top = sc[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, sc[j]);
    top = max_over_rows(top);
    const bool moves = top > ref + kSoftmaxSlack;
    if (__any(moves)) {
      const float f = moves ? __builtin_amdgcn_exp2f(ref - top) : 1.0f;
      ref = moves ? top : ref;
      sum *= f;
      ones_row *= f;
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
    const v8bf ones = __builtin_bit_cast(v8bf, v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    ones_row = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pf, ones_row, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kOut; i += 2) {  // values i and i + 1 of each lane's D/16
      uint32_t pair[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = ok[j] ? vx[j][i / 4] : 0u;
        pair[j] = (i & 2) ? e4m3x2_to_bf16<true>(w) : e4m3x2_to_bf16<false>(w);
      }
      v4u even, odd;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        even[j] = __builtin_amdgcn_perm(pair[2 * j + 1], pair[2 * j], 0x05040100u);
        odd[j] = __builtin_amdgcn_perm(pair[2 * j + 1], pair[2 * j], 0x07060302u);
      }
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, even), pf, o[i], 0, 0, 0);
      o[i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, odd), pf, o[i + 1], 0, 0, 0);
    }
  };

  int p0 = begin + turn * kDecTile;
  if (p0 < end) {
    int id = block_of(p0), id_next = block_of(p0 + cut.step);
    // Queries: column l % 16 is the query head; the order of the D values follows K's loads.
    const uint16_t* src = a.q + seq * a.qs + int64_t(head_of(hw) + min(col, rows - 1)) * D;
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
      qf[c] = __builtin_bit_cast(
          v8bf, *reinterpret_cast<const uint4*>(src + 64 * (c >> 1) + 16 * g + 8 * (c & 1)));
    load_k(p0, id);
    load_v();
    while (true) {
      const int p1 = p0 + cut.step;
      id = id_next;
      id_next = block_of(p1 + cut.step);
      scores();
      if (p1 < end) load_k(p1, id);
      weigh();
      if (p1 >= end) break;
      load_v();
      p0 = p1;
    }
  }

  // o[i][r] is value kOut (4g + r) + i of query column l % 16.
  Sums sums(ref, sum_over_rows(sum), ones_row[0]);
  // The waves of a head add up in pairs, the later half leaving its registers in LDS for the
  // earlier one, which holds the same values of the same queries.
  for (int half = turns / 2; half >= 1; half /= 2) {
    if (turn >= half && turn < 2 * half) {
#pragma unroll
      for (int i = 0; i < kOut; ++i) s_o[wave][i][lane] = o[i];
      s_stats[wave][lane] = sums.packed();
    }
    __syncthreads();
    if (turn < half) {
      const int from = wave + half * a.together;
      float f, h;
      sums.add(Sums(s_stats[from][lane]), &f, &h);
#pragma unroll
      for (int i = 0; i < kOut; ++i) o[i] = o[i] * f + s_o[from][i][lane] * h;
    }
  }
  if (turn == 0 && col < rows) {
    const int64_t at = (int64_t(sp.place(part)) * a.heads + hw) * a.rows_most + col;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = kOut * (4 * g + r);
      float v[kOut];
#pragma unroll
      for (int i = 0; i < kOut; ++i) v[i] = o[i][r];
      if (sp.parts == 1) {
        finish<D, kOut>(a, seq, head_of(hw) + col, d, sums, v);
      } else {
#pragma unroll
        for (int i = 0; i < kOut; i += 4)
          *reinterpret_cast<float4*>(a.parts + at * D + d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        if (d == 0) a.stats[at] = sums.packed();
      }
    }
  }
  step = piece_end;
  if (step >= share_end) break;
  ++seq;
  seq_start = sp.end;
  __syncthreads();  // every wave has read this piece's sums in LDS
  }
}

// Adds up the parts of the sequences that lie in several shares: one workgroup per sequence and
// query head.  The D/4 lanes of a slot take every kSlots-th part; the slots' sums add up in order.
template <int D, int kJoinThreads>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const DecodeArgs a, int waves) {
  constexpr int kLanes = D / 4, kSlots = kJoinThreads / kLanes;
  const int lane = threadIdx.x & 63;
  const int head = blockIdx.x % a.hq, seq = blockIdx.x / a.hq;
  FirstSeqs firsts;
  const Cut cut = cut_up(a, waves, &firsts);
  int start = 0;
  for (int s0 = 0; s0 <= seq; s0 += 64) {
    const int n = s0 == 0 ? firsts.steps : cut.steps_at(a, s0 + lane);
    const int upto = s0 == 0 ? firsts.upto : wave_prefix(n);
    const int j = min(seq - s0, 63);
    start += __builtin_amdgcn_readlane(upto, j) - (seq - s0 < 64 ? __builtin_amdgcn_readlane(n, j) : 0);
  }
  const SeqPlace sp = cut.seq_at(len_of(a, firsts, seq), start);
  if (sp.parts == 1) return;
  const int kvh = head / a.group, of_group = head - kvh * a.group;
  const int hw = kvh * a.row_tiles + of_group / kDecRows, r = of_group % kDecRows;
  const int slot = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  Sums sums(neg_inf(), 0.0f, 0.0f);
  float4 all = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const Sums& b, float4 x) {
    float f, h;
    sums.add(b, &f, &h);
    all.x = all.x * f + x.x * h; all.y = all.y * f + x.y * h;
    all.z = all.z * f + x.z * h; all.w = all.w * f + x.w * h;
  };
  for (int c = slot; c < sp.parts; c += kSlots * kJoinAtOnce) {
    float4 v[kJoinAtOnce];
    float4 st[kJoinAtOnce];
#pragma unroll
    for (int j = 0; j < kJoinAtOnce; ++j) {
      const int part = min(c + j * kSlots, sp.parts - 1);
      const int64_t at = (int64_t(sp.place(part)) * a.heads + hw) * a.rows_most + r;
      v[j] = *reinterpret_cast<const float4*>(a.parts + at * D + d);
      st[j] = a.stats[at];
    }
#pragma unroll
    for (int j = 0; j < kJoinAtOnce; ++j)
      if (c + j * kSlots < sp.parts) add(Sums(st[j]), v[j]);
  }
  __shared__ __attribute__((aligned(16))) float s_v[kSlots][D];
  __shared__ __attribute__((aligned(16))) float4 s_st[kSlots];
  *reinterpret_cast<float4*>(&s_v[slot][d]) = all;
  if (d == 0) s_st[slot] = sums.packed();
  __syncthreads();
  if (slot > 0) return;
#pragma unroll
  for (int u = 1; u < kSlots; ++u)
    add(Sums(s_st[u]), *reinterpret_cast<const float4*>(&s_v[u][d]));
  const float v[4] = {all.x, all.y, all.z, all.w};
  finish<D, 4>(a, seq, head, d, sums, v);
}

int decode_shape(int32_t seqs, int32_t hq, int32_t hkv, int32_t d) {
  if (seqs < 0 || seqs > kMostSeqs || hq <= 0 || hkv <= 0 || hq % hkv != 0 || hq > 65536)
    return FP8Q_EINVAL;
  if (d != 64 && d != 128 && d != 256) return FP8Q_EINVAL;
  return FP8Q_OK;
}

// How a call is cut up, and the workspace that takes.
struct DecodePlan {
  int row_tiles, heads, together, shares, rows;
  uint64_t parts_bytes, bytes;
};
// `most`: the longest history that the table has room for.
DecodePlan decode_plan(int32_t hq, int32_t hkv, int32_t d, int32_t seqs, int64_t most) {
  DecodePlan p = {};
  const int group = hq / hkv;
  p.row_tiles = (group + kDecRows - 1) / kDecRows;
  p.heads = hkv * p.row_tiles;
  p.rows = group < kDecRows ? group : kDecRows;
  p.together = 1;
  // Tables of short histories: a sequence is a share, with no second kernel, and one head for all the
  // waves of a workgroup as long as that leaves no CU with two.
  if (most <= kWholeMost) {
    while (p.together < waves_of(d) && p.heads % (2 * p.together) == 0 &&
           int64_t(seqs) * (p.heads / p.together) > num_cus())
      p.together *= 2;
    return p;
  }
  while (p.together < waves_of(d) && p.heads % (2 * p.together) == 0) p.together *= 2;
  const int sets = p.heads / p.together;
  p.shares = kDecPerCu * num_cus() / sets / 8 * 8;
  if (p.shares < 8) p.shares = 8;
  const uint64_t rows = uint64_t(2 * p.shares) * p.heads * p.rows;
  p.parts_bytes = rows * d * 4;
  p.bytes = p.parts_bytes + rows * 16;
  return p;
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
  if (num_seqs > 0)
    *bytes = decode_plan(num_q_heads, num_kv_heads, head_dim, num_seqs, int64_t(1) << 30).bytes;
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
  const int64_t most = int64_t(max_blocks) * block_size;
  if (most > (int64_t(1) << 30) || num_seqs * (most / kDecTile + 1) > (int64_t(1) << 30))
    return FP8Q_EINVAL;
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
  const DecodePlan p = decode_plan(num_q_heads, num_kv_heads, head_dim, num_seqs, most);
  uint64_t need = 0;
  if (fp8_attn_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, &need) != FP8Q_OK ||
      workspace_bytes < need)
    return FP8Q_EINVAL;
  DecodeArgs a = {};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.tables = block_tables, a.lens = context_lens;
  a.out = out, a.lse = lse, a.ts = table_stride, a.qs = q_stride, a.os = out_stride;
  a.cs = cache_stride, a.nblocks = num_blocks, a.seqs = num_seqs, a.width = max_blocks;
  a.hq = num_q_heads, a.hkv = num_kv_heads, a.group = num_q_heads / num_kv_heads;
  a.bs = block_size, a.row_tiles = p.row_tiles, a.heads = p.heads, a.together = p.together;
  a.shares = p.shares, a.rows_most = p.rows;
  a.parts = static_cast<float*>(workspace);
  a.stats = reinterpret_cast<float4*>(static_cast<uint8_t*>(workspace) + p.parts_bytes);
  a.scale_log2 = softmax_scale * k_scale * kLog2e;
  a.v_scale = v_scale;
  const int64_t blocks = (p.shares > 0 ? int64_t(p.shares) : (int64_t(num_seqs) + 7) / 8 * 8) *
                         (p.heads / p.together);
  const int64_t joins = int64_t(num_seqs) * num_q_heads;
  if (blocks > 0x7FFFFFFF || joins > 0x7FFFFFFF) return FP8Q_EINVAL;
  const int waves = waves_of(head_dim);
  auto kern = head_dim == 64 ? decode_kernel<64> : head_dim == 128 ? decode_kernel<128> : decode_kernel<256>;
  launch(kern, dim3(unsigned(blocks)), dim3(64 * waves), 0, stream, a);
  if (launch_status() != FP8Q_OK) return launch_status();
  if (p.shares == 0) return FP8Q_OK;
  // Long rows of parts (few sequences) take many threads, short ones few: 2 sequences of 100 000
  // positions join in 6.8 us with 512 threads a head, 9.3 us with 128; 64 of 4 000 in 11.3 and
  // 5.8 us.
  const bool wide = p.shares / num_seqs > 16;
  void (*join)(DecodeArgs, int) =
      head_dim == 64 ? (wide ? join_kernel<64, 512> : join_kernel<64, 128>)
      : head_dim == 128 ? (wide ? join_kernel<128, 512> : join_kernel<128, 128>)
                        : (wide ? join_kernel<256, 512> : join_kernel<256, 128>);
  launch(join, dim3(unsigned(joins)), dim3(wide ? 512 : 128), 0, stream, a, waves);
  return launch_status();
}
