// fp8q_attn_chunk.hip -- attention of chunks of new tokens over the paged E4M3 KV cache: packed
// bf16 queries of sequences with one new token or thousands, grouped heads, causal from the end.
//
// Mathematics, query i of a sequence of Lq new tokens and len cached positions (the new tokens'
// own among them), over the positions j that it sees (all of them, or causal j <= i + len - Lq):
//   s_j = softmax_scale * k_scale * q . K_j
//   out = v_scale * sum_j exp(s_j - r) V_j / sum_j exp(s_j - r),  lse = r + log sum_j exp(s_j - r)
// for any reference r.  A query that sees no position gets zeros and lse = -infinity.  Scores, sums and
// statistics are binary32; the weights are rounded to bf16 for the second product, and out's
// denominator sums the rounded ones, so that a weight above all others loses nothing by it.
//
// What bounds it: bytes where each position meets few queries (64 steps of 500 to 8100 positions,
// 32/8 heads x 128: 109 us for 525 MB, 4.8 TB/s, where a copy reaches 5.1), the vector ALUs where it meets
// many (512 tokens behind 8192, 40/4 heads x 128: 112 us; 44 % of the cycles the matrix cores and 67 % the
// vector ALUs are busy, 88.7 GFLOP at 0.79 PFLOP/s): there each of a tile's four waves widens every code from
// E4M3 to bf16 for itself, beside the exponentials.
//
// Layout.  A row is a query and a head of a KV head's group, so that grouped heads share what is read.  A
// wave owns 32 rows: S^T = K Q^T leaves a row's scores in two lanes, where they are the second
// product's operand (O^T = V^T P^T) as they lie.  Codes go global -> LDS by DMA, several steps ahead, and
// are widened in registers as each wave reads them; V comes through the transposing LDS read.  (Widened
// once a workgroup into bf16 tiles in LDS, the 512 tokens took 125 us when this took 123: half the
// conversions, twice the LDS bytes and two more barriers.)
//
// Two forms.  Many rows: a workgroup takes 128 rows and steps of 64 positions, a row wave each; with 33 to 64
// rows two waves, and the other two another KV head or every other step.  Up to 32 rows: each wave takes a KV
// head, or every second or fourth block of 32 positions, in a part of LDS of its own without barriers, and
// the waves of a head add up at the end.
//
// Work is cut into parts along the positions where the batch's rows leave room (kSplitSeqs and chunk_plan say
// where they are taken not to, and what that costs): every workgroup reads all lengths, estimates the time of 64
// ways to cut and takes the best (see find_limit); the parts' sums go through the workspace to a second kernel
// that adds them up in their order.  No atomics: the same bits every time.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp8q.h"
#include "fp8q_attn_tile.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kTileRows = 128;   // rows (query, head of a KV head's group) of a workgroup
constexpr int kThreads = 256;
// Batches of more sequences are not split along the positions: the estimate goes over all of them in every
// workgroup, which histories that are alike pay for and uneven ones would gain by.  32/8 heads x 128, as it is and
// with the estimate for any number: 300 steps of 500 positions 71 and 91 us, 300 of 100 to 1700 126 and 141, 1024
// of 500 210 and 234; but 300 of 500 and one of 8000 317 and 100, of 100000 3328 and 135: one workgroup for four KV
// heads then walks the longest history, and takes the longer the longer it is.
constexpr int kSplitSeqs = 256;
// Nor are those whose tables have room for so many positions at most, which one kernel is faster for: 200
// positions of 1, 5, 37 and 200 tokens, 40/4 heads: 12.7, 14.2, 13.4 and 12.2 us whole, 13.3, 14.9, 16.8 and 15.6
// with parts and their join; 400 positions: 17.4, 18.8, 16.8, 17.1 and 13.6, 15.7, 20.3, 20.3.
constexpr int kShort = 256;
// So many rows of a sequence and KV head at most: the waves divide heads and positions instead of rows.  64
// sequences of 12 tokens (48 rows) over 500 to 8100 positions 141 us, as part of a tile of 128 rows 185; 64
// steps (4 rows) 109, 172 there.
constexpr int kFewRows = 64;
constexpr int kMinPart = 4;      // tiles of positions of a part, at least (2 to 8: alike)
constexpr int kMinFewPart = 1;   // the same of few rows
// Times, in that of a tile of positions of a workgroup of many rows that shares its compute unit:
constexpr float kFewCost = 0.8f;    // a tile of positions of few rows, for each KV head
constexpr float kAloneCost = 0.6f;  // a tile of a workgroup alone on its compute unit (as if 1: 16
                                    // sequences of 4 tokens 32 -> 36 us)
constexpr float kPieceCost = 2.0f;  // a workgroup's start and end
constexpr float kJoinCost = 0.011f; // a part's sums, written and read again

struct ChunkArgs {
  const uint16_t* q;
  const uint8_t *kc, *vc;
  const int32_t *tables, *lens, *cu;
  uint16_t* out;
  float* lse;     // [tq, hq] or NULL
  float* sums;    // [hkv * slots][kTileRows][D]: sums of weighted values of parts
  float4* stats;  // [hkv * slots][kTileRows]: reference (log2 units), sums of the weights and of the
                  // rounded ones
  int4* parts;    // [hkv * slots], and one more: the number of those in use
  int64_t ts, qs, os, cs, nblocks;
  FastDiv by_group, by_block;
  int seqs, width, tq, hq, hkv, group, bs, causal;
  int most_heads;  // KV heads that a piece of few rows takes at most: 1, 2 or 4
  int slots;       // pieces of a KV head when sequences are split; 0: they are not
  float resident;  // pieces of a KV head that run at once
  float scale_log2, v_scale;
};

// The kernel's arguments, read again from where the launch left them: scalars that a loop does not need
// take no registers from it.
__device__ __forceinline__ const ChunkArgs& own_args() {
  typedef const __attribute__((address_space(4))) ChunkArgs* Kernarg;
  Kernarg p = (Kernarg)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ChunkArgs*)p;
}

// A sequence, whatever the lists hold: its first query row, queries and positions; and how its rows
// of a KV head are worked on.
struct Seq {
  int q0, lq, len;
  __device__ __forceinline__ Seq(const ChunkArgs& a, int s) {
    q0 = lq = len = 0;
    if (s >= a.seqs) return;
    const int from = min(max(a.cu[s], 0), a.tq);
    q0 = from;
    lq = min(max(a.cu[s + 1], from), a.tq) - from;
    len = min(max(a.lens[s], 0), a.width * a.bs);
  }
  __device__ __forceinline__ int rows(const ChunkArgs& a) const { return lq * a.group; }
  __device__ __forceinline__ bool few(const ChunkArgs& a) const { return rows(a) <= kFewRows; }
  __device__ __forceinline__ int tiles(const ChunkArgs& a) const { return (rows(a) + kTileRows - 1) / kTileRows; }
  // tiles of positions
  __device__ __forceinline__ int steps() const { return lq > 0 ? (len + kTileKeys - 1) / kTileKeys : 0; }
  // KV heads of a piece: a token's heads lie side by side in the pools, and one head's rows read
  // alone stream slower (64 steps over 32/8 heads: 137 us of one head a piece, 116 of two, 109 of four)
  __device__ __forceinline__ int heads(const ChunkArgs& a) const {
    return few(a) ? min(a.most_heads, rows(a) > kWaveRows ? 2 : 4) : 1;
  }
  // Time of a tile of positions in a piece.
  __device__ __forceinline__ float tile_cost(const ChunkArgs& a) const {
    return few(a) ? kFewCost * float(heads(a)) : 1.0f;
  }
  // Parts that the positions may be cut into.
  __device__ __forceinline__ int cap(const ChunkArgs& a) const {
    return max(steps() / (few(a) ? kMinFewPart : kMinPart), 1);
  }
};

template <int kCtrl, int kRowMask>
__device__ __forceinline__ float row_step(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRowMask, 0xF, false));
}

// Parts, `cap` at most, of a sequence whose pieces take `cost` when one takes at most about `most`.  The
// same arithmetic in every workgroup: all agree.
__device__ __forceinline__ float parts_of(float cost, int cap, float most) {
  return fmaxf(fminf(__builtin_ceilf(cost * __builtin_amdgcn_rcpf(most)), float(cap)), 1.0f);
}

// Sums, and largest of values that are not negative, over the wave.
template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
  v = op(v, row_step<0x111, 0xF>(v));  // row_shr:1
  v = op(v, row_step<0x112, 0xF>(v));
  v = op(v, row_step<0x114, 0xF>(v));
  v = op(v, row_step<0x118, 0xF>(v));
  v = op(v, row_step<0x142, 0xA>(v));  // row_bcast:15 into rows 1 and 3
  v = op(v, row_step<0x143, 0xC>(v));  // row_bcast:31 into rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float x, float y) { return fmaxf(x, y); });
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }

// A piece of work: a tile of rows of one sequence and KV head, or the few rows of a sequence for
// several KV heads; and the positions that it goes over.
struct Piece {
  int seq, q0, lq, len;  // the sequence's first query row, queries and positions
  int row0, rows;        // the tile's first row of the sequence's, and how many
  int kvh, heads;        // the first KV head, and how many
  int part, parts, from, to;  // tiles of positions [from, to)
  int slot;              // where the sums of a part go
  // positions [0, seen(i)) are seen by query i
  __device__ __forceinline__ int seen(const ChunkArgs& a, int i) const {
    return a.causal ? min(max(i + len - lq + 1, 0), len) : len;
  }
};

// The limit on the time of a piece, from which the parts of each sequence follow (none: 1e9).  64 limits
// are tried, a lane each: from the time that all pieces would take in equal shares on, in steps of
// 2.5 %; the least estimated time wins.  All threads call it; lds: 4 KB.
__device__ __forceinline__ float find_limit(const ChunkArgs& a, const Seq& first, uint8_t* lds) {
  const int lane = threadIdx.x & 63;
  float total = 0.0f, pieces = 0.0f;
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const Seq q = s0 == 0 ? first : Seq(a, s0 + lane);
    const float cost = float(q.steps()) * q.tile_cost(a), n = float(q.tiles(a)) * (1.0f / float(q.heads(a)));
    pieces += n;
    // (under a causal mask the mean tile sees half a chunk less than the last one)
    total += n * (a.causal ? fmaxf(cost - float(q.lq) * (0.5f / kTileKeys), 0.5f * cost) : cost);
  }
  total = wave_sum(total);
  pieces = wave_sum(pieces);
  if (pieces + 2.0f >= float(a.slots)) return 1e9f;
  const float share = total * __builtin_amdgcn_rcpf(a.resident);
  const float limit = lane == 63 ? 1e9f : share * 0.75f * __builtin_amdgcn_exp2f(float(lane) * 0.035624f);
  // (of many sequences the four waves take every fourth each)
  const bool shared = a.seqs > 8;
  float sum = 0.0f, split = 0.0f, top = 0.0f;  // pieces, those that are parts, the longest one's time
  for (int s0 = 0; s0 < a.seqs; s0 += 64) {
    const Seq q = s0 == 0 ? first : Seq(a, s0 + lane);
    const int cap = q.cap(a);
    const float cost = float(q.steps()) * q.tile_cost(a), n = float(q.tiles(a)) * (1.0f / float(q.heads(a)));
    for (int j = shared ? threadIdx.x >> 6 : 0; j < min(a.seqs - s0, 64); j += shared ? 4 : 1) {
      auto of = [&](float x) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), j)); };
      const float sc = of(cost), sn = of(n);
      const float p = parts_of(sc, __builtin_amdgcn_readlane(cap, j), limit);
      sum += sn * p;
      split += p > 1.0f ? sn * p : 0.0f;
      top = fmaxf(top, sn > 0.0f ? sc * __builtin_amdgcn_rcpf(p) : 0.0f);
    }
  }
  if (shared) {
    float4* const each = reinterpret_cast<float4*>(lds);
    each[threadIdx.x] = make_float4(sum, split, top, 0.0f);
    __syncthreads();
    sum = split = top = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 x = each[w * 64 + lane];
      sum += x.x;
      split += x.y;
      top = fmaxf(top, x.z);
    }
    __syncthreads();
  }
  // Pieces that run at once take the longest one's time, alone on a compute unit less; more pieces
  // share the time of all, and wait for half a last one.  Each piece takes kPieceCost to start, and
  // its sums' way through memory where it is a part.
  float time = sum <= a.resident ? (sum <= 0.5f * a.resident ? kAloneCost : 1.0f) * top + kPieceCost
                                 : (total + kPieceCost * sum) * __builtin_amdgcn_rcpf(a.resident) + 0.5f * top;
  time += kJoinCost * float(a.hkv) * split;
  if (sum + 2.0f > float(a.slots)) time = 1e30f;
  // the least time, as the largest difference of the bits from an upper end's
  const float key = __uint_as_float(0x7F000000u - __float_as_uint(time));
  const uint64_t where = __ballot(key == wave_max(key) && time < 1e30f);
  return where ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(limit), __builtin_ctzll(where))) : 1e9f;
}

// Piece `u` of those of KV head `kvh`, or false.  Pieces for several heads are dealt out to those heads'
// lists in turn.  Pieces of long time come first.  `used`: the slots that all parts take.  All threads
// call it; lds: 4 KB.
__device__ __forceinline__ bool find_piece(const ChunkArgs& a, int kvh, int u, uint8_t* lds, Piece* pc,
                                           int* used) {
  const int lane = threadIdx.x & 63;
  const Seq first(a, lane);
  const float most = a.slots > 0 ? find_limit(a, first, lds) : 1e9f;
  bool found = false;
  int before = 0;
  *used = 0;
  // (without a limit no piece's time is long, and no part takes a slot)
  const bool whole = most >= 1e9f;
  for (int order = whole ? 1 : 0; order < 2; ++order) {
    int dealt2 = 0, dealt4 = 0, slots = 0;  // of the sequences so far
    for (int s0 = 0; s0 < a.seqs && !(whole && found); s0 += 64) {
      const Seq q = s0 == 0 ? first : Seq(a, s0 + lane);
      const int n = q.tiles(a), heads = q.heads(a), shift = heads >> 1;
      const float cost = float(q.steps()) * q.tile_cost(a);
      const float fp = a.slots > 0 ? parts_of(cost, q.cap(a), most) : 1.0f;
      const int p = int(fp);
      // the parts of this sequence that fall to this head's list, and the first of them
      const int all = heads > 1 && n > 0 ? p : 0;
      const int upto2 = wave_prefix(heads == 2 ? all : 0), upto4 = wave_prefix(heads == 4 ? all : 0);
      const int base = heads == 2 ? dealt2 + upto2 - all : dealt4 + upto4 - all;
      dealt2 += last_lane(upto2);
      dealt4 += last_lane(upto4);
      const int r = kvh & (heads - 1), skip = heads - 1 - r;
      const int deal = ((base + all + skip) >> shift) - ((base + skip) >> shift);
      const int p0 = (r - base) & (heads - 1);
      const int own_slots = p == 1 || n == 0 ? 0 : heads > 1 ? p * (a.hkv >> shift) : n * p * a.hkv;
      const int slots_upto = wave_prefix(own_slots);
      const bool is_long = cost > 0.5f * most * fp;
      const int mine = is_long == (order == 0) ? heads > 1 ? deal : n * p : 0;
      const int upto = wave_prefix(mine), here = last_lane(upto);
      if (!found && u < before + here) {
        const int j = __builtin_ctzll(__ballot(upto > u - before));
        auto of = [&](int x) { return __builtin_amdgcn_readlane(x, j); };
        const int i = u - before - (of(upto) - of(mine));
        pc->seq = s0 + j;
        pc->q0 = of(q.q0);
        pc->lq = of(q.lq);
        pc->len = of(q.len);
        pc->parts = of(p);
        pc->heads = of(heads);
        int tile = 0;
        if (pc->heads > 1) {
          pc->part = of(p0) + i * pc->heads;
          pc->kvh = kvh & ~(pc->heads - 1);
        } else {
          tile = of(n) - 1 - i / pc->parts;
          pc->part = i % pc->parts;
          pc->kvh = kvh;
        }
        pc->row0 = tile * kTileRows;
        pc->slot = slots + of(slots_upto) - of(own_slots) +
                   (pc->heads > 1 ? (pc->kvh >> (pc->heads >> 1)) : tile * a.hkv + pc->kvh) * pc->parts + pc->part;
        found = true;
      }
      before += here;
      slots += last_lane(slots_upto);
    }
    *used = slots;
    if (found) break;
  }
  if (!found) return false;
  pc->rows = min(pc->lq * a.group - pc->row0, kTileRows);
  const int last = int(a.by_group.div(pc->row0 + pc->rows - 1));
  const int steps = (pc->seen(a, last) + kTileKeys - 1) / kTileKeys;
  // (an early tile of a prompt sees less: some of its parts may be empty)
  pc->from = int(int64_t(steps) * pc->part / pc->parts);
  pc->to = int(int64_t(steps) * (pc->part + 1) / pc->parts);
  return true;
}

// What the kernel's two forms share: a piece, and the lane's place in it.
template <int D>
struct Work {
  Piece pc;
  int kvh;
  int wave_end;    // positions [0, wave_end) are seen by some row of the wave
  bool any_bad;    // some position of the piece lies in a block that does not exist

  // A position's block (behind the last position: the last one's).
  __device__ __forceinline__ int block_at(const ChunkArgs& a, int pos) const {
    return a.tables[pc.seq * a.ts + a.by_block.div(min(pos, pc.len - 1))];
  }
  // Scores of positions that a row does not see, or that lie in blocks that do not exist, are
  // -infinity; s holds positions p0 .. p0 + 32 kBlocks - 1.  Returns a bit for each of the lane's positions that some
  // row of the wave sees: NaN codes of the others' values (stale ones behind a sequence's end, those of a block in
  // the place of one that does not exist) do not count, nor do they start take_nans, which goes over positions one
  // by one (64 steps of 500 to 8100 positions behind a block that does not exist, stale codes NaN: 2850 us with it, 186
  // without).
  template <int kBlocks>
  __device__ __forceinline__ uint32_t mask(v16f* s, int p0, int limit) const {
    const int half = (threadIdx.x & 63) >> 5, left = limit - p0 - 4 * half;
    // (of every eight positions the lane has four)
    const int any_left = wave_end - p0 - 4 * half;
    const int n = min(max(4 * (any_left >> 3) + min(any_left & 7, 4), 0), 16 * kBlocks);
    uint32_t counts = uint32_t((uint64_t(1) << n) - 1);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = 32 * b + 8 * (r >> 2) + (r & 3) < left ? s[b][r] : neg_inf();
        if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few conditions alive at a time
      }
    if (any_bad) {  // rare
      const ChunkArgs& a = own_args();
      uint32_t good = 0;
#pragma unroll 1
      for (int i = 0; i < 16 * kBlocks; ++i) {
        const int pos = p0 + 32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3) + 4 * half;
        good |= uint32_t(uint32_t(block_at(a, pos)) < a.nblocks) << i;
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = good >> (16 * b + r) & 1 ? s[b][r] : neg_inf();
      counts &= good;
    }
    return counts;
  }
  // NaN codes that were left out of positions from `first` on reach a row that sees them.
  __device__ __forceinline__ void take_nans(RowSums<D>& sums, int first, int limit) const {
    const ChunkArgs& a = own_args();
    const int half = (threadIdx.x & 63) >> 5, end = min(limit, min(pc.to * kTileKeys, pc.len));
    for (int pos = first; pos < end; ++pos) {
      const int id = block_at(a, pos);
      if (uint32_t(id) >= a.nblocks) continue;
      const int off = pos - int(a.by_block.div(pos)) * a.bs;
      const uint8_t* v = a.vc + id * a.cs + off * (int64_t(a.hkv) * D) + int64_t(kvh) * D + 4 * half;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const uint32_t nan = e4m3_nan_bytes(*reinterpret_cast<const uint32_t*>(v + 32 * i + 2 * r));
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (nan >> (8 * t + 7) & 1) sums.o[i][r + t] = __builtin_nanf("");
        }
    }
  }
};

// Rows of codes that a lane copies into LDS, tile after tile: where the next ones lie.  A row's
// block number is read one tile before the copy that it addresses.
template <int D, int kRows>
struct Rows {
  static constexpr int kLanes = D / 16;              // lanes that copy a row
  static constexpr int kAtOnce = 64 / kLanes;        // rows of a copy of 1 KB
  int block[kRows], off[kRows];  // of the rows whose block number is read next
  int id[kRows];                 // block numbers of the rows that are copied next
  int at[kRows];                 // their places within the blocks
  int step_blocks, step_off;     // from tile to tile

  __device__ __forceinline__ void start(const ChunkArgs& a, int pos0, int row_step, int step) {
    step_blocks = int(a.by_block.div(step));
    step_off = step - step_blocks * a.bs;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int pos = pos0 + j * row_step;
      block[j] = int(a.by_block.div(pos));
      off[j] = pos - block[j] * a.bs;
    }
  }
  // Rows behind the last position come from its block: what lies there is masked.
  __device__ __forceinline__ void read_ids(const ChunkArgs& a, const int32_t* table, int last_block) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      id[j] = table[min(block[j], last_block)];
      at[j] = off[j];
      off[j] += step_off;
      const bool over = off[j] >= a.bs;
      block[j] += step_blocks + (over ? 1 : 0);
      off[j] -= over ? a.bs : 0;
    }
  }
  // Where the rows that are copied next lie.  A block that does not exist is replaced by the first
  // one: what is read there does not count.
  __device__ __forceinline__ void places(const ChunkArgs& a, int64_t* to) const {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint32_t good = uint32_t(id[j]) < a.nblocks ? id[j] : 0;
      to[j] = int64_t(uint64_t(good) * uint32_t(a.cs) + uint64_t(uint32_t(at[j])) * uint32_t(a.hkv * D));
    }
  }
};

// A copy of 16 bytes a lane into 1 KB of LDS.
__device__ __forceinline__ void copy16(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 16, 0, 0);
}

// s_waitcnt's operands for vmcnt(n), alone and with lgkmcnt(0).
constexpr int until_vmcnt(int n) { return (n & 15) | (n >> 4) << 14 | 0x0F70; }
constexpr int until_read_and_vmcnt(int n) { return until_vmcnt(n) & ~0x0F00; }

// Workgroups of a compute unit: as many as registers allow without spills in the loops (two 64-wide prompts: 90 us
// at two, 87 at three, 97 at four).
template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 128 ? 2 : 3) void chunk_kernel(const ChunkArgs) {
  const ChunkArgs& a = own_args();
  // Four tiles of codes, keys then values
  constexpr int kTileBytes = kTileKeys * D;
  __shared__ __attribute__((aligned(16))) uint8_t t0[2 * kTileBytes], t1[2 * kTileBytes];
  __shared__ __attribute__((aligned(16))) uint8_t t2[2 * kTileBytes], t3[2 * kTileBytes];
  __shared__ int s_flags[2][4];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups go to the 8 XCDs in turn; where the KV heads divide, an XCD works on the same ones.
  int kvh, u;
  {
    const int x = blockIdx.x % 8, y = blockIdx.x / 8;
    if (a.hkv % 8 == 0) {
      kvh = x * (a.hkv / 8) + y % (a.hkv / 8);
      u = y / (a.hkv / 8);
    } else if (8 % a.hkv == 0) {
      kvh = x % a.hkv;
      u = y * (8 / a.hkv) + x / a.hkv;
    } else {
      kvh = blockIdx.x % a.hkv;
      u = blockIdx.x / a.hkv;
    }
  }
  // Whether `x` holds in any lane of any wave, at the next barrier.
  auto tell = [&](int i, bool x) {
    const bool mine = __any(x);
    if (lane == 0) s_flags[i][wave] = mine;
  };
  auto told = [&](int i) {
    return __builtin_amdgcn_readfirstlane(s_flags[i][0] | s_flags[i][1] | s_flags[i][2] | s_flags[i][3]) != 0;
  };
  Piece pc;
  int used;
  const bool any = find_piece(a, kvh, u, t3, &pc, &used);
  if (a.slots > 0 && blockIdx.x == 0 && tid == 0) a.parts[a.slots * a.hkv] = make_int4(used, 0, 0, 0);
  if (!any) return;

  // Few rows: the waves take different KV heads, and different positions, instead of different rows.
  const bool few = pc.lq * a.group <= kFewRows;
  const int row_waves = !few ? 4 : pc.rows > kWaveRows ? 2 : 1, width = row_waves * pc.heads;
  const int key_waves = 4 / width, key_wave = wave / width;
  const int head_wave = (wave & (width - 1)) / row_waves;
  const int mine = (wave & (row_waves - 1)) * kWaveRows;   // this wave's first row of the tile
  const int row = mine + col;                              // this lane's
  const int slot_row = head_wave * row_waves * kWaveRows + row;
  kvh = pc.kvh + head_wave;
  if (pc.parts > 1 && tid == 0)
    a.parts[pc.slot] = make_int4(pc.q0, pc.row0, pc.rows | row_waves << 8 | pc.heads << 12 | pc.kvh << 16,
                                 pc.part | pc.parts << 16);
  auto query_of = [&](int r) { return int(a.by_group.div(pc.row0 + r)); };
  // (later queries see more)
  const int wave_end = mine < pc.rows ? pc.seen(a, query_of(min(mine + kWaveRows, pc.rows) - 1)) : 0;
  Work<D> wk{pc, kvh, __builtin_amdgcn_readfirstlane(wave_end), false};
  const int my_row = min(row, pc.rows - 1), my_query = query_of(my_row);
  const int my_head = kvh * a.group + pc.row0 + my_row - my_query * a.group;
  const int limit = row < pc.rows ? pc.seen(a, my_query) : 0;
  // positions that all rows of the tile see
  const int all_see = __builtin_amdgcn_readfirstlane(pc.seen(a, query_of(0)));

  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(pc.q0 + my_query) * a.qs + int64_t(my_head) * D + 16 * half;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 32 * (s >> 1) + 8 * (s & 1)));
  }
  const int last_block = int(a.by_block.div(max(pc.len - 1, 0)));
  // Whether all blocks exist, which the table tells beside the first copies: a first number of each
  // thread's is read before those.
  const int first_block = int(a.by_block.div(pc.from * kTileKeys)) + tid;
  const int end_block = pc.from < pc.to ? int(a.by_block.div(min(pc.to * kTileKeys, pc.len) - 1)) + 1 : 0;
  const int32_t* const table = a.tables + pc.seq * a.ts;
  const int one_id = first_block < end_block ? table[first_block] : 0;
  auto look_for_bad = [&]() {
    bool bad = uint32_t(one_id) >= a.nblocks;
    for (int i = first_block + kThreads; i < end_block; i += kThreads) bad |= uint32_t(table[i]) >= a.nblocks;
    tell(0, bad);
    __syncthreads();
    wk.any_bad = told(0);
  };

  RowSums<D> sums;
  sums.clear();
  const float scale = a.scale_log2;
  uint32_t odd = 0;  // not 0: NaN codes of values were left out that some row sees, from first_left_out on
  int first_left_out = pc.from * kTileKeys;
  const uint8_t* const kc = a.kc + int64_t(kvh) * D;
  const uint8_t* const vc = a.vc + int64_t(kvh) * D;

  // A wave's rows over 32 kBlocks positions from p0 on, whose codes lie in LDS; with kEdge they may be
  // seen in part.
  auto attend = [&](const uint8_t* ks, const uint8_t* vs, int p0, auto blocks, auto edge,
                    int lane) __attribute__((always_inline)) {
    constexpr int kBlocks = decltype(blocks)::value;
    constexpr bool kEdge = decltype(edge)::value;
    v16f s[kBlocks];
    code_scores<D, kBlocks>(s, ks, qf, lane);
    // values are read before the weights are made, as registers allow (512 behind 8192 113 us, after them 116;
    // 256-wide heads 66 after them, before them 87: spills)
    constexpr int kSteps = 2 * kBlocks, kEarly = D == 256 ? 0 : kSteps;
    v2u y[kSteps][D / 32];
    auto read_values = [&](int st) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[st][i] = value_codes<D>(vs, st, i, lane);
    };
#pragma unroll
    for (int st = 0; st < kEarly; ++st) read_values(st);
    uint32_t counts = 0;
    if constexpr (kEdge) counts = wk.template mask<kBlocks>(s, p0, limit);
    v8bf p[kSteps];
    sums.template weigh<kBlocks>(s, scale, p);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      if (st >= kEarly) read_values(st);
      sums.template add_values<kEdge>(y[st], p[st], counts >> (8 * st), &odd);
    }
  };

  if (row_waves == 1) {
    // Each wave takes every key_waves-th block of 32 positions, two blocks ahead in LDS.
    const int lane = own_lane();
    const ChunkArgs& a = own_args();
    constexpr int kCopies = D / 32;                        // copies of a block's keys, or values
    typedef Rows<D, kCopies> R;
    const int f_row = lane / R::kLanes, f_place = lane % R::kLanes;
    const int end = min(2 * pc.to, (pc.len + 31) / 32);
    int n = 2 * pc.from + key_wave;
    R rows;
    // Copies of the next block, after the block numbers of the one behind it: what waits for those
    // need not wait for the copies.
    auto copy_at = [&](const int64_t* at, uint8_t* ks, uint8_t* vs) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int r = j * R::kAtOnce + f_row;
        copy16(kc + at[j] + (f_place ^ key_turn<D>(r)) * 16, ks + j * 1024);
        copy16(vc + at[j] + (f_place ^ value_turn<D>(r)) * 16, vs + j * 1024);
      }
    };
    auto copy_block = [&](uint8_t* ks, uint8_t* vs) {
      int64_t at[kCopies];
      rows.places(a, at);
      rows.read_ids(a, table, last_block);
      asm volatile("" ::: "memory");
      copy_at(at, ks, vs);
    };
    // Waits for block n, takes it, and copies the one after the next into its place.
    auto turn = [&](uint8_t* ks, uint8_t* vs, auto edge, int lane) __attribute__((always_inline)) {
      asm volatile("" ::: "memory");
      // this block's copies have landed: at most the next one's have not
      if (n + key_waves < end) __builtin_amdgcn_s_waitcnt(until_vmcnt(2 * kCopies));
      else __builtin_amdgcn_s_waitcnt(until_vmcnt(0));
      asm volatile("" ::: "memory");
      attend(ks, vs, 32 * n, std::integral_constant<int, 1>{}, edge, lane);
      if (n + 2 * key_waves < end) {
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this block has been read
        asm volatile("" ::: "memory");
        copy_block(ks, vs);
      }
      n += key_waves;
    };
    const int mine32 = wave * 32 * D;
    if (n < end) {
      rows.start(a, 32 * n + f_row, R::kAtOnce, 32 * key_waves);
      // (the first blocks' block numbers are read all at once)
      rows.read_ids(a, table, last_block);
      R next = rows;
      next.read_ids(a, table, last_block);
      int64_t at[2][kCopies];
      rows.places(a, at[0]);
      next.places(a, at[1]);
      rows = next;
      rows.read_ids(a, table, last_block);
      copy_at(at[0], t0 + mine32, t1 + mine32);
      if (n + key_waves < end) copy_at(at[1], t2 + mine32, t3 + mine32);
    }
    look_for_bad();
    if (n < end) {
      const int whole = wk.any_bad ? 0 : min(end, all_see / 32);  // blocks that all rows see
      first_left_out = max(first_left_out, 32 * whole);
      int odd_turn = 0;
      while (n < whole) {
        turn(t0 + mine32, t1 + mine32, std::false_type{}, lane);
        odd_turn = 1;
        if (n >= whole) break;
        turn(t2 + mine32, t3 + mine32, std::false_type{}, lane);
        odd_turn = 0;
      }
      while (n < end) {
        const int lane = own_lane();
        turn((odd_turn ? t2 : t0) + mine32, (odd_turn ? t3 : t1) + mine32, std::true_type{}, lane);
        odd_turn ^= 1;
      }
    }
  } else {
    // The waves share what is copied, four steps in LDS: of 64 positions, whose rows all waves go over,
    // or, with two waves of rows, of two times 32 positions (of two KV heads, or in a row), which two
    // waves each go over.
    auto go = [&](auto blocks) __attribute__((always_inline)) {
      constexpr int kBlocks = decltype(blocks)::value;
      // rows that a lane copies, of keys and values or of either
      constexpr int kRows = kBlocks == 2 ? D / 64 : D / 32;
      constexpr int kCopies = D / 32;                         // copies of a wave and step
      typedef Rows<D, kRows> R;
      const int lane = own_lane();
      const ChunkArgs& a = own_args();
      const int sub = kBlocks == 2 ? 0 : wave >> 1, side = wave & 1;
      const int step = kBlocks == 2 ? kTileKeys : 32 * key_waves;
      const int keys_at = sub * 64 * D, values_at = keys_at + (kBlocks == 2 ? kTileBytes : 32 * D);
      // the first position that this wave goes over
      const int start = pc.from * kTileKeys + (kBlocks == 1 && key_waves == 2 ? 32 * sub : 0);
      const int f_row = (kBlocks == 2 ? wave * kRows * R::kAtOnce : 0) + lane / R::kLanes, f_place = lane % R::kLanes;
      R rows;
      rows.start(a, start + f_row, R::kAtOnce, step);
      // Copies of the next step, after the block numbers of the one behind it: what waits for those
      // need not wait for the copies.
      auto copy_step = [&](const int64_t* at, uint8_t* to) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int r = f_row + j * R::kAtOnce;
          const int k = (f_place ^ key_turn<D>(r)) * 16, v = (f_place ^ value_turn<D>(r)) * 16;
          if constexpr (kBlocks == 2) {
            copy16(kc + at[j] + k, to + (wave * kRows + j) * 1024);
            copy16(vc + at[j] + v, to + kTileBytes + (wave * kRows + j) * 1024);
          } else {  // one of the two waves copies keys, the other values
            copy16((side ? vc + v : kc + k) + at[j], to + (side ? values_at : keys_at) + j * 1024);
          }
        }
      };
      auto copy_next = [&](uint8_t* to) {
        int64_t at[kRows];
        rows.places(a, at);
        rows.read_ids(a, table, last_block);
        asm volatile("" ::: "memory");
        copy_step(at, to);
      };
      const int steps = (min(pc.to * kTileKeys, pc.len) - pc.from * kTileKeys + step - 1) / step;
      if (steps > 0) {
        // (the first steps' block numbers are read all at once)
        rows.read_ids(a, table, last_block);
        R next = rows;
        next.read_ids(a, table, last_block);
        R third = next;
        third.read_ids(a, table, last_block);
        int64_t at[3][kRows];
        rows.places(a, at[0]);
        next.places(a, at[1]);
        third.places(a, at[2]);
        rows = third;
        rows.read_ids(a, table, last_block);
        copy_step(at[0], t0);
        copy_step(at[1], t1);
        copy_step(at[2], t2);
      }
      look_for_bad();
      if (steps <= 0) return;
      // steps that all rows see
      const int whole = wk.any_bad ? 0 : max(all_see - pc.from * kTileKeys, 0) / step;
      // Step t: at its barrier all waves' copies of it have landed (at most those of the two after it have
      // not), and the step before it has been read by all: step t + 3 takes its place.  (Nothing is
      // written to LDS but by copies: no fence is needed, which would wait for all of them.)  With kEdge it
      // may be seen in part.
      int t = 0;
      auto turn = [&](const uint8_t* here, uint8_t* free, auto edge, int lane) __attribute__((always_inline)) {
        constexpr bool kEdge = decltype(edge)::value;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(until_read_and_vmcnt(kEdge ? 0 : 2 * kCopies));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (!kEdge || t + 3 < steps) copy_next(free);
        attend(here + keys_at, here + values_at, start + t * step, blocks, edge, lane);
        ++t;
      };
      const int most = min(whole, steps);
      while (t < most) {
        turn(t0, t3, std::false_type{}, lane);
        if (t >= most) break;
        turn(t1, t0, std::false_type{}, lane);
        if (t >= most) break;
        turn(t2, t1, std::false_type{}, lane);
        if (t >= most) break;
        turn(t3, t2, std::false_type{}, lane);
      }
      first_left_out += t * step;
      while (t < steps) {  // the last steps, which may be seen in part
        auto slot_of = [&](int i) { return i & 2 ? i & 1 ? t3 : t2 : i & 1 ? t1 : t0; };
        turn(slot_of(t), slot_of(t + 3), std::true_type{}, own_lane());
      }
      __builtin_amdgcn_s_waitcnt(until_vmcnt(0));  // copies behind the last step: LDS is used again
    };
    if (row_waves == 4) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1>{});
  }

  // NaN codes that were left out reach the rows that see them.
  tell(1, odd != 0);
  __syncthreads();
  if (told(1) && key_wave == 0) wk.take_nans(sums, first_left_out, limit);

  {
  const ChunkArgs& a = own_args();
  float ref = sums.ref, total = sum_over_halves(sums.sum), of_rounded = sum_over_halves(sums.rounded[0]);
  v16f* const o = sums.o;
  // Waves that took different positions of the same rows add up in pairs, through LDS.
  float4* const s_stats = reinterpret_cast<float4*>(t2);
  for (int n = key_waves / 2; n >= 1; n /= 2) {
    __syncthreads();
    const int to = wave & (width * n - 1);
    float* const s_o = reinterpret_cast<float*>(to == 0 ? t0 : t1);
    if (key_wave >= n && key_wave < 2 * n) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<float4*>(s_o + ((i * 4 + r / 4) * 64 + lane) * 4) =
              make_float4(o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]);
      if (half == 0) s_stats[to * 32 + col] = make_float4(ref, total, of_rounded, 0.0f);
    }
    __syncthreads();
    if (key_wave < n) {
      const float4 st = s_stats[wave * 32 + col];
      const float up = fmaxf(ref, st.x);
      const float f = ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ref - up);
      const float h = st.x == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(st.x - up);
      ref = up;
      total = total * f + st.y * h;
      of_rounded = of_rounded * f + st.z * h;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 x = *reinterpret_cast<const float4*>(s_o + ((i * 4 + r / 4) * 64 + lane) * 4);
          o[i][r] = o[i][r] * f + x.x * h;
          o[i][r + 1] = o[i][r + 1] * f + x.y * h;
          o[i][r + 2] = o[i][r + 2] * f + x.z * h;
          o[i][r + 3] = o[i][r + 3] * f + x.w * h;
        }
    }
  }
  if (key_wave > 0 || row >= pc.rows) return;
  if (pc.parts > 1) {
    const int64_t to = int64_t(pc.slot) * kTileRows + slot_row;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(a.sums + to * D + 32 * i + 2 * r + 4 * half) =
            make_float4(o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]);
    if (half == 0) a.stats[to] = make_float4(ref, total, of_rounded, 0.0f);
    return;
  }
  const int64_t q_row = pc.q0 + my_query;
  if (a.lse && half == 0)
    a.lse[q_row * a.hq + my_head] = total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
  const float inv = total == 0.0f ? 0.0f : a.v_scale / of_rounded;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<uint2*>(a.out + q_row * a.os + int64_t(my_head) * D + 32 * i + 2 * r + 4 * half) =
          make_uint2(cvt_bf16x2(o[i][r] * inv, o[i][r + 1] * inv),
                     cvt_bf16x2(o[i][r + 2] * inv, o[i][r + 3] * inv));
  }
}

// Adds up the parts of a piece in order.  The workgroups of each part take a share of its rows, D/4 lanes
// a row: each such group of lanes a row of its own, or, of many parts, every kGroups-th part of the
// workgroup's row.
constexpr int kJoinThreads = 256;
constexpr int kJoinGroups = 4;   // workgroups of a part (64 steps of 500 to 8100 positions: 109 us, with eight 112)
constexpr int kJoinPerCu = 8;    // workgroups on a compute unit
constexpr int kManyParts = 16;   // (4 sequences of 1 and 4 tokens, 256-wide heads: 28 us, as if few 36; two
                                 // 64-wide prompts 87, as if many 132)
template <int D>
__global__ __launch_bounds__(kJoinThreads) void chunk_join_kernel(const ChunkArgs a) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  const int used = a.parts[a.slots * a.hkv].x;
  for (int item = blockIdx.x; item < a.slots * a.hkv * kJoinGroups; item += gridDim.x) {
  const int slot = item / kJoinGroups;
  const int4 x = a.parts[slot];
  if (slot >= used) return;
  const int part = x.w & 0xFFFF, parts = x.w >> 16;
  const int rows = x.z & 0xFF, row_waves = x.z >> 8 & 0xF, heads = x.z >> 12 & 0xF, kvh = int(uint32_t(x.z) >> 16);
  const int share = part * kJoinGroups + item % kJoinGroups, shares = parts * kJoinGroups;
  const int group = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  const int64_t first = int64_t(slot - part) * kTileRows;  // a piece's parts lie side by side
  const bool many = parts > kManyParts;
  __shared__ __attribute__((aligned(16))) float4 s_v[kGroups][kLanes];
  __shared__ __attribute__((aligned(16))) float4 s_st[kGroups];
  const int step = many ? shares : shares * kGroups;
  for (int i = many ? share : share * kGroups + group; i - (many ? 0 : group) < heads * rows; i += step) {
    const bool live = i < heads * rows;
    const int h = live ? i / rows : 0, r = live ? i - h * rows : 0;
    float ref = neg_inf(), total = 0.0f, rounded = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float4 st, float4 x) {
      const float to = fmaxf(ref, st.x);
      const float f = ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ref - to);
      const float g = st.x == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(st.x - to);
      ref = to;
      total = total * f + st.y * g;
      rounded = rounded * f + st.z * g;
      v.x = v.x * f + x.x * g; v.y = v.y * f + x.y * g;
      v.z = v.z * f + x.z * g; v.w = v.w * f + x.w * g;
    };
    const int64_t at0 = first + h * row_waves * kWaveRows + r;
    if (live) {
      const int by = many ? kGroups : 1;
      for (int p = many ? group : 0; p < parts; p += 4 * by) {
        float4 y[4], st[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t at = at0 + int64_t(min(p + k * by, parts - 1)) * kTileRows;
          y[k] = *reinterpret_cast<const float4*>(a.sums + at * D + d);
          st[k] = a.stats[at];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (p + k * by < parts) add(st[k], y[k]);
      }
    }
    if (many) {
      s_v[group][threadIdx.x % kLanes] = v;
      if (d == 0) s_st[group] = make_float4(ref, total, rounded, 0.0f);
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < kGroups; ++g) add(s_st[g], s_v[g][threadIdx.x]);
      __syncthreads();
      if (group > 0) continue;
    }
    if (!live) continue;
    const int q = int(a.by_group.div(x.y + r)), head = (kvh + h) * a.group + x.y + r - q * a.group;
    const int64_t q_row = x.x + q;
    const float inv = total == 0.0f ? 0.0f : a.v_scale / rounded;
    *reinterpret_cast<uint2*>(a.out + q_row * a.os + int64_t(head) * D + d) =
        make_uint2(cvt_bf16x2(v.x * inv, v.y * inv), cvt_bf16x2(v.z * inv, v.w * inv));
    if (a.lse && d == 0)
      a.lse[q_row * a.hq + head] = total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
  }
  }
}

int chunk_shape(int32_t seqs, int32_t tq, int32_t hq, int32_t hkv, int32_t d) {
  if (seqs < 0 || seqs > kMostSeqs || tq < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || hq > 65536)
    return FP8Q_EINVAL;
  if (int64_t(tq) * hq > (int64_t(1) << 30)) return FP8Q_EINVAL;
  if (d != 64 && d != 128 && d != 256) return FP8Q_EINVAL;
  return FP8Q_OK;
}

struct ChunkPlan {
  int slots;       // pieces of a KV head when sequences are split; 0: they are not
  float resident;  // pieces of a KV head that run at once
  int64_t whole;   // pieces that a KV head may have, when sequences are not split
  int64_t pieces;  // and when they are
  uint64_t sums_bytes, stats_bytes, bytes;
};
// KV heads that a piece of few rows takes at most.
int most_heads(int32_t hkv) { return hkv % 4 == 0 ? 4 : hkv % 2 == 0 ? 2 : 1; }

ChunkPlan chunk_plan(int32_t seqs, int32_t tq, int32_t hq, int32_t hkv, int32_t d) {
  ChunkPlan p = {};
  const int64_t rows = int64_t(tq) * (hq / hkv);
  const int64_t some = seqs < tq ? seqs : tq;  // sequences that have a query
  // Pieces of r rows for a KV head: (r + 127) / 128 at most, and 1 / heads + r (2 - 1 / heads) / 129 at most where
  // few rows share a piece with other heads (equal at 129 rows); lists that are dealt to: one more each.
  // Workgroups that find nothing read all lengths for it: by the first bound alone 1024 steps of 100 to 1700
  // positions take 420 us instead of 367, 8192 of 1 to 64 positions 7.3 ms instead of 1.7.
  const int64_t heads = most_heads(hkv);
  p.whole = (rows + some * (kTileRows - 1)) / kTileRows + 2;
  const int64_t shared = (some + (2 * heads - 1) * rows / (kTileRows + 1)) / heads + 4;
  if (heads > 1 && shared < p.whole) p.whole = shared;
  p.resident = float(num_cus() * (d == 256 ? 1 : d == 128 ? 2 : 3)) / float(hkv);
  // (room for the pieces that run at once: 64-wide prompts 105 us instead of 87; for three times as many:
  // 1 x 5 tokens 16.9 -> 17.8, the more workgroups that find nothing to do)
  const int slots = int(1.75f * p.resident);
  // With whole tiles for all slots nothing is split, uneven batches neither: a prompt of 4096 tokens beside one step
  // over 100000 positions, 32/8 heads x 128, takes 3.3 ms (the step's one workgroup for four KV heads), the prompt
  // alone 156 us and the step alone 50; a prompt of 3000 tokens, which leaves slots, and that step 154 us.
  if (seqs <= kSplitSeqs && slots > 3 && rows / kTileRows < slots) p.slots = slots;
  p.pieces = p.slots > p.whole ? p.slots : p.whole;
  if (p.slots == 0) return p;
  const uint64_t all = uint64_t(p.slots) * hkv * kTileRows;
  p.sums_bytes = all * d * 4;
  p.stats_bytes = all * 16;
  p.bytes = p.sums_bytes + p.stats_bytes + (uint64_t(p.slots) * hkv + 1) * 16;
  return p;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int fp8_attn_chunk_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             uint64_t* bytes) {
  if (!bytes) return FP8Q_ENULL;
  *bytes = 0;
  const int rc = chunk_shape(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
  if (num_seqs > 0 && total_q > 0)
    *bytes = chunk_plan(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim).bytes;
  return FP8Q_OK;
}

extern "C" int fp8_attn_chunk(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                              const int32_t* block_tables, const int32_t* context_lens,
                              const int32_t* cu_seqlens_q, uint16_t* out, float* lse,
                              int32_t num_seqs, int32_t total_q, int32_t max_blocks,
                              int64_t table_stride, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              float k_scale, float v_scale, float softmax_scale, int32_t causal,
                              int64_t q_stride, int64_t out_stride, int64_t cache_stride,
                              void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  const int rc = chunk_shape(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim);
  if (rc != FP8Q_OK) return rc;
  if (max_blocks < 0 || block_size <= 0 || num_blocks <= 0 || table_stride < max_blocks)
    return FP8Q_EINVAL;
  if (int64_t(max_blocks) * block_size > (int64_t(1) << 30)) return FP8Q_EINVAL;
  const int64_t eq = int64_t(num_q_heads) * head_dim, ek = int64_t(num_kv_heads) * head_dim;
  if (q_stride < eq || out_stride < eq || q_stride > (int64_t(1) << 30) ||
      out_stride > (int64_t(1) << 30) || table_stride > (int64_t(1) << 40))
    return FP8Q_EINVAL;
  if (cache_stride < int64_t(block_size) * ek || num_blocks > (int64_t(1) << 62) / cache_stride ||
      cache_stride >= (int64_t(1) << 32))
    return FP8Q_EINVAL;
  if (!(k_scale >= 0x1p-64f && k_scale <= 0x1p64f) || !(v_scale >= 0x1p-64f && v_scale <= 0x1p64f) ||
      !(softmax_scale > 0.0f && softmax_scale <= 0x1p32f))
    return FP8Q_EINVAL;
  if (num_seqs == 0 || total_q == 0) return FP8Q_OK;
  if (!q || !k_cache || !v_cache || !out || !context_lens || !cu_seqlens_q ||
      (max_blocks > 0 && !block_tables))
    return FP8Q_ENULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(lse, 4) || q_stride % 8 || out_stride % 8 || cache_stride % 16)
    return FP8Q_EALIGN;
  const ChunkPlan p = chunk_plan(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim);
  if (p.bytes > 0) {
    if (!workspace) return FP8Q_ENULL;
    if (!aligned(workspace, 256)) return FP8Q_EALIGN;
    if (workspace_bytes < p.bytes) return FP8Q_EINVAL;
  }
  const bool cut = p.slots > 0 && int64_t(max_blocks) * block_size > kShort;
  ChunkArgs a = {};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.tables = block_tables, a.lens = context_lens;
  a.cu = cu_seqlens_q, a.out = out, a.lse = lse;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  if (cut) {
    a.sums = reinterpret_cast<float*>(ws);
    a.stats = reinterpret_cast<float4*>(ws + p.sums_bytes);
    a.parts = reinterpret_cast<int4*>(ws + p.sums_bytes + p.stats_bytes);
  }
  a.ts = table_stride, a.qs = q_stride, a.os = out_stride, a.cs = cache_stride, a.nblocks = num_blocks;
  a.seqs = num_seqs, a.width = max_blocks, a.tq = total_q, a.hq = num_q_heads, a.hkv = num_kv_heads;
  a.group = num_q_heads / num_kv_heads, a.bs = block_size, a.causal = causal != 0;
  a.by_group = FastDiv(uint32_t(a.group)), a.by_block = FastDiv(uint32_t(block_size));
  a.most_heads = most_heads(num_kv_heads);
  a.slots = cut ? p.slots : 0, a.resident = p.resident, a.v_scale = v_scale;
  // Masked scores are -infinity before they are scaled, and a scale of 0 would make them NaN: where the product
  // leaves binary32 it is its smallest number, which takes the largest score below 2^-21, the weight 1.
  a.scale_log2 = fmaxf(softmax_scale * k_scale * kLog2e, 0x1p-149f);
  const int64_t per = num_kv_heads % 8 == 0 ? 8 : 8 % num_kv_heads == 0 ? 8 / num_kv_heads : 1;
  const int64_t pieces = cut ? p.pieces : p.whole;
  const int64_t blocks = num_kv_heads % 8 == 0 ? pieces * num_kv_heads
                                               : (pieces + per - 1) / per * per * num_kv_heads;
  if (blocks > 0x7FFFFFFF) return FP8Q_EINVAL;
  auto kern = head_dim == 64 ? chunk_kernel<64> : head_dim == 128 ? chunk_kernel<128> : chunk_kernel<256>;
  launch(kern, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a);
  if (launch_status() != FP8Q_OK || !cut) return launch_status();
  auto join = head_dim == 64 ? chunk_join_kernel<64>
              : head_dim == 128 ? chunk_join_kernel<128> : chunk_join_kernel<256>;
  const int joins = p.slots * num_kv_heads * kJoinGroups, most = kJoinPerCu * num_cus();
  launch(join, dim3(unsigned(joins < most ? joins : most)), dim3(kJoinThreads), 0, stream, a);
  return launch_status();
}
