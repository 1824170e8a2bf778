// fp8q_attn_chunk.hip -- attention of chunks of new tokens over the paged E4M3 KV cache: packed
// bf16 queries of sequences with one new token or thousands, grouped heads, causal from the end.
//
// Mathematics, query i of a sequence of Lq new tokens and len cached positions (the new tokens'
// own among them), over the positions j that it sees (all of them, or causal j <= i + len - Lq):
//   s_j = softmax_scale * k_scale * q . K_j
//   out = v_scale * sum_j exp(s_j - r) V_j / sum_j exp(s_j - r),  lse = r + log sum_j exp(s_j - r)
// for any reference r.  A query that sees no position gets zeros and lse = -infinity.
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
constexpr int kSplitSeqs = 256;  // batches of more sequences are not split along the positions
constexpr int kMinPart = 4;      // tiles of positions of a part, at least
constexpr int kFewRows = 64;     // tiles of so many rows at most divide positions among the waves
constexpr float kFewCost = 0.6f; // time of their tile of positions, of another's

struct ChunkArgs {
  const uint16_t* q;
  const uint8_t *kc, *vc;
  const int32_t *tables, *lens, *cu;
  uint16_t* out;
  float* lse;     // [tq, hq] or NULL
  float* sums;    // [hkv][slots][kTileRows][D]: sums of weighted values of parts
  float4* stats;  // [hkv][slots][kTileRows]: reference (log2 units), sums of the weights and of the
                  // rounded ones
  int4* pieces;   // [hkv][slots]: first query row, first row, rows, part | parts << 16
  int64_t ts, qs, os, cs, nblocks;
  FastDiv by_group, by_block;
  int seqs, width, tq, hq, hkv, group, bs, causal;
  int slots;      // pieces of a KV head when sequences are split; 0: they are not
  float scale_log2, v_scale;
};

// A piece of work: a tile of rows of one sequence and KV head, and the steps that it goes over.
struct Piece {
  int seq, q0, lq, len;  // the sequence's first query row, queries and positions
  int row0, rows;        // the tile's first row of the sequence's, and how many
  int part, parts, from, to;  // tiles of positions [from, to)
  // positions [0, seen(i)) are seen by query i
  __device__ __forceinline__ int seen(const ChunkArgs& a, int i) const {
    return a.causal ? min(max(i + len - lq + 1, 0), len) : len;
  }
};

// Sequence s: its first query row, queries and positions, whatever the lists hold.
__device__ __forceinline__ void seq_of(const ChunkArgs& a, int s, int* q0, int* lq, int* len) {
  const int from = min(max(a.cu[s], 0), a.tq);
  *q0 = from;
  *lq = min(max(a.cu[s + 1], from), a.tq) - from;
  *len = min(max(a.lens[s], 0), a.width * a.bs);
}

__device__ __forceinline__ int tiles_of(const ChunkArgs& a, int lq) {
  return (lq * a.group + kTileRows - 1) / kTileRows;
}
__device__ __forceinline__ int key_tiles(int positions) { return (positions + kTileKeys - 1) / kTileKeys; }

// Parts of a sequence of `steps` tiles of positions when a piece takes at most about `most` (in time
// of a tile of many rows).  The same arithmetic in every workgroup: all agree.
__device__ __forceinline__ int parts_of(const ChunkArgs& a, int lq, int steps, float most) {
  const float cost = float(steps) * (lq * a.group <= kFewRows ? kFewCost : 1.0f);
  const int n = int(__builtin_ceilf(cost * __builtin_amdgcn_rcpf(most)));
  return max(min(n, steps / kMinPart), 1);
}

__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_prefix(v), 63); }

// Piece `u` of a KV head's, or false.  Where all sequences' tiles together are fewer than the
// slots, each sequence's positions are cut into parts: as few as a limit on the steps of a piece
// makes, the smallest limit whose pieces the slots hold.
__device__ __forceinline__ bool find_piece(const ChunkArgs& a, int u, Piece* pc) {
  const int lane = threadIdx.x & 63;
  int tile = 0, tiles = 0, parts = 1, part = 0;
  if (a.seqs > kSplitSeqs) {
    bool found = false;
    for (int s0 = 0; s0 < a.seqs && !found; s0 += 64) {
      int q0 = 0, lq = 0, len = 0;
      if (s0 + lane < a.seqs) seq_of(a, s0 + lane, &q0, &lq, &len);
      const int n = tiles_of(a, lq), upto = wave_prefix(n), all = __builtin_amdgcn_readlane(upto, 63);
      if (u < all) {
        const int j = __builtin_ctzll(__ballot(upto > u));
        pc->seq = s0 + j;
        pc->q0 = __builtin_amdgcn_readlane(q0, j);
        pc->lq = __builtin_amdgcn_readlane(lq, j);
        pc->len = __builtin_amdgcn_readlane(len, j);
        tiles = __builtin_amdgcn_readlane(n, j);
        u -= __builtin_amdgcn_readlane(upto, j) - tiles;
        found = true;
      } else {
        u -= all;
      }
    }
    if (!found) return false;
    tile = tiles - 1 - u;
  } else {
    constexpr int kSets = kSplitSeqs / 64;
    int q0[kSets] = {}, lq[kSets] = {}, len[kSets] = {}, n[kSets] = {}, steps[kSets] = {};
    int all = 0, longest = 0;
#pragma unroll
    for (int c = 0; c < kSets; ++c) {
      if (c * 64 >= a.seqs) continue;
      if (c * 64 + lane < a.seqs) seq_of(a, c * 64 + lane, &q0[c], &lq[c], &len[c]);
      n[c] = tiles_of(a, lq[c]);
      steps[c] = lq[c] > 0 ? key_tiles(len[c]) : 0;
      all += wave_sum(n[c]);
      longest = max(longest, int(max_over_wave(float(steps[c]))));
    }
    float most = 1e9f;
    if (all < a.slots && longest > kMinPart) {
      auto pieces = [&](float limit) {
        int sum = 0;
#pragma unroll
        for (int c = 0; c < kSets; ++c)
          if (c * 64 < a.seqs) sum += n[c] * parts_of(a, lq[c], steps[c], limit);
        return wave_sum(sum);
      };
      // (one part each at the upper end, however the reciprocal is rounded)
      float lo = 1.0f, hi = 2.0f * float(longest);
      if (pieces(lo) <= a.slots) {
        hi = lo;
      } else {
        for (int i = 0; i < 12; ++i) {
          const float mid = 0.5f * (lo + hi);
          if (pieces(mid) <= a.slots) hi = mid; else lo = mid;
        }
      }
      most = hi;
    }
    bool found = false;
#pragma unroll
    for (int c = 0; c < kSets; ++c) {
      if (found || c * 64 >= a.seqs) continue;
      const int per = parts_of(a, lq[c], steps[c], most), upto = wave_prefix(n[c] * per);
      const int here = __builtin_amdgcn_readlane(upto, 63);
      if (u < here) {
        const int j = __builtin_ctzll(__ballot(upto > u));
        pc->seq = c * 64 + j;
        pc->q0 = __builtin_amdgcn_readlane(q0[c], j);
        pc->lq = __builtin_amdgcn_readlane(lq[c], j);
        pc->len = __builtin_amdgcn_readlane(len[c], j);
        tiles = __builtin_amdgcn_readlane(n[c], j);
        parts = __builtin_amdgcn_readlane(per, j);
        u -= __builtin_amdgcn_readlane(upto, j) - tiles * parts;
        found = true;
      } else {
        u -= here;
      }
    }
    if (!found) return false;
    tile = tiles - 1 - u / parts;
    part = u % parts;
  }
  pc->row0 = tile * kTileRows;
  pc->rows = min(pc->lq * a.group - pc->row0, kTileRows);
  const int last = int(a.by_group.div(pc->row0 + pc->rows - 1));
  const int steps = key_tiles(pc->seen(a, last));
  parts = max(min(parts, steps / kMinPart), 1);  // an early tile of a prompt sees less
  if (part >= parts) return false;
  pc->part = part;
  pc->parts = parts;
  pc->from = int(int64_t(steps) * part / parts);
  pc->to = int(int64_t(steps) * (part + 1) / parts);
  return true;
}

// What the kernel's two forms share: a piece, and the lane's place in it.
template <int D>
struct Work {
  const ChunkArgs& a;
  Piece pc;
  int kvh;
  const int32_t* table;
  bool any_bad;    // some position of the piece lies in a block that does not exist

  // The id of a position's block (behind the last position: the last one's).
  __device__ __forceinline__ int block_at(int pos) const {
    return table[a.by_block.div(min(pos, pc.len - 1))];
  }
  // Scores of positions that a row does not see, or that lie in blocks that do not exist, are
  // -infinity; s holds positions p0 .. p0 + 32 kBlocks - 1.
  template <int kBlocks>
  __device__ __forceinline__ void mask(v16f* s, int p0, int limit) const {
    const int half = (threadIdx.x & 63) >> 5, left = limit - p0 - 4 * half;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = 32 * b + 8 * (r >> 2) + (r & 3) < left ? s[b][r] : neg_inf();
        if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few conditions alive at a time
      }
    if (any_bad) {  // rare
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[b][r] = uint32_t(block_at(p0 + 32 * b + 8 * (r >> 2) + (r & 3) + 4 * half)) < a.nblocks ? s[b][r] : neg_inf();
    }
  }
  // NaN codes that were left out of positions from `first` on reach a row that sees them.
  __device__ __forceinline__ void take_nans(RowSums<D>& sums, int first, int limit) const {
    const int half = (threadIdx.x & 63) >> 5, end = min(limit, min(pc.to * kTileKeys, pc.len));
    for (int pos = first; pos < end; ++pos) {
      const int id = block_at(pos);
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
  // A block that does not exist is replaced by the first one: what is read there does not count.
  __device__ __forceinline__ int64_t place(const ChunkArgs& a, int j) const {
    const uint32_t good = uint32_t(id[j]) < a.nblocks ? id[j] : 0;
    return int64_t(uint64_t(good) * uint32_t(a.cs) + uint64_t(uint32_t(at[j])) * uint32_t(a.hkv * D));
  }
};

// A copy of 16 bytes a lane into 1 KB of LDS.
__device__ __forceinline__ void copy16(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 16, 0, 0);
}

// s_waitcnt's operand for vmcnt(n).
constexpr int until_vmcnt(int n) { return (n & 15) | (n >> 4) << 14 | 0x0F70; }

// The order of a turn: the score products with the weights and the widening of the keys between them,
// then the value products with the widening of the values.
template <int D>
__device__ __forceinline__ void pair_up() {
  constexpr int kMfma = 0x008, kVector = 0x002, kLdsRead = 0x100;
  __builtin_amdgcn_sched_group_barrier(kLdsRead, 4, 0);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kVector, 10, 0);
    __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kVector, 8, 0);
  }
}

template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 128 ? 2 : 3) void chunk_kernel(const ChunkArgs a) {
  // Four tiles of codes, keys then values
  constexpr int kTileBytes = kTileKeys * D;
  __shared__ __attribute__((aligned(16))) uint8_t t0[2 * kTileBytes], t1[2 * kTileBytes];
  __shared__ __attribute__((aligned(16))) uint8_t t2[2 * kTileBytes], t3[2 * kTileBytes];
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
  // Whether `x` holds in any lane of any wave; LDS is free before and after.
  auto any_of_all = [&](bool x) {
    int* const flags = reinterpret_cast<int*>(t3);
    const bool mine_any = __any(x);
    if (lane == 0) flags[wave] = mine_any;
    __syncthreads();
    const int all = flags[0] | flags[1] | flags[2] | flags[3];
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(all) != 0;
  };
  Piece pc;
  const bool any = find_piece(a, u, &pc);
  const int64_t slot = int64_t(kvh) * a.slots + u;
  if (u < a.slots && tid == 0)
    a.pieces[slot] = any ? make_int4(pc.q0, pc.row0, pc.rows, pc.part | pc.parts << 16)
                         : make_int4(0, 0, 0, 0);
  if (!any) return;

  Work<D> wk{a, pc, kvh, a.tables + pc.seq * a.ts, false};
  // Few rows: the waves take different positions instead of different rows.
  const bool few = pc.rows <= kFewRows;
  const int row_waves = !few ? 4 : pc.rows > 32 ? 2 : 1, key_waves = 4 / row_waves;
  const int mine = (wave & (row_waves - 1)) * kWaveRows;   // this wave's first row of the tile
  const int key_wave = wave / row_waves;
  const int row = mine + col;                              // this lane's
  auto query_of = [&](int r) { return int(a.by_group.div(pc.row0 + r)); };
  const int my_row = min(row, pc.rows - 1), my_query = query_of(my_row);
  const int my_head = kvh * a.group + pc.row0 + my_row - my_query * a.group;
  const int limit = row < pc.rows ? pc.seen(a, my_query) : 0;
  // positions that all rows of the wave see, and that all rows of the tile see
  const int wave_least = __builtin_amdgcn_readfirstlane(mine + kWaveRows <= pc.rows ? pc.seen(a, query_of(mine)) : 0);
  const int all_see = __builtin_amdgcn_readfirstlane(pc.seen(a, query_of(0)));

  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(pc.q0 + my_query) * a.qs + int64_t(my_head) * D + 16 * half;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 32 * (s >> 1) + 8 * (s & 1)));
  }
  const int last_block = int(a.by_block.div(max(pc.len - 1, 0)));
  {
    bool bad = false;
    const int first = a.by_block.div(pc.from * kTileKeys);
    const int last = pc.from < pc.to ? int(a.by_block.div(min(pc.to * kTileKeys, pc.len) - 1)) : first - 1;
    for (int i = first + tid; i <= last; i += kThreads) bad |= uint32_t(wk.table[i]) >= a.nblocks;
    wk.any_bad = any_of_all(bad);
  }

  RowSums<D> sums;
  sums.clear();
  const float scale = a.scale_log2;
  uint32_t odd = 0;  // not 0: NaN codes of values were left out, at positions from first_left_out on
  int first_left_out = pc.from * kTileKeys;
  const uint8_t* const kc = a.kc + int64_t(kvh) * D;
  const uint8_t* const vc = a.vc + int64_t(kvh) * D;

  if (few) {
    // Each wave takes every key_waves-th block of 32 positions, two blocks ahead in LDS.
    const int lane = own_lane();
    constexpr int kCopies = D / 32;                        // copies of a block's keys, or values
    typedef Rows<D, kCopies> R;
    const int f_row = lane / R::kLanes, f_place = lane % R::kLanes;
    const int end = min(2 * pc.to, (pc.len + 31) / 32);
    int n = 2 * pc.from + key_wave;
    R rows;
    // Copies of the next block, after the block numbers of the one behind it: what waits for those
    // need not wait for the copies.
    auto copy_block = [&](uint8_t* ks, uint8_t* vs) {
      int64_t at[kCopies];
#pragma unroll
      for (int j = 0; j < kCopies; ++j) at[j] = rows.place(a, j);
      rows.read_ids(a, wk.table, last_block);
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int r = j * R::kAtOnce + f_row;
        copy16(kc + at[j] + (f_place ^ key_turn<D>(r)) * 16, ks + j * 1024);
        copy16(vc + at[j] + (f_place ^ value_turn<D>(r)) * 16, vs + j * 1024);
      }
    };
    // Block n; with kEdge it may be seen in part.
    auto block = [&](const uint8_t* ks, const uint8_t* vs, auto edge, int lane) {
      constexpr bool kEdge = decltype(edge)::value;
      v16f s[1];
      code_scores<D, 1>(s, ks, qf, lane);
      if (kEdge) wk.template mask<1>(s, 32 * n, limit);
      const float base = sums.template move_to<1>(largest_score<1>(s) * scale, s, scale);
#pragma unroll
      for (int st = 0; st < 2; ++st)
        sums.template add_values<kEdge>(vs, st, sums.weights(s[0], st, scale, base), &odd, lane);
    };
    // Waits for block n, takes it, and copies the one after the next into its place.
    auto turn = [&](uint8_t* ks, uint8_t* vs, auto edge, int lane) {
      asm volatile("" ::: "memory");
      // this block's copies have landed: at most the next one's have not
      if (n + key_waves < end) __builtin_amdgcn_s_waitcnt(until_vmcnt(2 * kCopies));
      else __builtin_amdgcn_s_waitcnt(until_vmcnt(0));
      asm volatile("" ::: "memory");
      block(ks, vs, edge, lane);
      if (n + 2 * key_waves < end) {
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this block has been read
        asm volatile("" ::: "memory");
        copy_block(ks, vs);
      }
      n += key_waves;
    };
    if (n < end) {
      const int mine32 = wave * 32 * D;
      const int whole = wk.any_bad ? 0 : min(end, all_see / 32);  // blocks that all rows see
      first_left_out = max(first_left_out, 32 * whole);
      rows.start(a, 32 * n + f_row, R::kAtOnce, 32 * key_waves);
      rows.read_ids(a, wk.table, last_block);
      copy_block(t0 + mine32, t1 + mine32);
      if (n + key_waves < end) copy_block(t2 + mine32, t3 + mine32);
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
    // All waves go over all positions, 64 at a time.
    const int lane = own_lane();
    constexpr int kCopies = D / 64;                        // 1 KB copies of a wave of a tile's keys, or values
    typedef Rows<D, kCopies> R;
    const int f_row = wave * kCopies * R::kAtOnce + lane / R::kLanes, f_place = lane % R::kLanes;
    R rows;
    rows.start(a, pc.from * kTileKeys + f_row, R::kAtOnce, kTileKeys);
    // Copies of the next tile, after the block numbers of the one behind it: what waits for those
    // need not wait for the copies.
    auto copy_next = [&](uint8_t* to) {
      int64_t at[kCopies];
#pragma unroll
      for (int j = 0; j < kCopies; ++j) at[j] = rows.place(a, j);
      rows.read_ids(a, wk.table, last_block);
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int r = f_row + j * R::kAtOnce;
        copy16(kc + at[j] + (f_place ^ key_turn<D>(r)) * 16, to + (wave * kCopies + j) * 1024);
        copy16(vc + at[j] + (f_place ^ value_turn<D>(r)) * 16, to + kTileBytes + (wave * kCopies + j) * 1024);
      }
    };
    const int tiles = pc.to - pc.from;
    const int whole = wk.any_bad ? 0 : all_see / kTileKeys - pc.from;   // tiles that all rows see
    float base = 0.0f;
    // At the barrier of tile t all waves' copies of tile t + 1 have landed (at most those of t + 2
    // have not), and the tile before t has been read by all: tile t + 3 takes its place.
    auto next_tile = [&](uint8_t* free) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(until_vmcnt(2 * kCopies));
      __syncthreads();
      copy_next(free);
    };
    auto scores = [&](int t, v16f* s, const uint8_t* kt, int lane) {
      code_scores<D, 2>(s, kt, qf, lane);
      const int p0 = (pc.from + t) * kTileKeys;
      if (p0 + kTileKeys > wave_least || wk.any_bad) wk.template mask<2>(s, p0, limit);
      base = sums.template move_to<2>(largest_score<2>(s) * scale, s, scale);
    };
    // Tile t, whose scores are s, while the whole tiles last: the scores of t + 1 (matrix cores) beside
    // the weights of t (vector ALUs), then the values of t beside the largest of the new scores.
    auto turn = [&](const v16f* s, v16f* next, const uint8_t* here, const uint8_t* then, uint8_t* free) {
      next_tile(free);
      code_scores<D, 2>(next, then, qf, lane);
      v8bf p[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) p[st] = sums.weights(s[st >> 1], st & 1, scale, base);
#pragma unroll
      for (int st = 0; st < 4; ++st) sums.template add_values<false>(here + kTileBytes, st, p[st], &odd, lane);
      const float top = largest_score<2>(next);
      if constexpr (D == 128) pair_up<D>();
      base = sums.template move_to<2>(top * scale, next, scale);
    };
    if (tiles > 0) {
      v16f sa[2];
      rows.read_ids(a, wk.table, last_block);
      copy_next(t0);
      copy_next(t1);
      copy_next(t2);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(until_vmcnt(4 * kCopies));
      __syncthreads();
      scores(0, sa, t0, lane);
      int t = 0;
      while (t + 2 < whole && t + 2 < tiles) {
        v16f sb[2];
        turn(sa, sb, t0, t1, t3);
        turn(sb, sa, t1, t2, t0);
        t += 2;
        if (!(t + 2 < whole && t + 2 < tiles)) break;
        turn(sa, sb, t2, t3, t1);
        turn(sb, sa, t3, t0, t2);
        t += 2;
      }
      first_left_out += t * kTileKeys;
      for (; t < tiles; ++t) {  // the last tiles, among them those that are seen in part
        const int lane = own_lane();
        auto slot_of = [&](int i) { return i & 2 ? i & 1 ? t3 : t2 : i & 1 ? t1 : t0; };
        next_tile(slot_of(t + 3));
#pragma unroll
        for (int st = 0; st < 4; ++st)
          sums.template add_values<true>(slot_of(t) + kTileBytes, st, sums.weights(sa[st >> 1], st & 1, scale, base), &odd, lane);
        __builtin_amdgcn_sched_barrier(0);
        if (t + 1 < tiles) scores(t + 1, sa, slot_of(t + 1), lane);
      }
      __builtin_amdgcn_s_waitcnt(until_vmcnt(0));  // copies behind the last tile: LDS is used again
    }
  }

  // NaN codes that were left out reach the rows that see them.
  __syncthreads();
  if (any_of_all(odd != 0) && key_wave == 0) wk.take_nans(sums, first_left_out, limit);

  float ref = sums.ref, total = sum_over_halves(sums.sum), of_rounded = sum_over_halves(sums.rounded[0]);
  v16f* const o = sums.o;
  // Waves that took different positions of the same rows add up in pairs, through LDS.
  float4* const s_stats = reinterpret_cast<float4*>(t2);
  for (int n = key_waves / 2; n >= 1; n /= 2) {
    __syncthreads();
    const int to = wave & (row_waves * n - 1);
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
    const int64_t to = slot * kTileRows + row;
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

// Adds up the parts of a tile in order: the workgroups of each part take a share of its rows, D/4
// lanes a row.
constexpr int kJoinThreads = 256;
constexpr int kJoinGroups = 4;  // workgroups of a part
template <int D>
__global__ __launch_bounds__(kJoinThreads) void chunk_join_kernel(const ChunkArgs a) {
  constexpr int kLanes = D / 4, kRows = kJoinThreads / kLanes;
  const int slot = blockIdx.x / kJoinGroups, kvh = slot / a.slots;
  const int4 p = a.pieces[slot];
  const int part = p.w & 0xFFFF, parts = p.w >> 16;
  if (parts <= 1) return;
  const int share = part * kJoinGroups + blockIdx.x % kJoinGroups, shares = parts * kJoinGroups;
  const int d = threadIdx.x % kLanes * 4;
  const int64_t first = int64_t(slot - part) * kTileRows;  // an item's parts lie side by side
  for (int r = p.z * share / shares + int(threadIdx.x) / kLanes; r < p.z * (share + 1) / shares; r += kRows) {
    float ref = neg_inf(), total = 0.0f, rounded = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const int64_t at = first + int64_t(i) * kTileRows + r;
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
    const int q = int(a.by_group.div(p.y + r)), head = kvh * a.group + p.y + r - q * a.group;
    const int64_t q_row = p.x + q;
    const float inv = total == 0.0f ? 0.0f : a.v_scale / rounded;
    *reinterpret_cast<uint2*>(a.out + q_row * a.os + int64_t(head) * D + d) =
        make_uint2(cvt_bf16x2(v.x * inv, v.y * inv), cvt_bf16x2(v.z * inv, v.w * inv));
    if (a.lse && d == 0)
      a.lse[q_row * a.hq + head] = total == 0.0f ? neg_inf() : (ref + __builtin_amdgcn_logf(total)) * kLn2;
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
  int64_t pieces;  // that a KV head may have
  uint64_t sums_bytes, stats_bytes, bytes;
};
ChunkPlan chunk_plan(int32_t seqs, int32_t tq, int32_t hq, int32_t hkv, int32_t d) {
  ChunkPlan p = {};
  const int64_t rows = int64_t(tq) * (hq / hkv);
  const int64_t some = seqs < tq ? seqs : tq;  // sequences that have a query
  p.pieces = (rows + some * (kTileRows - 1)) / kTileRows;
  const int at_once = num_cus() * (d == 256 ? 1 : d == 128 ? 2 : 3);
  const int slots = at_once / hkv;
  // (with whole tiles for all slots nothing is split)
  if (seqs <= kSplitSeqs && slots > 1 && rows / kTileRows < slots) p.slots = slots;
  if (p.slots > p.pieces) p.pieces = p.slots;
  const uint64_t all = uint64_t(p.slots) * hkv * kTileRows;
  p.sums_bytes = all * d * 4;
  p.stats_bytes = all * 16;
  p.bytes = p.sums_bytes + p.stats_bytes + uint64_t(p.slots) * hkv * 16;
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
  ChunkArgs a = {};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.tables = block_tables, a.lens = context_lens;
  a.cu = cu_seqlens_q, a.out = out, a.lse = lse;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  if (p.slots > 0) {
    a.sums = reinterpret_cast<float*>(ws);
    a.stats = reinterpret_cast<float4*>(ws + p.sums_bytes);
    a.pieces = reinterpret_cast<int4*>(ws + p.sums_bytes + p.stats_bytes);
  }
  a.ts = table_stride, a.qs = q_stride, a.os = out_stride, a.cs = cache_stride, a.nblocks = num_blocks;
  a.seqs = num_seqs, a.width = max_blocks, a.tq = total_q, a.hq = num_q_heads, a.hkv = num_kv_heads;
  a.group = num_q_heads / num_kv_heads, a.bs = block_size, a.causal = causal != 0;
  a.by_group = FastDiv(uint32_t(a.group)), a.by_block = FastDiv(uint32_t(block_size));
  a.slots = p.slots, a.scale_log2 = softmax_scale * k_scale * kLog2e, a.v_scale = v_scale;
  const int64_t per = num_kv_heads % 8 == 0 ? 8 : 8 % num_kv_heads == 0 ? 8 / num_kv_heads : 1;
  const int64_t blocks = num_kv_heads % 8 == 0 ? p.pieces * num_kv_heads
                                               : (p.pieces + per - 1) / per * per * num_kv_heads;
  if (blocks > 0x7FFFFFFF) return FP8Q_EINVAL;
  auto kern = head_dim == 64 ? chunk_kernel<64> : head_dim == 128 ? chunk_kernel<128> : chunk_kernel<256>;
  launch(kern, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a);
  if (launch_status() != FP8Q_OK || p.slots == 0) return launch_status();
  auto join = head_dim == 64 ? chunk_join_kernel<64>
              : head_dim == 128 ? chunk_join_kernel<128> : chunk_join_kernel<256>;
  launch(join, dim3(unsigned(p.slots * num_kv_heads * kJoinGroups)), dim3(kJoinThreads), 0, stream, a);
  return launch_status();
}
