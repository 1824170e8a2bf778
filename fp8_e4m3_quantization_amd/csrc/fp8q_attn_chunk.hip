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
  static constexpr int kLanes = D / 16;              // lanes that fetch a row of codes
  static constexpr int kRowsAtOnce = 64 / kLanes;    // rows that a wave's copy of 1 KB holds
  const ChunkArgs& a;
  Piece pc;
  int kvh;
  const int32_t* table;
  bool any_bad;    // some position of the piece lies in a block that does not exist

  // The id of a position's block (behind the last position: the last one's).
  __device__ __forceinline__ int block_at(int pos) const {
    return table[a.by_block.div(min(pos, pc.len - 1))];
  }
  // Where a position's row of this KV head lies in the pools.  A block that does not exist is
  // replaced by the first one: what is read there does not count.
  __device__ __forceinline__ int64_t row_at(int pos, int id) const {
    pos = min(pos, pc.len - 1);
    const int off = pos - int(a.by_block.div(pos)) * a.bs;
    const bool good = uint32_t(id) < a.nblocks;
    return (good ? id : 0) * a.cs + off * (int64_t(a.hkv) * D) + int64_t(kvh) * D;
  }
  // A copy of 16 bytes a lane into 1 KB of LDS.
  static __device__ __forceinline__ void copy(const uint8_t* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void*)to, 16, 0, 0);
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
      const uint8_t* v = a.vc + row_at(pos, id) + 4 * half;
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

// NaN codes of w become 0; `odd` is not 0 where there were any.
__device__ __forceinline__ uint32_t without_nans(uint32_t w, uint32_t* odd) {
  const uint32_t nan = e4m3_nan_bytes(w);
  *odd |= nan;
  return w & ~((nan >> 7) * 0xFFu);
}

__device__ __forceinline__ v8bf e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(v8bf, v4u{e4m3x2_to_bf16<false>(lo), e4m3x2_to_bf16<true>(lo),
                                      e4m3x2_to_bf16<false>(hi), e4m3x2_to_bf16<true>(hi)});
}

template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 128 ? 2 : 3) void chunk_kernel(const ChunkArgs a) {
  // Two tiles each of keys and values in bf16, and one each of codes on their way there
  __shared__ __attribute__((aligned(16))) uint16_t k0[kTileKeys * D], k1[kTileKeys * D];
  __shared__ __attribute__((aligned(16))) uint16_t v0[kTileKeys * D], v1[kTileKeys * D];
  __shared__ __attribute__((aligned(16))) uint8_t rk[kTileKeys * D], rv[kTileKeys * D];
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
    int* const flags = reinterpret_cast<int*>(k1);
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

  // Queries, in the order in which a form reads keys: 16 values a step of two halves, or 32 a pair
  // of steps.
  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(pc.q0 + my_query) * a.qs + int64_t(my_head) * D;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const int at = few ? 32 * (s >> 1) + 16 * half + 8 * (s & 1) : 16 * s + 8 * half;
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + at));
    }
  }
  {
    bool bad = false;
    const int first = a.by_block.div(pc.from * kTileKeys), last = pc.from < pc.to ? a.by_block.div(min(pc.to * kTileKeys, pc.len) - 1) : first - 1;
    for (int i = first + tid; i <= last; i += kThreads) bad |= uint32_t(wk.table[i]) >= a.nblocks;
    wk.any_bad = any_of_all(bad);
  }

  RowSums<D> sums;
  sums.clear();
  const float scale = a.scale_log2;
  uint32_t odd = 0;  // not 0: NaN codes of values were left out of tiles that not all rows see

  if (few) {
    // Each wave takes every key_waves-th block of 32 positions: codes go to LDS, one block ahead, and
    // are widened when they are read.
    constexpr int kCopies = D / 32;                        // copies of a block's keys, or values
    const int f_row = lane / Work<D>::kLanes, f_place = lane % Work<D>::kLanes;
    // order of the 16-byte chunks within a row: keys are read eight rows at a time, values rows
    // 0..3 and 8..11 of 16 (or the others)
    auto k_turn = [&](int r) { return D == 64 ? (r >> 1) & 3 : r & 7; };
    auto v_turn = [&](int r) {
      return D == 64 ? ((r >> 1) & 1) | ((r >> 2) & 2) : (r & 3) | ((r >> 1) & 4);
    };
    int ids[kCopies];
    auto fetch_ids = [&](int n) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) ids[j] = wk.block_at(32 * n + j * Work<D>::kRowsAtOnce + f_row);
    };
    auto copy_block = [&](int n, uint8_t* ks, uint8_t* vs) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int r = j * Work<D>::kRowsAtOnce + f_row;
        const int64_t at = wk.row_at(32 * n + r, ids[j]);
        Work<D>::copy(a.kc + at + (f_place ^ k_turn(r)) * 16, ks + j * 1024);
        Work<D>::copy(a.vc + at + (f_place ^ v_turn(r)) * 16, vs + j * 1024);
      }
    };
    auto block = [&](int n, const uint8_t* ks, const uint8_t* vs) {
      v16f s[1];
#pragma unroll
      for (int r = 0; r < 16; ++r) s[0][r] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(ks + col * D + ((2 * c + half) ^ k_turn(col)) * 16);
        s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(x.x, x.y), qf[2 * c], s[0], 0, 0, 0);
        s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(x.z, x.w), qf[2 * c + 1], s[0], 0, 0, 0);
      }
      const bool edge = 32 * (n + 1) > all_see || wk.any_bad;
      if (32 * (n + 1) > wave_least || wk.any_bad) wk.template mask<1>(s, 32 * n, limit);
      const float base = sums.template move_to<1>(largest_score<1>(s) * scale, s, scale);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const v8bf p = sums.weights(s[0], st, scale, base);
        const int i16 = lane & 15, side = (lane >> 4) & 1;
        const int r = 16 * st + 4 * half + ((i16 >> 1) & 3) + 8 * (i16 >> 3);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          typedef int v2i __attribute__((ext_vector_type(2)));
          typedef __attribute__((address_space(3))) v2i lds_v2i;
          v2u w = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_v2i*)(vs + r * D + ((2 * i + side) ^ v_turn(r)) * 16 + 8 * (i16 & 1))));
          if (edge) w = v2u{without_nans(w[0], &odd), without_nans(w[1], &odd)};
          sums.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3x8_to_bf16(w[0], w[1]), p, sums.o[i], 0, 0, 0);
        }
      }
    };
    uint8_t* const ks0 = reinterpret_cast<uint8_t*>(k0) + wave * 32 * D;
    uint8_t* const vs0 = reinterpret_cast<uint8_t*>(v0) + wave * 32 * D;
    uint8_t* const ks1 = reinterpret_cast<uint8_t*>(k1) + wave * 32 * D;
    uint8_t* const vs1 = reinterpret_cast<uint8_t*>(v1) + wave * 32 * D;
    const int end = min(2 * pc.to, (pc.len + 31) / 32);
    int n = 2 * pc.from + key_wave;
    if (n < end) {
      fetch_ids(n);
      copy_block(n, ks0, vs0);
      fetch_ids(n + key_waves);
      if (n + key_waves < end) copy_block(n + key_waves, ks1, vs1);
      auto turn = [&](uint8_t* ks, uint8_t* vs) {
        const bool more = n + key_waves < end;
        fetch_ids(n + 2 * key_waves);
        asm volatile("" ::: "memory");
        // the copies of this block have landed: at most those of the next one, and its ids, have not
        if (more) __builtin_amdgcn_s_waitcnt((2 * kCopies & 15) | (2 * kCopies >> 4) << 14 | 0x0F70);
        else __builtin_amdgcn_s_waitcnt(0x0F70);
        asm volatile("" ::: "memory");
        block(n, ks, vs);
        if (n + 2 * key_waves < end) {
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this block has been read
          asm volatile("" ::: "memory");
          copy_block(n + 2 * key_waves, ks, vs);
        }
        n += key_waves;
        return more;
      };
      while (turn(ks0, vs0) && turn(ks1, vs1)) {}
    }
  } else {
    // All waves go over all positions, 64 at a time.
    constexpr int kCopies = D / 64;                        // 1 KB copies of a wave and tile
    const int f_row = lane / Work<D>::kLanes, f_place = lane % Work<D>::kLanes;
    int ids[kCopies];          // of the keys' next tile
    int64_t at[kCopies];       // rows of the values' next tile
    int next_k = pc.from, next_ids = pc.from;              // tiles
    auto fetch_ids = [&]() {
#pragma unroll
      for (int j = 0; j < kCopies; ++j)
        ids[j] = wk.block_at(next_ids * kTileKeys + (wave * kCopies + j) * Work<D>::kRowsAtOnce + f_row);
      ++next_ids;
    };
    // Copies of the next tile of values, whose place the keys' copies left, and of the one of keys
    // after it.
    auto copy_values = [&]() {
#pragma unroll
      for (int j = 0; j < kCopies; ++j)
        Work<D>::copy(a.vc + at[j] + f_place * 16, rv + (wave * kCopies + j) * 1024);
    };
    auto copy_keys = [&]() {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        at[j] = wk.row_at(next_k * kTileKeys + (wave * kCopies + j) * Work<D>::kRowsAtOnce + f_row, ids[j]);
        Work<D>::copy(a.kc + at[j] + f_place * 16, rk + (wave * kCopies + j) * 1024);
      }
      ++next_k;
    };
    // A wave widens the codes that it copied: eight of a row a lane.
    constexpr int kWide = 64 / (D / 8);                    // rows at a time
    const int w_row = lane / (D / 8), w_chunk = lane % (D / 8);
    auto widen = [&](const uint8_t* codes, uint16_t* to, auto chunk_of, bool clean) {
#pragma unroll
      for (int j = 0; j < 2 * kCopies; ++j) {
        const int r = wave * kCopies * Work<D>::kRowsAtOnce + j * kWide + w_row;
        uint2 x = *reinterpret_cast<const uint2*>(codes + r * D + w_chunk * 8);
        if (clean) x = make_uint2(without_nans(x.x, &odd), without_nans(x.y, &odd));
        *reinterpret_cast<v8bf*>(to + r * D + chunk_of(r, w_chunk) * 8) = e4m3x8_to_bf16(x.x, x.y);
      }
    };
    auto widen_keys = [&](uint16_t* to) { widen(rk, to, [](int r, int c) { return k_chunk<D>(r, c); }, false); };
    auto widen_values = [&](uint16_t* to, bool clean) {
      widen(rv, to, [](int r, int c) { return v_chunk<D>(r, c); }, clean);
    };
    const int tiles = pc.to - pc.from;
    const int whole = wk.any_bad ? 0 : all_see / kTileKeys - pc.from;   // tiles that all rows see
    auto landed = [&]() {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's copies
      asm volatile("" ::: "memory");
    };
    float base = 0.0f;
    auto scores = [&](int t, v16f* s, const uint16_t* kt) {
      tile_scores<D>(s, kt, qf);
      const int p0 = (pc.from + t) * kTileKeys;
      if (p0 + kTileKeys > wave_least || wk.any_bad) wk.template mask<2>(s, p0, limit);
      base = sums.template move_to<2>(largest_score<2>(s) * scale, s, scale);
    };
    // At the barrier of tile t of the piece the other waves' codes are wide, and the places of the
    // keys of tile t and of the values before them are free: this wave widens its codes of the keys of
    // tile t + 2 and of the values of t + 1, and starts the copies of the next ones.
    auto next_tile = [&](uint16_t* k_free, uint16_t* v_free, bool clean) {
      landed();
      __syncthreads();
      widen_keys(k_free);
      widen_values(v_free, clean);
      asm volatile("" ::: "memory");
      copy_values();
      copy_keys();
      fetch_ids();
    };
    // Tile t, whose scores are s, while the whole tiles last: the scores of t + 1 (matrix cores) beside
    // the weights of t (vector ALUs), then the values of t beside the largest of the new scores.
    auto turn = [&](const v16f* s, v16f* next, const uint16_t* kn, const uint16_t* vt,
                    uint16_t* k_free, uint16_t* v_free) {
      next_tile(k_free, v_free, false);
      tile_scores<D>(next, kn, qf);
      v8bf p[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) p[st] = sums.weights(s[st >> 1], st & 1, scale, base);
#pragma unroll
      for (int st = 0; st < 4; ++st) sums.add_values(vt, st, p[st]);
      base = sums.template move_to<2>(largest_score<2>(next) * scale, next, scale);
    };
    if (tiles > 0) {
      v16f sa[2];
      fetch_ids();
      copy_keys();           // keys of tile 0
      fetch_ids();
      copy_values();         // values of tile 0
      landed();
      widen_keys(k0);
      widen_values(v0, 0 >= whole);
      asm volatile("" ::: "memory");
      copy_keys();           // keys of tile 1 (behind the last one: of the last position again)
      fetch_ids();
      landed();
      widen_keys(k1);
      asm volatile("" ::: "memory");
      copy_values();         // values of tile 1
      copy_keys();           // keys of tile 2
      fetch_ids();
      __syncthreads();
      scores(0, sa, k0);
      int t = 0;
      for (; t + 2 < whole && t + 2 < tiles; t += 2) {
        v16f sb[2];
        turn(sa, sb, k1, v0, k0, v1);
        turn(sb, sa, k0, v1, k1, v0);
      }
      for (; t < tiles; ++t) {  // the last tiles, among them those that are seen in part
        const uint16_t *kn = t & 1 ? k0 : k1, *vt = t & 1 ? v1 : v0;
        next_tile(t & 1 ? k1 : k0, t & 1 ? v0 : v1, t + 1 >= whole);
#pragma unroll
        for (int st = 0; st < 4; ++st) sums.add_values(vt, st, sums.weights(sa[st >> 1], st & 1, scale, base));
        __builtin_amdgcn_sched_barrier(0);
        if (t + 1 < tiles) scores(t + 1, sa, kn);
      }
    }
  }

  // NaN codes that were left out reach the rows that see them.
  __syncthreads();
  if (any_of_all(odd != 0) && key_wave == 0) {
    const int first = wk.any_bad ? pc.from : max(pc.from, all_see / kTileKeys);
    wk.take_nans(sums, first * kTileKeys, limit);
  }

  float ref = sums.ref, total = sum_over_halves(sums.sum), of_rounded = sum_over_halves(sums.rounded[0]);
  v16f* const o = sums.o;
  // Waves that took different positions of the same rows add up in pairs, through LDS.
  float4* const s_stats = reinterpret_cast<float4*>(rk);
  for (int n = key_waves / 2; n >= 1; n /= 2) {
    __syncthreads();
    const int to = wave & (row_waves * n - 1);
    float* const s_o = reinterpret_cast<float*>(to == 0 ? k0 : k1);
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
  if (cache_stride < int64_t(block_size) * ek || num_blocks > (int64_t(1) << 62) / cache_stride)
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
