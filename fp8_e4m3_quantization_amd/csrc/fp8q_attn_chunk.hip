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
#include "fp8q_attn.h"
#include "fp8q_launch.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kStepKeys = 128;   // positions staged at a time
constexpr int kTileRows = 128;   // rows (query, head of a KV head's group) of a workgroup
constexpr int kThreads = 256;
constexpr int kSplitSeqs = 256;  // batches of more sequences are not split along the positions
constexpr int kMinPart = 2;      // steps of a part, at least

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
  int part, parts, from, to;  // steps [from, to)
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
__device__ __forceinline__ int steps_of(int positions) { return (positions + kStepKeys - 1) / kStepKeys; }

// Parts of a sequence of `steps` steps when a piece takes about `most` steps.  The same arithmetic in
// every workgroup: all agree.
__device__ __forceinline__ int parts_of(int steps, float most) {
  const int n = int(__builtin_ceilf(float(steps) * __builtin_amdgcn_rcpf(most)));
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
      steps[c] = lq[c] > 0 ? steps_of(len[c]) : 0;
      all += wave_sum(n[c]);
      longest = max(longest, int(max_over_wave(float(steps[c]))));
    }
    float most = 1e9f;
    if (all < a.slots && longest > kMinPart) {
      auto pieces = [&](float limit) {
        int sum = 0;
#pragma unroll
        for (int c = 0; c < kSets; ++c)
          if (c * 64 < a.seqs) sum += n[c] * parts_of(steps[c], limit);
        return wave_sum(sum);
      };
      // (one part each at the upper end, however the reciprocal is rounded)
      float lo = float(kMinPart), hi = 2.0f * float(longest);
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
      const int per = parts_of(steps[c], most), upto = wave_prefix(n[c] * per);
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
  const int steps = steps_of(pc->seen(a, last));
  parts = max(min(parts, steps / kMinPart), 1);  // an early tile of a prompt sees less
  if (part >= parts) return false;
  pc->part = part;
  pc->parts = parts;
  pc->from = int(int64_t(steps) * part / parts);
  pc->to = int(int64_t(steps) * (part + 1) / parts);
  return true;
}

// Order of the 16-byte chunks within a row of a tile in LDS.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return D == 64 ? c ^ ((row >> 1) & 7) : c ^ (row & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 64 ? c ^ (((row >> 1) & 1) << 2) : c ^ ((row & 3) << 2);
}

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void chunk_kernel(const ChunkArgs a) {
  constexpr int kLanes = D / 16;                     // lanes that fetch a row
  constexpr int kFetchRows = kThreads / kLanes;      // rows fetched at a time
  constexpr int kFetches = kStepKeys / kFetchRows;
  __shared__ __attribute__((aligned(16))) uint16_t s_k[kStepKeys * D], s_v[kStepKeys * D];
  __shared__ __attribute__((aligned(16))) float4 s_stats[4][32];
  __shared__ int s_bad;   // the last step with a position in a block that does not exist
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
  Piece pc;
  const bool any = find_piece(a, u, &pc);
  const int64_t slot = int64_t(kvh) * a.slots + u;
  if (u < a.slots && tid == 0)
    a.pieces[slot] = any ? make_int4(pc.q0, pc.row0, pc.rows, pc.part | pc.parts << 16)
                         : make_int4(0, 0, 0, 0);
  if (!any) return;

  // Few rows: the waves take different positions instead of different rows.
  const int row_waves = pc.rows > 64 ? 4 : pc.rows > 32 ? 2 : 1, key_waves = 4 / row_waves;
  const int mine = (wave & (row_waves - 1)) * 32;        // this wave's first row of the tile
  const int key_wave = wave / row_waves;
  const int row = mine + col;                            // this lane's
  auto query_of = [&](int r) { return int(a.by_group.div(pc.row0 + r)); };
  const int my_row = min(row, pc.rows - 1), my_query = query_of(my_row);
  const int my_head = kvh * a.group + pc.row0 + my_row - my_query * a.group;
  const int limit = row < pc.rows ? pc.seen(a, my_query) : 0;
  // positions that the wave's last row sees, that its first row sees, that the tile's first sees
  const int wave_most = mine < pc.rows ? pc.seen(a, query_of(min(mine + 32, pc.rows) - 1)) : 0;
  const int wave_least = mine + 32 <= pc.rows ? pc.seen(a, query_of(mine)) : 0;
  const int all_see = pc.seen(a, query_of(0));
  if (tid == 0) s_bad = -1;

  v8bf qf[D / 16];
  {
    const uint16_t* src = a.q + int64_t(pc.q0 + my_query) * a.qs + int64_t(my_head) * D + 8 * half;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      qf[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(src + 16 * s));
  }

  const int32_t* table = a.tables + pc.seq * a.ts;
  const int64_t e = int64_t(a.hkv) * D;
  const int f_row = tid / kLanes, f_chunk = tid % kLanes;
  int ids[kFetches];
  uint4 kx[kFetches], vx[kFetches];
  bool bad = false;
  // block numbers of a step's positions (behind the last one: the last one's)
  auto fetch_ids = [&](int step) {
#pragma unroll
    for (int j = 0; j < kFetches; ++j) {
      const int pos = min(step * kStepKeys + f_row + j * kFetchRows, pc.len - 1);
      ids[j] = table[a.by_block.div(pos)];
    }
  };
  auto fetch = [&](int step) {
    bad = false;
#pragma unroll
    for (int j = 0; j < kFetches; ++j) {
      const int pos = min(step * kStepKeys + f_row + j * kFetchRows, pc.len - 1);
      const int off = pos - int(a.by_block.div(pos)) * a.bs;
      const bool good = ids[j] >= 0 && ids[j] < a.nblocks;
      bad |= !good;
      const int64_t at = (good ? ids[j] : 0) * a.cs + off * e + int64_t(kvh) * D + f_chunk * 16;
      kx[j] = *reinterpret_cast<const uint4*>(a.kc + at);
      vx[j] = *reinterpret_cast<const uint4*>(a.vc + at);
    }
  };
  uint32_t odd = 0;  // not 0: NaN codes of values were left out of steps that not all rows see
  auto stage = [&](int step) {
    const bool edge = (step + 1) * kStepKeys > all_see;
    if (bad) s_bad = step;
#pragma unroll
    for (int j = 0; j < kFetches; ++j) {
      const int r = f_row + j * kFetchRows;
      uint32_t k[4] = {kx[j].x, kx[j].y, kx[j].z, kx[j].w};
      uint32_t v[4] = {vx[j].x, vx[j].y, vx[j].z, vx[j].w};
      if (edge || __any(bad)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t nan = e4m3_nan_bytes(v[i]);
          odd |= nan;
          v[i] &= ~((nan >> 7) * 0xFFu);
        }
      }
      uint32_t kb[8], vb[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kb[2 * i] = e4m3x2_to_bf16<false>(k[i]);
        kb[2 * i + 1] = e4m3x2_to_bf16<true>(k[i]);
        vb[2 * i] = e4m3x2_to_bf16<false>(v[i]);
        vb[2 * i + 1] = e4m3x2_to_bf16<true>(v[i]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 2 * f_chunk + h;
        *reinterpret_cast<uint4*>(s_k + r * D + k_chunk<D>(r, c) * 8) =
            make_uint4(kb[4 * h], kb[4 * h + 1], kb[4 * h + 2], kb[4 * h + 3]);
        *reinterpret_cast<uint4*>(s_v + r * D + v_chunk<D>(r, c) * 8) =
            make_uint4(vb[4 * h], vb[4 * h + 1], vb[4 * h + 2], vb[4 * h + 3]);
      }
    }
  };

  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  float ref = neg_inf(), sum = 0.0f;
  v4f rounded = {0.0f, 0.0f, 0.0f, 0.0f};
  const float scale = a.scale_log2;

  // 32 positions of the staged ones, from row b on; p0 is the first one's position.
  auto block = [&](int b, int p0, int step) {
    v16f s;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      const int r = b + col;
      const v8bf kf = __builtin_bit_cast(
          v8bf, *reinterpret_cast<const uint4*>(s_k + r * D + k_chunk<D>(r, 2 * st + half) * 8));
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st], s, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] *= scale;
    if (p0 + 32 > wave_least) {
      const int left = limit - p0 - 4 * half;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = 8 * (r >> 2) + (r & 3) < left ? s[r] : neg_inf();
    }
    if (s_bad == step) {  // rare: positions in blocks that do not exist
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int pos = min(p0 + 8 * (r >> 2) + (r & 3) + 4 * half, pc.len - 1);
        const int id = table[a.by_block.div(pos)];
        s[r] = id >= 0 && id < a.nblocks ? s[r] : neg_inf();
      }
    }
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    top = max_over_halves(top);
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
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      uint32_t w[4];
#pragma unroll
      for (int t = 0; t < 8; t += 2) {
        const float x = __builtin_amdgcn_exp2f(s[8 * st + t] - base);
        const float y = __builtin_amdgcn_exp2f(s[8 * st + t + 1] - base);
        sum += x + y;
        w[t / 2] = cvt_bf16x2(x, y);
      }
      const v8bf p = __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
      const v4s ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
      rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[0], w[1]}), rounded, 0, 0, 0);
      rounded = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(v4s, v2u{w[2], w[3]}), rounded, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int i16 = lane & 15, side = (lane >> 4) & 1;
        const int ra = b + 16 * st + 4 * half + (i16 >> 2), c = 4 * i + 2 * side + ((i16 & 3) >> 1);
        const int within = 4 * (i16 & 1);
        const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s*)(s_v + ra * D + v_chunk<D>(ra, c) * 8 + within)));
        const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_v4s*)(s_v + (ra + 8) * D + v_chunk<D>(ra + 8, c) * 8 + within)));
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(v8bf, v4u{lo[0], lo[1], hi[0], hi[1]}), p, o[i], 0, 0, 0);
      }
    }
  };

  if (pc.from < pc.to) {
    fetch_ids(pc.from);
    fetch(pc.from);
    if (pc.from + 1 < pc.to) fetch_ids(pc.from + 1);
    for (int step = pc.from; step < pc.to; ++step) {
      __syncthreads();  // what was staged before has been read
      stage(step);
      if (step + 1 < pc.to) {
        fetch(step + 1);
        if (step + 2 < pc.to) fetch_ids(step + 2);
      }
      __syncthreads();
      const int own = kStepKeys / key_waves;
      for (int b = key_wave * own; b < (key_wave + 1) * own; b += 32) {
        const int p0 = step * kStepKeys + b;
        if (p0 < wave_most) block(b, p0, step);
      }
    }
  }

  // NaN codes that were left out reach the rows that see them.
  if (__syncthreads_or(int(odd))) {
    if (key_wave == 0) {
      const int first = max(pc.from, all_see / kStepKeys) * kStepKeys;
      const int end = min(limit, min(pc.to * kStepKeys, pc.len));
      const int64_t at0 = int64_t(kvh) * D + 4 * half;
      for (int pos = s_bad >= 0 ? pc.from * kStepKeys : first; pos < end; ++pos) {
        const uint32_t blk = a.by_block.div(pos);
        const int id = table[blk];
        if (id < 0 || id >= a.nblocks) continue;
        const uint8_t* v = a.vc + id * a.cs + (pos - int(blk) * a.bs) * e + at0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const uint32_t nan = e4m3_nan_bytes(*reinterpret_cast<const uint32_t*>(v + 32 * i + 2 * r));
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (nan >> (8 * t + 7) & 1) o[i][r + t] = __builtin_nanf("");
          }
      }
    }
  }

  float total = sum_over_halves(sum), of_rounded = sum_over_halves(rounded[0]);
  // Waves that took different positions of the same rows add up in pairs, through LDS.
  float* const s_o = reinterpret_cast<float*>(s_k);
  for (int n = key_waves / 2; n >= 1; n /= 2) {
    __syncthreads();
    const int to = wave & (row_waves * n - 1);
    if (key_wave >= n && key_wave < 2 * n) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s_o[((to * (D / 32) + i) * 16 + r) * 64 + lane] = o[i][r];
      if (half == 0) s_stats[to][col] = make_float4(ref, total, of_rounded, 0.0f);
    }
    __syncthreads();
    if (key_wave < n) {
      const float4 st = s_stats[wave][col];
      const float up = fmaxf(ref, st.x);
      const float f = ref == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(ref - up);
      const float h = st.x == neg_inf() ? 0.0f : __builtin_amdgcn_exp2f(st.x - up);
      ref = up;
      total = total * f + st.y * h;
      of_rounded = of_rounded * f + st.z * h;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          o[i][r] = o[i][r] * f + s_o[((wave * (D / 32) + i) * 16 + r) * 64 + lane] * h;
    }
  }
  if (key_wave > 0 || row >= pc.rows) return;
  if (pc.parts > 1) {
    const int64_t at = slot * kTileRows + row;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(a.sums + at * D + 32 * i + 2 * r + 4 * half) =
            make_float4(o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]);
    if (half == 0) a.stats[at] = make_float4(ref, total, of_rounded, 0.0f);
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
  const int at_once = num_cus() * (d == 256 ? 1 : 2);
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
