// Work decomposition shared by the dense-attention kernels.
//
// Grouped heads: the `group` query heads that read one key/value head are packed into rows, row
// r = (token, query head of the group) = (r / group, r % group), so that a tile's rows share every
// key and value and a single token still fills `group` rows.
//
// Prompt: a unit is (sequence, key/value head, block of ROWS packed rows) and runs over the keys up
// to its last token. CTAs take units in descending row-block index over all sequences: the longest
// runs first, the short ones fill up behind them.
//
// Tree: a unit is (batch entry, key/value head, row block); its keys are the cached rows, in tiles
// of KT, followed by the drafted nodes in tiles of KT. All units' tiles form one line that is cut
// into gridDim.x equal shares, whatever the lengths; units cut in two or more are joined by
// k_dense_join.
#pragma once

#include "common.cuh"
#include "dense.h"

namespace iskv {
namespace dense {

// status: one int64 word, bit (1 << code).
// (Out of line: the callers run once per unit, and their instructions come from L2 each time.)
static __device__ __noinline__ void report(int64_t *status, int code) {
  atomicOr(reinterpret_cast<unsigned long long *>(status), 1ull << code);
}

// One unit's place: tiles [t0, t1) of its n_tiles.
struct Unit {
  int b;          // sequence / batch entry; -1: nothing to do
  int kvh;
  int row0;       // first packed row of the block
  int n_rows;     // packed rows of the block (<= ROWS)
  int64_t base;   // prompt: first packed row of the sequence in q / k / v
  int len;        // prompt: tokens of the sequence; tree: cached rows
  int cache_tiles;  // tree: key tiles over the cache (the drafted nodes' follow)
  int n_tiles;
  int t0, t1;
  int open;       // first key (prompt: token; tree: cached row) that some row must not see
};

// Rows of sequence s from lo on; -1 (reported) if its bounds contradict each other or the rows.
ISKV_DEV int seq_len(const DenseArgs &a, int s, int64_t &lo) {
  if (!a.cu) {  // one sequence of all rows
    lo = 0;
    return (int)a.rows;
  }
  const int64_t b = a.cu[s], e = a.cu[s + 1];
  lo = b;
  if (b < 0 || e < b || e > a.rows) {
    report(a.status, ISKV_ERR_SHAPE);
    return -1;
  }
  return (int)(e - b);
}

// Whole warp: the rank-th unit (without its head) of a prompt call. F(m) = sum over sequences of
// max(blocks - m, 0) counts the blocks with index >= m; the unit has the largest m with
// F(m) > rank. Sequences count up to the first whose bounds are inconsistent: those before it are
// disjoint, so that no row belongs to two units and the grid, made for n_rows rows, has a CTA for
// each.
// Every CTA walks the list of sequences at every step of the search, 32 at a time: 32 sequences of
// 16 tokens take 23 us in all, 256 of them 162 us and 4,096 16.5 ms (32 over 8 heads of 128, bf16).
template <int ROWS>
ISKV_DEV bool find_prompt_unit(const DenseArgs &a, int rank, Unit &u) {
  const int lane = threadIdx.x & 31;
  if (a.batch == 1) {
    u.len = seq_len(a, 0, u.base);
    const int n = (int)(((int64_t)u.len * a.group + ROWS - 1) / ROWS);
    if (rank >= n) return false;  // (n <= 0 for -1 rows)
    u.b = 0;
    u.row0 = (n - 1 - rank) * ROWS;
    u.n_rows = min(ROWS, u.len * a.group - u.row0);
    return true;
  }
  int seqs = a.batch;  // consistent ones, once every lane has looked at its own
  auto blocks = [&](int s) {
    if (s >= seqs) return 0;
    int64_t lo;
    const int n = seq_len(a, s, lo);
    if (n < 0) seqs = s;
    return (int)(((int64_t)max(n, 0) * a.group + ROWS - 1) / ROWS);
  };
  int mine = blocks(lane);  // the first 32 sequences stay in registers
  int top = mine;
#pragma unroll 1
  for (int s = 32 + lane; s < a.batch; s += 32) top = max(top, blocks(s));
  top = __reduce_max_sync(0xffffffffu, top);  // (of a sequence that does not count at worst)
  seqs = __reduce_min_sync(0xffffffffu, seqs);
  if (lane >= seqs) mine = 0;
  auto F = [&](int m) {
    int n = max(mine - m, 0);
#pragma unroll 1
    for (int s = 32 + lane; s < seqs; s += 32) n += max(blocks(s) - m, 0);
    return __reduce_add_sync(0xffffffffu, n);
  };
  if (top == 0) return false;
  int lo = -1, hi = top, above = 0;  // F(lo) > rank >= F(hi) = above, but for lo = -1
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2, f = F(mid);
    if (f > rank) {
      lo = mid;
    } else {
      hi = mid;
      above = f;
    }
  }
  if (lo < 0) return false;
  int skip = rank - above;  // among the sequences with more than lo blocks
#pragma unroll 1
  for (int s0 = 0; s0 < seqs; s0 += 32) {
    const unsigned has = __ballot_sync(0xffffffffu, (s0 == 0 ? mine : blocks(s0 + lane)) > lo);
    const int n = __popc(has);
    if (skip >= n) {
      skip -= n;
      continue;
    }
    const unsigned pick = __ballot_sync(
        0xffffffffu, (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == skip);
    u.b = s0 + __ffs(pick) - 1;
    break;
  }
  u.len = seq_len(a, u.b, u.base);
  u.row0 = lo * ROWS;
  u.n_rows = min(ROWS, u.len * a.group - u.row0);
  return true;
}

// |scale| log2(e), the factor on the scores (its sign goes into the queries). Never 0, because
// masked scores are -inf: with scale 0 it is the smallest float, 2^-149, which takes any finite
// score to 2^-21 or less.
ISKV_DEV float score_factor(const DenseArgs &a) {
  return fmaxf(fabsf(a.scale) * 1.4426950408889634f, __int_as_float(1));
}

// Tokens of the first and last row of a block.
ISKV_DEV int first_token(const DenseArgs &a, const Unit &u) { return u.row0 / a.group; }
ISKV_DEV int last_token(const DenseArgs &a, const Unit &u) {
  return (u.row0 + u.n_rows - 1) / a.group;
}

ISKV_DEV int cached_rows(const DenseArgs &a, int b) {
  if (!a.n_cached) return (int)a.rows;
  const int n = a.n_cached[b];
  if (n < 0 || n > a.rows) {
    report(a.status, ISKV_ERR_SHAPE);
    return n < 0 ? 0 : (int)a.rows;
  }
  return n;
}

// The line of a tree call's tiles (fewer than 2^31, which the entry point checks) and a CTA's way
// along its share of it (whole-warp calls). Shares are `per` tiles each, the last ones may be
// empty.
template <int ROWS, int KT>
struct TreeLine {
  int blocks, draft_tiles;
  int len0;  // cached rows of entry `lane`: the first 32 entries stay in registers
  int per, x, end;

  // b: the lane itself or from 32 on
  ISKV_DEV int len_of(const DenseArgs &a, int b) const { return b < 32 ? len0 : cached_rows(a, b); }
  ISKV_DEV int entry_tiles(const DenseArgs &a, int b) const {
    return b < a.batch ? ((len_of(a, b) + KT - 1) / KT + draft_tiles) * (a.n_kv * blocks) : 0;
  }
  ISKV_DEV void begin(const DenseArgs &a, int grid, int cta) {
    const int lane = threadIdx.x & 31;
    if (a.whole) {  // the CTA's number is its unit's
      blocks = (a.nodes * a.group + ROWS - 1) / ROWS;
      draft_tiles = (a.nodes + KT - 1) / KT;
      x = cta;
      end = cta + 1;
      return;
    }
    blocks = (a.nodes * a.group + ROWS - 1) / ROWS;
    draft_tiles = (a.nodes + KT - 1) / KT;
    len0 = lane < a.batch ? cached_rows(a, lane) : 0;
    int total = 0;
    for (int b = lane; b < a.batch; b += 32) total += entry_tiles(a, b);
    total = __reduce_add_sync(0xffffffffu, total);
    per = (int)((unsigned)(total - 1) / (unsigned)grid) + 1;
    x = (int)min((int64_t)total, (int64_t)per * cta);
    end = min(total - x, per) + x;
  }
  // Everything of entry u.b's idx-th unit but its tile range.
  ISKV_DEV void place(const DenseArgs &a, int idx, Unit &u) const {
    u.base = 0;
    u.cache_tiles = (u.len + KT - 1) / KT;
    u.n_tiles = u.cache_tiles + draft_tiles;
    u.kvh = blocks == 1 ? idx : idx / blocks;
    u.row0 = (idx - u.kvh * blocks) * ROWS;
    u.n_rows = min(ROWS, a.nodes * a.group - u.row0);
  }
  // The next unit of the share, or false.
  ISKV_DEV bool next(const DenseArgs &a, Unit &u) {
    if (x >= end) return false;
    const int lane = threadIdx.x & 31;
    int before = 0;
    if (a.whole) {
      const int units = a.n_kv * blocks;
      u.b = x / units;
      u.len = cached_rows(a, u.b);
      place(a, x - u.b * units, u);
      u.t0 = 0;
      u.t1 = u.n_tiles;
      ++x;
      return true;
    }
    if (a.batch == 1) {
      u.b = 0;
      u.len = __shfl_sync(0xffffffffu, len0, 0);
    }
    for (int b0 = 0; a.batch > 1; b0 += 32) {
      const int n = entry_tiles(a, b0 + lane);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + sum > x);
      if (past) {
        const int l = __ffs(past) - 1;
        before += __shfl_sync(0xffffffffu, sum - n, l);
        u.b = b0 + l;
        u.len = __shfl_sync(0xffffffffu, b0 + lane < a.batch ? len_of(a, b0 + lane) : 0, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    const int idx = (x - before) / ((u.len + KT - 1) / KT + draft_tiles);
    place(a, idx, u);
    u.t0 = x - before - idx * u.n_tiles;
    u.t1 = min(u.n_tiles, u.t0 + (end - x));
    x += u.t1 - u.t0;
    return true;
  }
};

// Whole warp: bits of the nodes that each lane's node i sees, given its entry's parents: itself and
// its ancestors. par[i] is the index of an earlier node, or -1 (a child of the last cached token);
// an entry below -1 is padding. Padding, a node whose chain reaches padding, and an entry that is
// not below its own index (reported) see nothing. The parents sit in four registers of the warp, a
// step up the chain is a shuffle.
ISKV_DEV void node_mask(const DenseArgs &a, const int32_t *par, int i, uint32_t (&m)[4]) {
  const int lane = threadIdx.x & 31;
  int p[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    p[w] = w * 32 + lane < a.nodes ? par[w * 32 + lane] : -2;
    m[w] = 0;
  }
  int cur = i;
  bool live = true;
  while (__any_sync(0xffffffffu, live && cur >= 0)) {
    int up = -1;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int x = __shfl_sync(0xffffffffu, p[w], cur & 31);
      if ((cur >> 5) == w) up = x;
    }
    if (!live || cur < 0) continue;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if ((cur >> 5) == w) m[w] |= 1u << (cur & 31);
    if (up >= cur) report(a.status, ISKV_ERR_SHAPE);
    if (up >= cur || up < -1) live = false;
    cur = up;
  }
  if (!live) m[0] = m[1] = m[2] = m[3] = 0;
}

}  // namespace dense
}  // namespace iskv
