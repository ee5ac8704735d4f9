// Shared by the kernels for drafted tokens: the plan's workspace, and how the
// attention's work is cut into ranges.
//
// Unit: consecutive cached tokens of an item. Item: all units of one (sequence, KV head,
// block of rows), a row being a drafted token and one of the KV head's query heads (row r of a
// sequence: token r / G, head r % G). Items stand one behind the other on a cost axis,
// sequence by sequence, head by head, block by block: an item with n units takes n unit
// costs and a fixed one, its unit t beginning at t unit costs (all units of a short item begin
// at its start: splitting it would cost more than it evens out). CTA c takes the units that
// begin in [c chunk, (c + 1) chunk). An item that lies in one CTA's range is finished there;
// the parts of one that does not (unnormalised sums, maximum, row sum) are joined in CTA order.
//
// Two ways to cut (TreeCut): for sequences with few rows on average, items of up to 16 rows
// for the kernel of the decode step (paged_rows.cuh); else items of up to 256 rows for the
// tcgen05 kernel and the float32 one.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mgb {

constexpr int TREE_MAX = MGB_TREE_MAX_TOKENS;
constexpr int TREE_WORDS = TREE_MAX / 32;  // of a token's mask: bit j, the sequence's drafted token j is seen
// the cut for many rows
constexpr int TREE_ROWS = 256;             // rows of an item at most
constexpr int TREE_KEYS = 128;             // keys of a unit
constexpr int TREE_LONGEST = INT32_MAX - 1024;  // cached tokens (so that keys behind the last one stay below 2^31)
constexpr int TREE_RANGES = 304;           // two per SM of a GB300 (the bf16 kernel takes two at a time)
constexpr int TREE_UNIT = 4;               // cost of a unit
constexpr int TREE_ITEM = 4;               // fixed cost of an item
constexpr int TREE_WHOLE = 2;              // units of an item that is never split
constexpr int TREE_MIN_CHUNK = TREE_UNIT;  // of a range: none between two others is empty

struct TreeHeader {
  int64_t cost, chunk;  // of all items; of a range
  int32_t live;         // sequences with items
  int32_t rows;         // rows behind this one belong to no sequence
};
// A sequence's rows of q and o begin at row `row`, `m` of them; `len` cached tokens
// with the drafted ones; `s` its row of the block table.
struct TreeSeq {
  int32_t row, m, len, s;
};
// Where a range begins: unit t of item (live sequence i, KV head h, block b), the
// item at `at` on the cost axis.
struct TreeStart {
  int64_t at;
  int32_t i, h, b, t;
};
// What a drafted token is to the cache: its sequence (-1: none), slot and depth position.
struct TreeToken {
  int32_t s, slot, pos, pad;
};

struct TreeLayout {
  size_t header, start, seq, live, prefix, token, mask, counter, ml, part, total;
  int rows;  // of a part
};

// How the work is cut, by the sizes that the host knows.
struct TreeCut {
  int narrow;
  int keys, rows;        // of a unit; of an item at most
  int unit, item;        // costs of a unit and of an item
  int whole;             // units of an item that is never split
  int min_chunk, ranges;
};
TreeCut tree_cut(int n, int tokens, int nq, int nkv, int d);
TreeLayout tree_layout(int n, int tokens, int nq, int nkv, int d);

__host__ __device__ inline int tree_units(int len) { return (int)(((int64_t)len + TREE_KEYS - 1) / TREE_KEYS); }
__host__ __device__ inline int tree_blocks(int m, int G) {
  return (int)(((int64_t)m * G + TREE_ROWS - 1) / TREE_ROWS);
}
__host__ __device__ inline int64_t tree_cost(int units) { return (int64_t)units * TREE_UNIT + TREE_ITEM; }
// where unit t of an item with n units begins on its part of the cost axis
__host__ __device__ inline int64_t tree_begin(int t, int n) {
  return n > TREE_WHOLE ? (int64_t)t * TREE_UNIT : 0;
}

struct TreeParams {
  int nq, nkv, G;
  const TreeHeader* hdr;
  const TreeStart* start;
  const TreeSeq* live;
  const uint32_t* mask;
  uint32_t* counter;  // (few rows: a split item's arrivals)
  float2* ml;   // [2 CTAs][rows] (maximum in log2 units, row sum) of a part
  float* part;  // [2 CTAs][rows][d]
  int rows;
  const void *k, *v;
  const int32_t* table;
  int64_t s_page, s_tok, s_head, ld_table;
  int n_pages, page_size;
  int cap;      // tokens a row of the table holds
  const void* q;
  int64_t ld_q;
  void* o;
  int64_t ld_o;
  float* lse;
  float sl2;    // log2(e) / sqrt(d)
  int* err;
};

// The units of one item that a CTA takes.
struct TreeSeg {
  TreeSeq q;      // the sequence
  int h, b, rows; // KV head, row block, its rows
  int t0, t1;     // units
  int64_t at;     // the item on the cost axis
  int nt;         // its units
};

// A CTA's segments in order, the same for every role. The next sequence is
// requested one sequence ahead.
struct TreeSegs {
  int64_t at, end;
  int i, h, b, t, n;
  TreeSeq cur, nxt;
  __device__ void fetch(const TreeParams& p) {
    if (i + 1 < n) {
      const int4 x = *reinterpret_cast<const int4*>(p.live + i + 1);
      nxt = TreeSeq{x.x, x.y, x.z, x.w};
    }
  }
  // the units from st on that begin before range_end; false: none
  __device__ bool begin(const TreeParams& p, const TreeHeader& hd, const TreeStart& st, int64_t range_end) {
    at = st.at; i = st.i; h = st.h; b = st.b; t = st.t;
    n = hd.live;
    end = range_end;
    if (i >= n) return false;
    const int4 x = *reinterpret_cast<const int4*>(p.live + i);
    cur = TreeSeq{x.x, x.y, x.z, x.w};
    fetch(p);
    return true;
  }
  // false: no more. Sequences longer than the table are passed over.
  __device__ bool next(const TreeParams& p, TreeSeg& w) {
    for (;;) {
      if (i >= n) return false;
      const int nt = tree_units(cur.len);
      if (at + tree_begin(t, nt) >= end) return false;
      const int nb = tree_blocks(cur.m, p.G);
      w.q = cur;
      w.h = h; w.b = b; w.at = at; w.nt = nt; w.t0 = t;
      w.rows = min(TREE_ROWS, cur.m * p.G - b * TREE_ROWS);
      const int64_t left = (end - at + TREE_UNIT - 1) / TREE_UNIT;
      w.t1 = nt > TREE_WHOLE && left < nt ? (int)left : nt;
      const bool skip = cur.len > p.cap;
      t = 0;
      at += tree_cost(nt);
      if (++b == nb) {
        b = 0;
        if (++h == p.nkv) {
          h = 0;
          ++i;
          cur = nxt;
          fetch(p);
        }
      }
      if (!skip) return true;
      if (threadIdx.x % 32 == 0) record_error(p.err, kErrIndex);
    }
  }
};

// The part of the workspace with CTA cc's share of the item at `at`: 2 cc when the
// CTA's range begins at or inside the item, 2 cc + 1 when before it.
__device__ __forceinline__ int tree_part(int cc, int64_t chunk, int64_t at) {
  return 2 * cc + (cc * chunk < at ? 1 : 0);
}

// The 32 mask bits of drafted tokens first .. first + 31 (those before 0 are cached
// tokens, seen by all; those behind the mask are none).
__device__ __forceinline__ uint32_t tree_window(const uint32_t* mask, int first) {
  if (first <= -32) return ~0u;
  if (first < 0) return (mask[0] << -first) | ((1u << -first) - 1u);
  const int w = first >> 5, s = first & 31;
  if (w >= TREE_WORDS) return 0u;
  const uint32_t lo = mask[w] >> s;
  return s == 0 || w + 1 >= TREE_WORDS ? lo : lo | (mask[w + 1] << (32 - s));
}

mgb_status check_tree_plan(const mgb_attention_tree_plan* plan);
// Joins the parts of split items (bf16 or float32 output).
mgb_status tree_join(const TreeParams& p, int d, int dtype, int ctas, int mult, cudaStream_t st);
mgb_status attention_tree_rows(const TreeParams& p, int d, int dtype, cudaStream_t st);
mgb_status attention_tree_bf16(const TreeParams& p, int d, cudaStream_t st);
mgb_status attention_tree_f32(const TreeParams& p, int d, cudaStream_t st);

}  // namespace mgb
