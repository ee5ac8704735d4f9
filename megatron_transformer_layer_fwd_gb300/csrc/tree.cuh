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
// Ways to cut (TreeCut): for sequences with few rows on average, items of up to 16 rows for
// the kernel of the decode step (paged_rows.cuh); else items of up to 256 rows for the tcgen05
// kernel, and a second table with items of up to 64 rows for the float32 kernel.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mgb {

constexpr int TREE_MAX = MGB_TREE_MAX_TOKENS;
constexpr int TREE_WORDS = TREE_MAX / 32;  // of a token's mask: bit j, the sequence's drafted token j is seen
constexpr int TREE_LONGEST = INT32_MAX - 1024;  // cached tokens (so that keys behind the last one stay below 2^31)

// The cuts for many rows: keys of a unit, rows of an item, units of an item that is never split,
// its fixed cost, CTAs, and the cost of a unit by the item's rows. A range costs at least one
// unit, so that none between two others is empty.
// bf16: more than 64 rows keep the warps busy whose schedulers run the loaders too, which with pages
// of 16 slots takes up to a fifth longer, with large pages nothing: 9 / 8 is between (32
// sequences of 33 to 16000 tokens, 8 to 96 rows: with one cost for both 61 us at pages of 16 and
// 54.7 at 64, with 9 / 8 57.4 and 55.0, with 10 / 8 57.2 and 55.4). Two halves: 4550 cycles at head dim 128, one 2612.
// An item's fixed cost, 64 sequences of 33 to 4000 tokens, 240 rows: 127, 113, 97 and 96 us with 8,
// 16, 24 and 32, 20 rows 76, 67.7, 68.2 and 70.7.
struct CutTc {
  static constexpr int KEYS = 128, ROWS = 256, WHOLE = 2, ITEM = 24, RANGES = 152;
  static constexpr int R1 = 64, R2 = 128, C1 = 8, C2 = 9, C3 = 14;
};
template <int D>
struct CutF32 {
  static constexpr int KEYS = D == 64 ? 64 : 32, ROWS = 64, WHOLE = 2, ITEM = 4, RANGES = 304;
  static constexpr int R1 = 16, R2 = 32, C1 = 2, C2 = 3, C3 = 5;
};
template <typename Cut>
__host__ __device__ constexpr int unit_cost(int rows) {
  return rows <= Cut::R1 ? Cut::C1 : rows <= Cut::R2 ? Cut::C2 : Cut::C3;
}

constexpr int TREE_FEW = 4;
constexpr int TREE_ROW_STEP = 8;  // rows of a part in the workspace: a multiple of it
struct TreeHeader {
  int64_t cost, chunk;  // of all items; of a range
  int32_t live, bad;    // sequences with items; (of many) the first one with an offset outside its range
  int32_t few, many;    // items in up to TREE_FEW parts, in more: from the front and from the back of the list
};
// A sequence's rows of q and o begin at row `row`, `m` of them; `len` cached tokens
// with the drafted ones; `s` its row of the block table.
struct TreeSeq {
  int32_t row, m, len, s;
};
// Where a range begins: unit t of item (live sequence i, KV head h, block b), the
// item at `at` on the cost axis. The sequence and the next one are beside it, which saves the
// kernels a dependent read.
struct TreeStart {
  int64_t at;
  int32_t i, h, b, t;
  TreeSeq q, next;
};
// An item in the parts of several CTAs, c the first of them: its part in the workspace at
// `first`, those of the others at 2 CTA.
struct TreeSplit {
  int32_t c, parts, first, row;  // row: the sequence's first one
  int32_t r0, rows, h, len;      // the block's first row, its rows, the KV head, the sequence's length
};
// What a drafted token is to the cache: its sequence (-1: none), slot and depth position.
struct TreeToken {
  int32_t s, slot, pos, pad;
};

struct TreeTable {
  size_t header, start, split, live, prefix, counter;
  int rows;  // of a part
};
struct TreeLayout {
  size_t seq, token, mask, ml, part, total;
  TreeTable table[2];  // for bf16, for float32
};

// How the work is cut, by the sizes that the host knows.
struct TreeCut {
  int narrow;
  int keys, rows;              // of a unit; of an item at most
  int r1, r2, c1, c2, c3;      // cost of a unit: c1 up to r1 rows, c2 up to r2, c3
  int item, whole, min_chunk, ranges;
};
TreeCut tree_cut(int n, int tokens, int nq, int nkv, int d, int table);
TreeLayout tree_layout(int n, int tokens, int nq, int nkv, int d);

struct TreeParams {
  int n, nq, nkv, G, tokens;
  const TreeHeader* hdr;
  const TreeStart* start;
  const TreeSplit* split;
  const TreeSeq* live;
  const uint32_t* mask;
  uint32_t* counter;  // (few rows: a split item's arrivals)
  float2* ml;   // [2 CTAs][rows] (maximum in log2 units, row sum) of a part
  float* part;  // [2 CTAs][d / 4][rows][4] (few rows: [2 CTAs][rows][d])
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

template <typename Cut>
__host__ __device__ inline int tree_units(int len) {
  return (int)(((int64_t)len + Cut::KEYS - 1) / Cut::KEYS);
}
// where unit t of an item with n units begins on its part of the cost axis
template <typename Cut>
__host__ __device__ inline int64_t tree_begin(int t, int n, int rows) {
  return n > Cut::WHOLE ? (int64_t)t * unit_cost<Cut>(rows) : 0;
}

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
template <typename Cut>
struct TreeSegs {
  int64_t at, begin_at, end;
  int i, h, b, t, n;
  TreeSeq cur, nxt;
  __device__ void fetch(const TreeParams& p) {
    if (i + 1 < n) {
      const int4 x = *reinterpret_cast<const int4*>(p.live + i + 1);
      nxt = TreeSeq{x.x, x.y, x.z, x.w};
    }
  }
  // CTA c's units; false: none (and next() says so too)
  __device__ bool begin(const TreeParams& p, int c) {
    const TreeHeader hd = *p.hdr;
    const TreeStart st = p.start[c];
    at = st.at; i = st.i; h = st.h; b = st.b; t = st.t;
    n = hd.live;
    begin_at = c * hd.chunk;
    end = min(begin_at + hd.chunk, hd.cost);
    cur = st.q;
    nxt = st.next;
    return i < n;
  }
  // false: no more. Sequences longer than the table are passed over.
  __device__ bool next(const TreeParams& p, TreeSeg& w) {
    for (;;) {
      if (i >= n) return false;
      const int nt = tree_units<Cut>(cur.len), left_rows = cur.m * p.G - b * Cut::ROWS;
      const int rows = min(Cut::ROWS, left_rows), unit = unit_cost<Cut>(rows);
      if (at + tree_begin<Cut>(t, nt, rows) >= end) return false;
      w.q = cur;
      w.h = h; w.b = b; w.at = at; w.nt = nt; w.t0 = t; w.rows = rows;
      const int64_t room = end - at;  // (a division only where the range ends inside the item)
      w.t1 = nt > Cut::WHOLE && room <= (int64_t)(nt - 1) * unit ? (int)((room + unit - 1) / unit) : nt;
      const bool skip = cur.len > p.cap;
      t = 0;
      at += (int64_t)nt * unit + Cut::ITEM;
      ++b;
      if (left_rows <= Cut::ROWS) {
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
  // whether all units of a segment's item are this CTA's
  __device__ bool whole(const TreeSeg& w) const {
    return w.at >= begin_at && w.at + tree_begin<Cut>(w.nt - 1, w.nt, w.rows) < end;
  }
};

// The part of the workspace with the share of the item at `at` of CTA cc, whose range begins at
// `begin`: 2 cc when that is at or inside the item, 2 cc + 1 when before it.
__device__ __forceinline__ int tree_part(int cc, int64_t begin, int64_t at) {
  return 2 * cc + (begin < at ? 1 : 0);
}

// Place of columns 4 c .. of a row of a part: rows lie next to each other, as the threads that
// write and read them do.
__device__ __forceinline__ float4* tree_part_at(const TreeParams& p, int part, int d, int c, int row) {
  return reinterpret_cast<float4*>(p.part) + ((int64_t)part * (d / 4) + c) * p.rows + row;
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
// Joins the parts of split items (in tree_plan.cu).
template <typename T, int D>
mgb_status tree_join(const TreeParams& p, int ranges, cudaStream_t st);
mgb_status attention_tree_rows(const TreeParams& p, int d, int dtype, cudaStream_t st);
mgb_status attention_tree_bf16(const TreeParams& p, int d, cudaStream_t st);
mgb_status attention_tree_f32(const TreeParams& p, int d, cudaStream_t st);

}  // namespace mgb
