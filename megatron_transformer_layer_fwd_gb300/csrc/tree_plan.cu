// Drafted tokens over a paged cache: the plan of a step, the join of split
// items, and the attention's entry points.
//
// The plan says what each drafted token sees and where it stands. Its mask is its own
// bit and its parent's mask, found by doubling: with anc(i) the token 2^r steps
// up, mask(i) |= mask(anc(i)), anc(i) = anc(anc(i)), at most eight rounds for 256
// tokens; its depth adds up along the same steps. One sequence 4.5 us, 96 5.7: dependent reads and
// block-wide steps, once for all layers of a step; 4000 32 and 70000 399, a step of the tables' blocks
// for every 256 sequences.
#include "paged_rows.cuh"

namespace mgb {

namespace {

constexpr int PT = 256;  // threads of the prepare kernel

// What a sequence's offsets and length say; `ok`: no offset up to it is bad.
enum : int { SEQ_LIVE, SEQ_IDLE, SEQ_BAD };
__device__ __forceinline__ int seq_kind(bool ok, int m, int len) {
  if (!ok || len < 0) return SEQ_BAD;
  if (m == 0 || len == 0) return SEQ_IDLE;  // no rows, or padding
  return m <= TREE_MAX && m <= len ? SEQ_LIVE : SEQ_BAD;
}

struct PlanArgs {
  int n, tokens, G, nkv;
  const int32_t *cu, *lens, *parents;
  TreeSeq* seq;
  TreeToken* token;
  uint32_t* mask;
  int32_t* bad;  // first sequence with a bad offset (NULL: each block looks at all those before its own)
  int* err;
  // per table
  TreeCut cut[2];
  TreeHeader* hdr[2];
  TreeStart* start[2];
  TreeSplit* split[2];
  uint32_t* counter[2];
  TreeSeq* live[2];
  int64_t* prefix[2];
};

// a / b for a >= 0, b > 0: most are small, and a division of 64 bits takes some hundred instructions
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int unit_of(const TreeCut& c, int rows) {
  return rows <= c.r1 ? c.c1 : rows <= c.r2 ? c.c2 : c.c3;
}
// A sequence's items for one KV head: blocks of cut.rows rows, the last one smaller.
struct SeqCost {
  int units, blocks, unit_full, unit_last;
  int64_t full, last;  // cost of an item of either kind
  __device__ SeqCost(const TreeCut& c, int len, int64_t rows) {
    units = (int)quot((int64_t)len + c.keys - 1, c.keys);
    blocks = (int)quot(rows + c.rows - 1, c.rows);
    unit_full = unit_of(c, c.rows);
    unit_last = unit_of(c, (int)(rows - (int64_t)(blocks - 1) * c.rows));
    full = (int64_t)units * unit_full + c.item;
    last = (int64_t)units * unit_last + c.item;
  }
  __device__ int64_t head() const { return (blocks - 1) * full + last; }
};

__device__ __forceinline__ bool pair_ok(const PlanArgs& a, int s, int c0, int c1) {
  return c0 >= 0 && c1 >= c0 && c1 <= a.tokens && (s > 0 || c0 == 0);
}

// With many sequences the first bad offset is found once, by one block, which writes n if all are good:
// where each sequence's block looks at all those before its own, the reads go with the square of
// their number. The whole prepare, this way and the other: 2000 sequences 19.4 and 18.3 us, 4000 31.8
// and 32.3, 8000 55.8 and 64.5, 70000 399 and 2590.
constexpr int MANY_SEQS = 4096;
constexpr int BT = 1024;
__global__ void __launch_bounds__(BT) tree_first_bad_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int first;
  if (threadIdx.x == 0) first = a.n;
  __syncthreads();
  int mine = a.n;
#pragma unroll 4
  for (int s = threadIdx.x; s < a.n; s += BT)
    if (!pair_ok(a, s, a.cu[s], a.cu[s + 1])) mine = min(mine, s);
  if (mine < a.n) atomicMin(&first, mine);
  __syncthreads();
  if (threadIdx.x == 0) *a.bad = first;
}

// The blocks behind the sequences' (one per table): the live sequences in order, their costs
// summed up, the first unit of every range. Block s: what the tokens of sequence s see.
__global__ void __launch_bounds__(PT) tree_prepare_kernel(const __grid_constant__ PlanArgs a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();  // the attention kernel may start up; it waits for this one's end
  if ((int)blockIdx.x < a.n) {
    __shared__ uint32_t m[TREE_MAX][TREE_WORDS + 1];
    __shared__ int anc[TREE_MAX], dep[TREE_MAX];
    const int s = blockIdx.x;
    const int c0 = a.cu[s], c1 = a.cu[s + 1], len = a.lens[s];
    bool good = pair_ok(a, s, c0, c1);
    if (!good && tid == 0) record_error(a.err, kErrIndex);
    if (a.bad != nullptr) good = good && s < *a.bad;  // (a bad offset before it: the sequence counts as empty)
    else if (c1 != c0)
      for (int i = tid; i < s; i += PT) good = good && pair_ok(a, i, a.cu[i], a.cu[i + 1]);
    good = __syncthreads_and(good);
    const int rows = c1 - c0;
    const int kind = good ? seq_kind(true, rows, len) : SEQ_BAD;
    if (tid == 0) {
      if (good && kind == SEQ_BAD) record_error(a.err, kErrIndex);
      *reinterpret_cast<int4*>(a.seq + s) =
          make_int4(kind == SEQ_LIVE ? c0 : 0, kind == SEQ_LIVE ? rows : 0, max(len, 0), s);
    }
    if (!good) return;
    if (kind != SEQ_LIVE) {
      for (int i = tid; i < rows; i += PT)
        *reinterpret_cast<int4*>(a.token + c0 + i) = make_int4(-1, 0, 0, 0);
      return;
    }
    // PT >= TREE_MAX: a thread per token
    const int i = tid;
    if (i < rows) {
      int up = i - 1;
      if (a.parents != nullptr) {
        up = a.parents[c0 + i];
        if (up < -1 || up >= i) {  // counts as a child of the last cached token
          record_error(a.err, kErrIndex);
          up = -1;
        }
      }
#pragma unroll
      for (int w = 0; w < TREE_WORDS; ++w) m[i][w] = w == (i >> 5) ? 1u << (i & 31) : 0u;
      anc[i] = up;
      dep[i] = up >= 0 ? 1 : 0;
    }
    for (;;) {
      const int x = i < rows ? anc[i] : -1;
      if (!__syncthreads_or(x >= 0)) break;
      uint32_t add[TREE_WORDS];
      int xa = -1, xd = 0;
      if (x >= 0) {
#pragma unroll
        for (int w = 0; w < TREE_WORDS; ++w) add[w] = m[x][w];
        xa = anc[x];
        xd = dep[x];
      }
      __syncthreads();
      if (x >= 0) {
#pragma unroll
        for (int w = 0; w < TREE_WORDS; ++w) m[i][w] |= add[w];
        anc[i] = xa;
        dep[i] += xd;
      }
      __syncthreads();
    }
    if (i < rows) {
      uint4* out = reinterpret_cast<uint4*>(a.mask + (int64_t)(c0 + i) * TREE_WORDS);
      static_assert(TREE_WORDS == 8, "two stores per token");
      out[0] = make_uint4(m[i][0], m[i][1], m[i][2], m[i][3]);
      out[1] = make_uint4(m[i][4], m[i][5], m[i][6], m[i][7]);
      *reinterpret_cast<int4*>(a.token + c0 + i) = make_int4(s, len - rows + i, len - rows + dep[i], 0);
    }
    return;
  }

  // ---------------- a table's ranges
  const int tab = blockIdx.x - a.n;
  const TreeCut cut = a.cut[tab];
  TreeSeq* const live_out = a.live[tab];
  // (read back below: from shared memory if they fit)
  __shared__ TreeSeq live_s[PT];
  __shared__ int64_t prefix_s[PT + 1];
  const bool fits = a.n <= PT;
  TreeSeq* const live_at = fits ? live_s : live_out;
  int64_t* const prefix = fits ? prefix_s : a.prefix[tab];
  __shared__ int64_t warp_cost[PT / 32];
  __shared__ int warp_live[PT / 32];
  int64_t cost = 0;
  int live = 0, rows = 0;
  bool good = true;
  for (int base = 0; base < a.n; base += PT) {
    const int s = base + tid;
    int c0 = 0, c1 = 0, len = 0;
    bool ok = true;
    if (s < a.n) {
      c0 = a.cu[s];
      c1 = a.cu[s + 1];
      len = a.lens[s];
      ok = pair_ok(a, s, c0, c1);
    }
    // the first bad offset among these
    __shared__ int first_bad;
    if (tid == 0) first_bad = INT32_MAX;
    __syncthreads();
    if (!ok) atomicMin(&first_bad, s);
    __syncthreads();
    const bool in = good && s < a.n && s < first_bad;
    const bool is_live = in && seq_kind(true, c1 - c0, len) == SEQ_LIVE;
    const int64_t v =
        is_live ? SeqCost(cut, len, (int64_t)(c1 - c0) * a.G).head() * a.nkv : 0;
    int64_t x = v;
    int y = is_live;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x1 = __shfl_up_sync(0xffffffffu, x, o);
      const int y1 = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += x1, y += y1;
    }
    if (lane == 31) warp_cost[warp] = x, warp_live[warp] = y;
    __syncthreads();
    int64_t before = cost, all = cost;
    int ybefore = live, yall = live;
    for (int w = 0; w < PT / 32; ++w) {
      if (w < warp) before += warp_cost[w], ybefore += warp_live[w];
      all += warp_cost[w];
      yall += warp_live[w];
    }
    if (is_live) {
      const int at = ybefore + y - 1;
      *reinterpret_cast<int4*>(live_out + at) = make_int4(c0, c1 - c0, len, s);
      if (fits) live_s[at] = TreeSeq{c0, c1 - c0, len, s};
      prefix[at] = before + x - v;
    }
    cost = all;
    live = yall;
    if (good) {
      const int last = min(min(first_bad, a.n), base + PT);  // sequences base .. last - 1 are good
      if (last > base) rows = a.cu[last];
      good = first_bad == INT32_MAX;
    }
    __syncthreads();
  }
  __shared__ int few, many;
  if (tid == 0) prefix[live] = cost, few = 0, many = 0;
  __syncthreads();
  if (tab == 0)  // rows of no sequence
    for (int t = rows + tid; t < a.tokens; t += PT) *reinterpret_cast<int4*>(a.token + t) = make_int4(-1, 0, 0, 0);
  int64_t chunk = quot(cost + cut.ranges - 1, cut.ranges);
  if (chunk < cut.min_chunk) chunk = cut.min_chunk;
  if (tid == 0) a.hdr[tab]->cost = cost, a.hdr[tab]->chunk = chunk, a.hdr[tab]->live = live;
  for (int c = tid; c <= cut.ranges; c += PT) {
    if (c < cut.ranges) a.counter[tab][c] = 0;
    const int64_t u = c * chunk;
    TreeStart st{cost, live, 0, 0, 0, {}, {}};
    if (u < cost) {
      int lo = 0, hi = live - 1;  // the largest i with prefix[i] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (prefix[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      const TreeSeq q = live_at[lo];
      const SeqCost k(cut, q.len, (int64_t)q.m * a.G);
      int64_t r = u - prefix[lo];
      st.h = (int)quot(r, k.head());
      r -= st.h * k.head();
      st.b = (int)min(quot(r, k.full), (int64_t)k.blocks - 1);
      const int64_t into = r - st.b * k.full;
      const bool last = st.b == k.blocks - 1;
      const int unit = last ? k.unit_last : k.unit_full;
      const int64_t t = quot(into + unit - 1, unit);
      st.at = u - into;
      st.i = lo;
      if (into == 0 || (k.units > cut.whole && t < k.units)) {
        st.t = (int)t;
        if (t > 0 && st.at >= u - chunk) {  // begun in the range before
          const int64_t end = st.at + (int64_t)(k.units - 1) * unit;
          TreeSplit sp;
          sp.c = c - 1;
          sp.parts = (int)quot(end, chunk) - c + 2;
          sp.first = 2 * (c - 1) + (u - chunk < st.at ? 1 : 0);
          sp.row = q.row;
          sp.r0 = st.b * cut.rows;
          sp.rows = (int)min((int64_t)cut.rows, (int64_t)q.m * a.G - sp.r0);
          sp.h = st.h;
          sp.len = q.len;
          // (their order changes no result)
          a.split[tab][sp.parts <= TREE_FEW ? atomicAdd(&few, 1) : cut.ranges - 1 - atomicAdd(&many, 1)] = sp;
        }
      } else {  // the item's last unit begins before: the next item
        st.at += last ? k.last : k.full;
        if (++st.b == k.blocks) {
          st.b = 0;
          if (++st.h == a.nkv) {
            st.h = 0;
            ++st.i;
          }
        }
      }
    }
    if (st.i < live) st.q = live_at[st.i];
    if (st.i + 1 < live) st.next = live_at[st.i + 1];
    a.start[tab][c] = st;
  }
  __syncthreads();
  if (tid == 0) a.hdr[tab]->few = few, a.hdr[tab]->many = many;
}

// ---------------------------------------------------------------- join
// A warp takes 32 rows of a split item, a lane each, and some of their columns. 16 loads are
// under way at a time: of 16 parts for 4 columns, or, where there are few parts, of 4 parts for
// 16 columns.
constexpr int JOIN_WARPS = 8, JOIN_BLOCKS = 2;  // warps per block, blocks per SM

template <typename T, int D, int NP, int NC>
__device__ __forceinline__ void join_rows(const TreeParams& p, const TreeSplit& sp, int r, int c0) {
  auto part = [&](int i) { return i == 0 ? sp.first : 2 * (sp.c + i); };
  const int row = min(r, sp.rows - 1);  // (lanes without a row: the last one's, not stored)
  float M = -INFINITY, L = 0.0f, x[NC][4] = {};
  for (int i0 = 0; i0 < sp.parts; i0 += NP) {
    float2 y[NP];
    float4 z[NP][NC];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      y[i] = make_float2(-INFINITY, 0.0f);
      if (i0 + i < sp.parts) {
        y[i] = __ldcg(&p.ml[(int64_t)part(i0 + i) * p.rows + row]);
#pragma unroll
        for (int c = 0; c < NC; ++c) z[i][c] = __ldcg(tree_part_at(p, part(i0 + i), D, c0 + c, row));
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) z[i][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < NP; ++i) mn = fmaxf(mn, y[i].x);
    const float base = mn == -INFINITY ? 0.0f : mn;  // (no token so far: every factor is 0)
    const float f = exp2f(M - base);
    M = mn;
    L *= f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[c][j] *= f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float w = exp2f(y[i].x - base);
      // (a part without a reference has a row sum of 0, or NaN, which stays)
      L += y[i].x > -INFINITY ? y[i].y * w : y[i].y;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c][0] = fmaf(w, z[i][c].x, x[c][0]);
        x[c][1] = fmaf(w, z[i][c].y, x[c][1]);
        x[c][2] = fmaf(w, z[i][c].z, x[c][2]);
        x[c][3] = fmaf(w, z[i][c].w, x[c][3]);
      }
    }
  }
  if (r >= sp.rows) return;
  const float inv = 1.0f / L;
  const int rr = sp.r0 + r, tok = rr / p.G, head = sp.h * p.G + rr - tok * p.G;
  T* o = static_cast<T*>(p.o) + (sp.row + tok) * p.ld_o + (int64_t)head * D + c0 * 4;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float* v = x[c];
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(o + 4 * c) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    else
      *reinterpret_cast<uint2*>(o + 4 * c) =
          make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
  }
  if (p.lse != nullptr && c0 == 0)
    p.lse[(int64_t)(sp.row + tok) * p.nq + head] = (M + log2f(L)) * LN2;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS, JOIN_BLOCKS) tree_join_kernel(const TreeParams p, int ranges) {
  // The plan is read before the attention kernel ends: that kernel let this one start only
  // when what came before it, the plan among it, was complete.
  const int groups = (p.rows + 31) / 32, step = gridDim.x * JOIN_WARPS;
  const int first = blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5);
  const int few = p.hdr->few * groups * (D / 16), all = few + p.hdr->many * groups * (D / 4);
  // task t: a split item, 32 of its rows, 16 or 4 columns
  auto item = [&](int t) {
    const int i = t < few ? t / (groups * (D / 16)) : ranges - 1 - (t - few) / (groups * (D / 4));
    return p.split[i];
  };
  int t = first;
  TreeSplit sp{};
  if (t < all) sp = item(t);
  pdl_wait();
  pdl_trigger();
  while (t < all) {
    const int u = (t < few ? t : t - few) / groups, g = (t < few ? t : t - few) - u * groups;
    const int r = g * 32 + (threadIdx.x & 31);
    if (g * 32 < sp.rows && sp.len <= p.cap) {
      if (t < few) join_rows<T, D, TREE_FEW, 4>(p, sp, r, u % (D / 16) * 4);
      else join_rows<T, D, 16, 1>(p, sp, r, u % (D / 4));
    }
    t += step;
    if (t < all) sp = item(t);
  }
}

mgb_status check_shape(int n, int tokens, int nq, int nkv, int d) {
  if (n < 0 || tokens < 0 || nq < 1 || nkv < 1 || nq % nkv || nq > (1 << 20)) return MGB_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? MGB_OK : MGB_ERR_UNSUPPORTED;
}

}  // namespace

// Rows per sequence up to which, on average, the decode step's kernel is taken, which streams
// through the caches of many short items at a time but reads a sequence again for every 16 rows.
// bf16, head dim 64, 16 heads: 64 sequences of 2000 tokens, 12 rows 93 us (by the tcgen05 kernel
// 131), 16 rows 95 (131), 24 174 (131); 200 of 100 to 600 90 (138), 94 (140), 164 (141). Head dim 128,
// 8 KV heads: 10 rows 93 (94) and 77 (80), 12 rows 92 (94) and 71 (79), but 4 to 20 rows, some of
// them read twice, 109 (96) and 86 (81). float32, 4 heads of 128, 64 of 2000: 12 rows 166
// (by the tiled kernel 213); 64 of 100 to 600 50 (46).
constexpr int few_rows(int d, int table) { return table == 0 && d == 64 ? 16 : 10; }
// .. and up to which its items have 8 rows, else 16. 8 rows each, 64 of 2000 and 200 of 100 to 600
// tokens: bf16 86.4 and 57 us at head dim 64 (as 16 rows 89 and 71), 86.6 and 54 at 128 (87.5
// and 61), float32 97 (162). 1 to 15 rows, some in two items: bf16, head dim 64, 117 and 64 (100
// and 80).
constexpr int EIGHT_ROWS = TREE_ROW_STEP;

template <typename Cut>
TreeCut cut_of() {
  return TreeCut{0, Cut::KEYS, Cut::ROWS, Cut::R1, Cut::R2, Cut::C1, Cut::C2, Cut::C3, Cut::ITEM, Cut::WHOLE,
                 Cut::C3, Cut::RANGES};
}

TreeCut tree_cut(int n, int tokens, int nq, int nkv, int d, int table) {
  const int64_t rows = (int64_t)tokens * (nq / nkv);
  if (rows <= (int64_t)few_rows(d, table) * n)
    return TreeCut{1, unit_tokens(d), rows <= (int64_t)EIGHT_ROWS * n ? EIGHT_ROWS : MAXR, MAXR,
                   MAXR, UNIT, UNIT, UNIT, tree_item_cost(d, table == 0), WHOLE, MIN_CHUNK, SMS * ctas_per_sm(d)};
  if (table == 0) return cut_of<CutTc>();
  return d == 64 ? cut_of<CutF32<64>>() : cut_of<CutF32<128>>();
}

TreeLayout tree_layout(int n, int tokens, int nq, int nkv, int d) {
  TreeLayout l;
  size_t o = 0;
  auto take = [&](size_t b) { const size_t at = o; o += (b + 255) & ~(size_t)255; return at; };
  const size_t live = n < tokens ? n : tokens;
  const int64_t most = (int64_t)tokens * (nq / nkv);
  size_t parts = 0;
  for (int i = 0; i < 2; ++i) {
    const TreeCut cut = tree_cut(n, tokens, nq, nkv, d, i);
    TreeTable& t = l.table[i];
    t.header = take(sizeof(TreeHeader));
    t.start = take(sizeof(TreeStart) * (cut.ranges + 1));
    t.split = take(sizeof(TreeSplit) * cut.ranges);
    t.live = take(sizeof(TreeSeq) * live);
    t.prefix = take(8 * (live + 1));
    t.rows = most < cut.rows ? (int)((most + TREE_ROW_STEP - 1) / TREE_ROW_STEP * TREE_ROW_STEP) : cut.rows;
    if ((size_t)2 * cut.ranges * t.rows > parts) parts = (size_t)2 * cut.ranges * t.rows;
    t.counter = take(4 * (size_t)cut.ranges);
  }
  l.seq = take(sizeof(TreeSeq) * (size_t)n);
  l.token = take(sizeof(TreeToken) * (size_t)tokens);
  l.mask = take(4 * TREE_WORDS * (size_t)tokens);
  l.ml = take(8 * parts);
  l.part = take(4 * parts * d);
  l.total = o;
  return l;
}

template <typename T, int D>
mgb_status tree_join(const TreeParams& p, int ranges, cudaStream_t st) {
  const int blocks = device_sm_count() * JOIN_BLOCKS;
  return launch_pdl(tree_join_kernel<T, D>, blocks, dim3(32 * JOIN_WARPS), 0, st, p, ranges);
}
template mgb_status tree_join<bf16, 64>(const TreeParams&, int, cudaStream_t);
template mgb_status tree_join<bf16, 128>(const TreeParams&, int, cudaStream_t);
template mgb_status tree_join<float, 64>(const TreeParams&, int, cudaStream_t);
template mgb_status tree_join<float, 128>(const TreeParams&, int, cudaStream_t);

mgb_status check_tree_plan(const mgb_attention_tree_plan* plan) {
  if (plan == nullptr || plan->ws == nullptr) return MGB_ERR_INVALID_ARG;
  const mgb_status s =
      check_shape(plan->n_seqs, plan->tokens, plan->n_q_heads, plan->n_kv_heads, plan->head_dim);
  if (s != MGB_OK) return s;
  if (!is_aligned16(plan->ws)) return MGB_ERR_MISALIGNED;
  const TreeLayout l =
      tree_layout(plan->n_seqs, plan->tokens, plan->n_q_heads, plan->n_kv_heads, plan->head_dim);
  return plan->ws_bytes < l.total ? MGB_ERR_WORKSPACE_TOO_SMALL : MGB_OK;
}

}  // namespace mgb

using namespace mgb;

extern "C" {

size_t mgb_attention_tree_ws_bytes(int32_t n_seqs, int32_t tokens, int32_t n_q_heads,
                                   int32_t n_kv_heads, int32_t head_dim) {
  if (check_shape(n_seqs, tokens, n_q_heads, n_kv_heads, head_dim) != MGB_OK) return 0;
  return tree_layout(n_seqs, tokens, n_q_heads, n_kv_heads, head_dim).total;
}

mgb_status mgb_attention_tree_prepare(int32_t n_seqs, int32_t tokens, int32_t n_q_heads,
                                      int32_t n_kv_heads, int32_t head_dim,
                                      const int32_t* cu_seqlens, const int32_t* seq_lens,
                                      const int32_t* parents, void* ws, size_t ws_bytes,
                                      mgb_attention_tree_plan* plan, void* stream) {
  if (fault_injected() || plan == nullptr) return MGB_ERR_INVALID_ARG;
  mgb_status s = check_shape(n_seqs, tokens, n_q_heads, n_kv_heads, head_dim);
  if (s != MGB_OK) return s;
  if (ws == nullptr || (n_seqs > 0 && (cu_seqlens == nullptr || seq_lens == nullptr)))
    return MGB_ERR_INVALID_ARG;
  if (!is_aligned16(ws) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) || (reinterpret_cast<uintptr_t>(parents) & 3u))
    return MGB_ERR_MISALIGNED;
  const TreeLayout l = tree_layout(n_seqs, tokens, n_q_heads, n_kv_heads, head_dim);
  if (ws_bytes < l.total) return MGB_ERR_WORKSPACE_TOO_SMALL;
  s = check_arch();
  if (s != MGB_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return MGB_ERR_CUDA;
  if (n_seqs > 0) {
    char* b = static_cast<char*>(ws);
    PlanArgs a{};
    a.n = n_seqs; a.tokens = tokens; a.G = n_q_heads / n_kv_heads; a.nkv = n_kv_heads;
    a.cu = cu_seqlens; a.lens = seq_lens; a.parents = parents;
    a.seq = reinterpret_cast<TreeSeq*>(b + l.seq);
    a.token = reinterpret_cast<TreeToken*>(b + l.token);
    a.mask = reinterpret_cast<uint32_t*>(b + l.mask);
    for (int i = 0; i < 2; ++i) {
      a.cut[i] = tree_cut(n_seqs, tokens, n_q_heads, n_kv_heads, head_dim, i);
      a.hdr[i] = reinterpret_cast<TreeHeader*>(b + l.table[i].header);
      a.start[i] = reinterpret_cast<TreeStart*>(b + l.table[i].start);
      a.split[i] = reinterpret_cast<TreeSplit*>(b + l.table[i].split);
      a.counter[i] = reinterpret_cast<uint32_t*>(b + l.table[i].counter);
      a.live[i] = reinterpret_cast<TreeSeq*>(b + l.table[i].live);
      a.prefix[i] = reinterpret_cast<int64_t*>(b + l.table[i].prefix);
    }
    a.err = err;
    const bool many = n_seqs > MANY_SEQS;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LaunchScope scope(PROF_ATTN_TREE, st, many ? 2 : 1);
    if (many) {
      a.bad = &a.hdr[0]->bad;
      tree_first_bad_kernel<<<1, BT, 0, st>>>(a);
    }
    tree_prepare_kernel<<<(unsigned)n_seqs + 2, PT, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return MGB_ERR_CUDA;
  }
  *plan = mgb_attention_tree_plan{n_seqs, tokens, n_q_heads, n_kv_heads, head_dim, ws, ws_bytes};
  return MGB_OK;
}

mgb_status mgb_attention_tree(const mgb_attention_tree_plan* plan, const mgb_kv_cache* c,
                              const void* q, int64_t ld_q, void* o, int64_t ld_o, float* lse,
                              void* stream) {
  if (fault_injected()) return MGB_ERR_INVALID_ARG;
  mgb_status s = check_tree_plan(plan);
  if (s != MGB_OK) return s;
  const int n = plan->n_seqs, nq = plan->n_q_heads, nkv = plan->n_kv_heads, d = plan->head_dim;
  s = check_kv_cache(c, n);
  if (s != MGB_OK) return s;
  if (c->n_kv_heads != nkv || c->head_dim != d || (plan->tokens > 0 && (!q || !o)))
    return MGB_ERR_INVALID_ARG;
  if (plan->tokens > 1 && (ld_q < (int64_t)nq * d || ld_o < (int64_t)nq * d)) return MGB_ERR_INVALID_ARG;
  const int vn = c->dtype == MGB_BF16 ? 8 : 4;
  if (!is_aligned16(q) || !is_aligned16(o) || ld_q % vn || ld_o % vn ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MGB_ERR_MISALIGNED;
  if (o != nullptr && o == q) return MGB_ERR_INVALID_ARG;  // the CTAs of a split item read q late
  s = check_arch();
  if (s != MGB_OK) return s;
  if (n == 0 || plan->tokens == 0) return MGB_OK;
  const TreeLayout l = tree_layout(n, plan->tokens, nq, nkv, d);
  char* b = static_cast<char*>(plan->ws);
  TreeParams p{};
  p.n = n; p.nq = nq; p.nkv = nkv; p.G = nq / nkv; p.tokens = plan->tokens;
  const int table = c->dtype == MGB_F32 ? 1 : 0;
  const bool narrow = tree_cut(n, plan->tokens, nq, nkv, d, table).narrow;
  const TreeTable& t = l.table[table];
  p.hdr = reinterpret_cast<const TreeHeader*>(b + t.header);
  p.start = reinterpret_cast<const TreeStart*>(b + t.start);
  p.split = reinterpret_cast<const TreeSplit*>(b + t.split);
  p.live = reinterpret_cast<const TreeSeq*>(b + t.live);
  p.mask = reinterpret_cast<const uint32_t*>(b + l.mask);
  p.ml = reinterpret_cast<float2*>(b + l.ml);
  p.part = reinterpret_cast<float*>(b + l.part);
  p.counter = reinterpret_cast<uint32_t*>(b + t.counter);
  p.rows = t.rows;
  p.k = c->k; p.v = c->v; p.table = c->block_table;
  p.s_page = c->stride_page; p.s_tok = c->stride_token; p.s_head = c->stride_head;
  p.ld_table = c->ld_table;
  p.n_pages = c->n_pages; p.page_size = c->page_size;
  const int64_t cap = (int64_t)c->max_pages * c->page_size;
  p.cap = cap < TREE_LONGEST ? (int)cap : TREE_LONGEST;
  p.q = q; p.ld_q = ld_q; p.o = o; p.ld_o = ld_o; p.lse = lse;
  p.sl2 = LOG2E / sqrtf((float)d);
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(PROF_ATTN_TREE, st, narrow ? 1 : 2);
  if (narrow) return attention_tree_rows(p, d, c->dtype, st);
  return c->dtype == MGB_BF16 ? attention_tree_bf16(p, d, st) : attention_tree_f32(p, d, st);
}

}  // extern "C"
