// Attention of a few query rows per sequence over a paged key/value cache: the kernel of
// the decode step (a row per query head of a KV head's group) and of small drafts (a row
// per drafted token and query head). What it does and why stands in attention_decode.cu.
#pragma once

#include "tree.cuh"

namespace mgb {

namespace {

constexpr int WARPS = 4;
constexpr int NT = WARPS * 32;
constexpr int MAXR = 16;               // query heads per item
constexpr int SMS = 152;               // of a GB300 (fewer: the same ranges, in more waves)
__host__ __device__ constexpr int ctas_per_sm(int d) { return d == 64 ? 3 : 2; }
__host__ __device__ constexpr int unit_tokens(int d) { return d == 64 ? 128 : 64; }
// fixed cost of an item (ITEM); 16 heads, 200 sequences of 20 to 600 tokens: 55.3 us
// with 4 at D = 128, 59.7 with 8, 64 with 12; D = 64, to 1200 tokens, 45 with 2, 47 with 6
__host__ __device__ constexpr int item_cost(int d) { return d == 64 ? 2 : 4; }
constexpr int UNIT = 4;                // cost of a unit
// .. of an item of drafted tokens. bf16, head dim 64, 16 heads, 96 sequences of 20 to 1200
// tokens: 38.3 us with 2, 33.6 with 4, 31.9 with 8, 32.6 with 12; head dim 128 75, 65, 55.9 and
// 56.4 with 4, 6, 10 and 16, and 32 query and 8 KV heads, 64 of 33 to 4000 69.6, 60.8, 54.1,
// 52.4 and 54.4 with 4, 6, 10, 12 and 16. float32, whose products take longer: 47.6, 52.5 and 50.5
// with 2, 4 and 6 (96 of 20 to 600, head dim 64), 71.4, 68.3, 69.3 and 72.2 with 2, 4, 6 and 8 (128).
__host__ __device__ constexpr int tree_item_cost(int d, bool bf) {
  return !bf ? item_cost(d) : d == 64 ? 8 : 12;
}
constexpr int PARTS = 16;              // of a split item, joined at a time (at most 32)
constexpr int WHOLE = 4;               // units of an item that is never split
constexpr int MIN_CHUNK = 2 * UNIT;    // of a CTA (at least UNIT: no CTA between two others is empty)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float TAU = 8.0f;            // the reference maximum moves in steps above this (log2 units)

struct Header {
  int64_t cost;  // of all items
  int64_t chunk;
};
struct Start {
  int64_t at;       // where the item of the CTA's first unit begins on the cost axis
  int32_t s, h, t;  // the unit: sequence, head group, token tile
  int32_t len, next_len, pad;  // lengths of sequences s and s + 1
};

// where unit t of an item with n units begins on its part of the cost axis
__host__ __device__ inline int64_t begin_of(int t, int n) { return n > WHOLE ? (int64_t)t * UNIT : 0; }
__host__ __device__ inline int64_t cost_of(int tiles, int item) { return (int64_t)tiles * UNIT + item; }
// units of a sequence: at least one, so that an empty one gets its zeros
__host__ __device__ inline int tiles_of(int len, int tk) {
  return len > tk ? (int)(((int64_t)len + tk - 1) / tk) : 1;
}

// ---------------------------------------------------------------- main kernel
// (drafted tokens: the units of a plan, in tree.cuh's terms: `n` and a sequence's groups come
// from the device)
struct Params {
  int n, nkv, groups, per_kv, rows, G;  // head groups per sequence / per KV head, rows per group
  const Header* hdr;
  const Start* start;
  const TreeHeader* thdr;
  const TreeStart* tstart;
  const TreeSeq* live;
  const uint32_t* mask;
  uint32_t* counter;
  const int32_t* len;
  float2* ml;    // [2 CTAs][rows] (maximum, row sum) of a part
  float* part;   // [2 CTAs][rows][d]
  const void *k, *v;
  const int32_t* table;
  int64_t s_page, s_tok, s_head, ld_table;
  int n_pages, page_size;
  int cap;       // tokens a row of the table holds
  const void* q;
  int64_t ld_q;
  void* o;
  int64_t ld_o;
  float* lse;
  int nq;
  float sl2;     // log2(e) / sqrt(d)
  int* err;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit values, row lane / 4, columns 2 (lane % 4) + {0, 1} -> its transpose
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Position in a CTA's range of units of TK tokens. TREE: of drafted tokens.
template <typename T, int D, bool TREE>
struct Cursor {
  static constexpr int TK = unit_tokens(D), ITEM = TREE ? tree_item_cost(D, sizeof(T) == 2) : item_cost(D);
  int64_t at;  // the item on the cost axis
  int s, h, t, nt, len, next_len;
  TreeSeq q, nq;  // TREE: sequences s and s + 1 of the plan's
  int n, per;     // TREE: sequences; groups of rows per KV head
  __device__ void init(const Start& st) {
    at = st.at; s = st.s; h = st.h; t = st.t; len = st.len; next_len = st.next_len;
    nt = tiles_of(len, TK);
  }
  __device__ void init(const Params& p, const TreeStart& st, int live) {
    at = st.at; s = st.i; t = st.t; n = live;
    q = st.q;
    nq = st.next;
    take(p);
    h = st.h * per + st.b;
  }
  __device__ void take(const Params& p) {
    len = q.len;
    nt = tiles_of(len, TK);
    per = (q.m * p.G + p.rows - 1) / p.rows;
  }
  __device__ void request(const Params& p) {
    if (s + 1 < n) {
      const int4 x = *reinterpret_cast<const int4*>(p.live + s + 1);
      nq = TreeSeq{x.x, x.y, x.z, x.w};
    }
  }
  __device__ int per_kv(const Params& p) const { return TREE ? per : p.per_kv; }
  __device__ int group_rows(const Params& p) const {  // rows from the group's first one on
    const int first = (h % per_kv(p)) * p.rows;
    return (TREE ? q.m * p.G : p.G) - first;
  }
  // to the next unit; the next sequence's length was requested one sequence ago. A
  // length past the table counts as 0, and its units behind the first one looked
  // at are passed over, however many they are
  __device__ void next(const Params& p) {
    if (len <= p.cap && ++t < nt) return;
    t = 0;
    at += cost_of(nt, ITEM);
    if (++h < (TREE ? per * p.nkv : p.groups)) return;
    h = 0;
    ++s;
    if constexpr (TREE) {
      q = nq;
      take(p);
      request(p);
    } else {
      len = next_len;
      nt = tiles_of(len, TK);
      next_len = s + 1 < p.n ? p.len[s + 1] : 0;
    }
  }
  __device__ bool before(int64_t end) const { return at + begin_of(t, nt) < end; }
};

template <typename T, int D, int NR>
struct Cfg {
  static constexpr int ES = sizeof(T);
  static constexpr int TK = unit_tokens(D);
  static constexpr int SK = 4096 / (D * ES);         // tokens per warp and stage: 4 KB of keys
  static constexpr int SUB = TK / (WARPS * SK);      // stages per unit
  static constexpr uint32_t ALL = SK == 32 ? ~0u : (1u << SK) - 1u;  // a bit per token of a stage
  static constexpr int ROW = D * ES;                 // bytes of a token's vector
  static constexpr int CH = ROW / 16;                // 16-byte chunks of it
  static constexpr int KV = SK * ROW;                // bytes of a stage's keys (or values)
  static constexpr int STAGES = D == 128 ? 3 : 2;
  static constexpr int RING = STAGES * 2 * KV;       // per warp
  static constexpr int MR = ES == 2 ? 8 : 4;         // rows joined at a time
  static constexpr int JS = D + 4;                   // row stride of the join buffer (floats)
  static constexpr int OFF_JOIN = WARPS * RING;      // [WARPS][MR][JS] float
  static constexpr int OFF_Q = OFF_JOIN + WARPS * MR * JS * 4;  // float32: [NR][D]
  static constexpr int OFF_ML = OFF_Q + (ES == 4 ? NR * D * 4 : 0);  // [WARPS][MAXR] float2
  static constexpr int SMEM = OFF_ML + WARPS * MAXR * 8;
  static_assert((SMEM + 1024) * ctas_per_sm(D) <= 228 * 1024, "CTAs per SM");
};

// Shared-memory offset of chunk c of a stage's token row (rotated by the row
// so that eight rows' same chunk fall into different banks).
template <int CH>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return (uint32_t)(row * CH + (c ^ (row & 7))) * 16u;
}

// NR: rows per item at most, a row being a query head of a KV head's group, or (TREE) one of
// a drafted token
template <typename T, int D, int NR, bool TREE>
__global__ void __launch_bounds__(NT, ctas_per_sm(D)) paged_rows_kernel(const Params p) {
  using C = Cfg<T, D, NR>;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int ST = C::STAGES, TK = C::TK;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  pdl_wait();  // everything the call reads may come from the kernel before
  Header hd;
  Cursor<T, D, TREE> ld, cu;
  int64_t end;
  if constexpr (TREE) {
    const TreeHeader th = *p.thdr;
    const TreeStart st0 = p.tstart[c];
    hd = Header{th.cost, th.chunk};
    end = min((int64_t)(c + 1) * hd.chunk, hd.cost);
    if (st0.i >= th.live || st0.at + (int64_t)st0.t * UNIT >= end) return;  // no unit begins in the range
    ld.init(p, st0, th.live);
  } else {
    hd = *p.hdr;
    const Start st0 = p.start[c];
    end = min((int64_t)(c + 1) * hd.chunk, hd.cost);
    if (st0.s >= p.n || st0.at + (int64_t)st0.t * UNIT >= end) return;  // no unit begins in the range
    ld.init(st0);
  }
  cu = ld;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  float* join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
  float* sq = reinterpret_cast<float*>(smem + C::OFF_Q);
  float2* sml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  int* flag = reinterpret_cast<int*>(sml);  // once sml is read

  // ---------------- loader: a cursor one stage ahead of the copies, whose
  // page number is in flight while the previous stage's copies are issued
  int ld_sub = 0, ld_n = 0;
  int pg = 0, slot = 0, hkv = 0;
  bool on = false, look = false;
  // which tokens of the ST stages fetched last are to be seen, the oldest first
  uint32_t seen[ST] = {};
  auto peek = [&]() {  // request the page of this lane's token of the next stage
    on = false;
    look = ld.before(end);
    if (!look) return;
    const int key = ld.t * TK + ld_sub * (WARPS * C::SK) + warp * C::SK + (lane % C::SK);
    hkv = ld.h / ld.per_kv(p);
    on = key < ld.len && ld.len <= p.cap;
    if (on) {
      const int i = key / p.page_size;
      slot = key - i * p.page_size;
      pg = p.table[(TREE ? ld.q.s : ld.s) * p.ld_table + i];
    }
    if (++ld_sub == C::SUB) {
      ld_sub = 0;
      ld.next(p);
    }
  };
  auto fetch = [&]() {  // copy the stage the last peek looked at, then peek
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) seen[i] = seen[i + 1];
    seen[ST - 1] = 0;
    if (look) {
      bool ok = on && pg >= 0 && pg < p.n_pages;
      if (on && !ok) record_error(p.err, kErrIndex);
      seen[ST - 1] = __ballot_sync(0xffffffffu, ok) & C::ALL;
      const int64_t off = ok ? pg * p.s_page + slot * p.s_tok + hkv * p.s_head : -1;
      const uint32_t dst = ring + (ld_n % ST) * 2 * C::KV;
      if (seen[ST - 1] != 0) {
#pragma unroll
        for (int i = 0; i < C::SK * C::CH / 32; ++i) {
          const int row = (i * 32 + lane) / C::CH, ch = (i * 32 + lane) % C::CH;
          const int64_t ro = __shfl_sync(0xffffffffu, off, row);
          const T* ks = static_cast<const T*>(p.k) + (ro >= 0 ? ro : 0) + ch * (16 / C::ES);
          const T* vs = static_cast<const T*>(p.v) + (ro >= 0 ? ro : 0) + ch * (16 / C::ES);
          const uint32_t at = dst + chunk_at<C::CH>(row, ch);
          cp_async16(at, ks, ro >= 0);
          cp_async16(at + C::KV, vs, ro >= 0);
        }
      }
    }
    cp_async_commit();
    ++ld_n;
    peek();
  };
  peek();
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) fetch();

  // ---------------- queries: the next item's are requested one item ahead
  // row r of the cursor's group: its offset in q (or, with the strides of o, in o), or -1
  auto row_at = [&](const Cursor<T, D, TREE>& x, int r, int64_t ld_row) -> int64_t {
    const int per = x.per_kv(p), kv = x.h / per, first = (x.h - kv * per) * p.rows + r;
    if constexpr (TREE) {
      if (r >= p.rows || first >= x.q.m * p.G) return -1;
      const int tok = first / p.G;
      return (x.q.row + tok) * ld_row + (int64_t)(kv * p.G + first - tok * p.G) * D;
    } else {
      return r < p.rows && first < p.G ? x.s * ld_row + (int64_t)(kv * p.G + first) * D : -1;
    }
  };
  constexpr int HT = BF ? NR / 8 : 1;  // bf16: tiles of 8 query heads
  constexpr int NQ = BF ? D / 16 * 2 * HT : (NR * D / 4 + NT - 1) / NT * 4;
  uint32_t qn[NQ];
  auto request_q = [&](const Cursor<T, D, TREE>& at) {
    const T* qs = static_cast<const T*>(p.q);
    if constexpr (BF) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const int64_t row = row_at(at, (lane >> 2) + 8 * ht, p.ld_q);
        const T* x = qs + (row < 0 ? 0 : row) + (lane & 3) * 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qn[(kk * HT + ht) * 2] = row < 0 ? 0u : *reinterpret_cast<const uint32_t*>(x + kk * 16);
          qn[(kk * HT + ht) * 2 + 1] =
              row < 0 ? 0u : *reinterpret_cast<const uint32_t*>(x + kk * 16 + 8);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NQ / 4; ++i) {
        const int e = (i * NT + tid) * 4;
        const int64_t row = e < NR * D ? row_at(at, e / D, p.ld_q) : -1;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) x = *reinterpret_cast<const float4*>(qs + row + e % D);
        qn[4 * i] = __float_as_uint(x.x);
        qn[4 * i + 1] = __float_as_uint(x.y);
        qn[4 * i + 2] = __float_as_uint(x.z);
        qn[4 * i + 3] = __float_as_uint(x.w);
      }
    }
  };
  request_q(cu);

  int n_use = 0;  // stages consumed
  while (cu.before(end)) {
    const Cursor<T, D, TREE> it = cu;  // the item
    const int nt = cu.nt, t0 = cu.t;
    const int len = cu.len <= p.cap ? cu.len : 0;
    if (cu.len > p.cap && tid == 0) record_error(p.err, kErrIndex);
    const int64_t at = cu.at;
    const int rows = min(p.rows, cu.group_rows(p));
    uint32_t qa[BF ? NQ : 1];
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) qa[i] = qn[i];
    } else {
#pragma unroll
      for (int i = 0; i < NQ / 4; ++i)
        if ((i * NT + tid) * 4 < NR * D) *reinterpret_cast<float4*>(sq + (i * NT + tid) * 4) =
            make_float4(__uint_as_float(qn[4 * i]), __uint_as_float(qn[4 * i + 1]),
                        __uint_as_float(qn[4 * i + 2]), __uint_as_float(qn[4 * i + 3]));
      __syncthreads();
    }
    {  // the next item's queries
      Cursor<T, D, TREE> nx = cu;
      nx.t = nx.nt - 1;
      nx.next(p);
      if (nx.before(end) && (!TREE || nx.s < nx.n)) request_q(nx);
    }

    // bf16: acc[i] holds d = 16 (i / HT) + lane / 4 (+ 8 in the upper two) of
    // heads 8 (i % HT) + 2 (lane % 4) + {0, 1}; m, l those heads' (l of the
    // lane's tokens only). float32: acc all rows, columns lane * (D / 32) ..; m, l
    // rows 4 i + lane / 8 (l of the lane's tokens only)
    constexpr int CPL = D / 32;
    constexpr int NO = BF ? D / 16 * HT : NR;
    constexpr int NI = BF ? 4 : CPL;
    constexpr int NM = BF ? 2 * HT : NR / 4;
    float acc[NO][NI], m[NM], l[NM];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < NM; ++i) m[i] = -INFINITY, l[i] = 0.0f;

    for (bool more = true; more;) {
#pragma unroll
      for (int sub = 0; sub < C::SUB; ++sub) {
        cp_async_wait<ST - 2>();
        __syncwarp();  // the stage is complete and the one before it no longer read
        fetch();
        const uint32_t sk = ring + (n_use % ST) * 2 * C::KV, sv = sk + C::KV;
        ++n_use;
        const uint32_t see = seen[0];  // the slice's visible tokens
        if (see == 0) continue;
        // TREE: whether row r sees the slice's token k, and whether some token may be hidden
        const int drafted = TREE ? cu.t * TK + sub * (WARPS * C::SK) + warp * C::SK - (it.q.len - it.q.m) : 0;
        const bool hides = TREE && drafted + C::SK > 0;
        auto sees = [&](int r, int k) {
          const int d = drafted + k;
          if (d < 0 || r >= rows) return true;
          const int tok = ((it.h % it.per) * p.rows + r) / p.G;
          return ((p.mask[(int64_t)(it.q.row + tok) * TREE_WORDS + (d >> 5)] >> (d & 31)) & 1u) != 0;
        };
        if constexpr (BF) {
          // sc[mt][ht]: token 16 mt + lane / 4 (+ 8 in the upper two), heads 8 ht +
          // 2 (lane % 4) + {0, 1}
          constexpr int MT = C::SK / 16;
          float sc[MT][HT][4] = {};
          const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a[4];
              ldsm4(sk + chunk_at<C::CH>(16 * mt + (mi & 1) * 8 + r8, 2 * kk + (mi >> 1)), a);
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
                mma_bf16(sc[mt][ht], a, qa[(kk * HT + ht) * 2], qa[(kk * HT + ht) * 2 + 1]);
            }
          if (see != C::ALL) {
            const uint32_t sl = see >> (lane >> 2);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!((sl >> (16 * mt + (e >> 1) * 8)) & 1u)) sc[mt][ht][e] = -INFINITY;
          }
          if (TREE && hides) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int k = 16 * mt + (lane >> 2) + (e >> 1) * 8;
                  if (((see >> k) & 1u) && !sees(8 * ht + 2 * (lane & 3) + (e & 1), k)) sc[mt][ht][e] = -INFINITY;
                }
          }
          bool up[NM], any = false;
          float mx[NM];
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            float x = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              // scaled before the maximum and before it is subtracted: one rounding for
              // both, so that the largest weight is 1 for scores of any size (a fused
              // x sl2 - m is off by the product's rounding, powers of 2 past 2^24)
              float &a = sc[mt][i / 2][i & 1], &b = sc[mt][i / 2][2 + (i & 1)];
              a = __fmul_rn(a, p.sl2);
              b = __fmul_rn(b, p.sl2);
              x = fmax3(x, a, b);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            mx[i] = x;
            up[i] = mx[i] > m[i] + TAU;
            any |= up[i];
          }
          // the reference moves only when it must: P stays below 2^TAU
          if (__any_sync(0xffffffffu, any)) {
#pragma unroll
            for (int i = 0; i < NM; ++i) {
              const float a = up[i] ? exp2f(m[i] - mx[i]) : 1.0f;
              if (up[i]) m[i] = mx[i];
              l[i] *= a;
#pragma unroll
              for (int nn = 0; nn < D / 16; ++nn) {
                acc[nn * HT + i / 2][i & 1] *= a;
                acc[nn * HT + i / 2][2 + (i & 1)] *= a;
              }
            }
          }
          // P in two bf16 parts, the second what the first leaves: a weight is off by
          // 2^-16 relative at most. (Rounded to one part, 2^-8, the weights' errors shrink
          // in the average over the tokens exactly as the result does, so they add as
          // much again as the output's own rounding.)
          uint32_t pb[MT][HT][2], pl[MT][HT][2];
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) {
            const float r0 = m[2 * ht] == -INFINITY ? 0.0f : m[2 * ht];
            const float r1 = m[2 * ht + 1] == -INFINITY ? 0.0f : m[2 * ht + 1];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float(&x)[4] = sc[mt][ht];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = ex2_ftz(x[e] - ((e & 1) ? r1 : r0));
              l[2 * ht] += x[0] + x[2];
              l[2 * ht + 1] += x[1] + x[3];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t hi = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                const float2 f = unpack_bf16x2(hi);
                pb[mt][ht][i] = transpose8x8(hi);
                pl[mt][ht][i] = transpose8x8(pack_bf16x2(x[2 * i] - f.x, x[2 * i + 1] - f.y));
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nn = 0; nn < D / 16; ++nn) {
              uint32_t a[4];
              ldsm4_t(sv + chunk_at<C::CH>(16 * mt + (mi >> 1) * 8 + r8, 2 * nn + (mi & 1)), a);
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
                mma_bf16(acc[nn * HT + ht], a, pb[mt][ht][0], pb[mt][ht][1]);
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
                mma_bf16(acc[nn * HT + ht], a, pl[mt][ht][0], pl[mt][ht][1]);
            }
        } else {
          // no branch on `rows`: heads that do not exist have zero queries, and
          // NR independent chains hide what four dependent ones did not
          const int key = lane & 7, part = lane >> 3;  // token, quarter of d
          float* sp = join + warp * 8 * NR;  // [token][head] (join is free until the item's end)
#pragma unroll
          for (int kt = 0; kt < C::SK / 8; ++kt) {  // eight tokens at a time
            if ((see >> (8 * kt)) == 0) break;
            float d0[NR] = {}, d1[NR] = {};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              float4 kx;
              asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                           : "=f"(kx.x), "=f"(kx.y), "=f"(kx.z), "=f"(kx.w)
                           : "r"(sk + chunk_at<C::CH>(8 * kt + key, i * 4 + part)));
#pragma unroll
              for (int r = 0; r < NR; ++r) {
                const float4 qx = *reinterpret_cast<const float4*>(sq + r * D + (i * 4 + part) * 4);
                fma2(d0[r], d1[r], qx.x, qx.y, kx.x, kx.y, d0[r], d1[r]);
                fma2(d0[r], d1[r], qx.z, qx.w, kx.z, kx.w, d0[r], d1[r]);
              }
            }
            // sums over the quarters, dealt out: this lane gets heads 4 i + part
            float pr[NM], mx[NM];
            bool up[NM], any = false;
#pragma unroll
            for (int i = 0; i < NM; ++i) {
              float x[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) x[r] = d0[4 * i + r] + d1[4 * i + r];
              const bool hi = part & 2, odd = part & 1;
              const float y0 = (hi ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, hi ? x[0] : x[2], 16);
              const float y1 = (hi ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, hi ? x[1] : x[3], 16);
              const float sc = (odd ? y1 : y0) + __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 8);
              pr[i] = (see >> (8 * kt + key)) & 1u ? __fmul_rn(sc, p.sl2) : -INFINITY;
              if (TREE && hides && ((see >> (8 * kt + key)) & 1u) && !sees(4 * i + part, 8 * kt + key))
                pr[i] = -INFINITY;
              mx[i] = pr[i];
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
              for (int i = 0; i < NM; ++i)
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
#pragma unroll
            for (int i = 0; i < NM; ++i) {
              up[i] = mx[i] > m[i] + TAU;
              any |= up[i];
            }
            if (__any_sync(0xffffffffu, any)) {
              float a[NM];
#pragma unroll
              for (int i = 0; i < NM; ++i) {
                a[i] = up[i] ? exp2f(m[i] - mx[i]) : 1.0f;
                if (up[i]) m[i] = mx[i];
                l[i] *= a[i];
              }
#pragma unroll
              for (int r = 0; r < NR; ++r) {
                const float f = __shfl_sync(0xffffffffu, a[r / 4], (r % 4) * 8);
#pragma unroll
                for (int j = 0; j < CPL; ++j) acc[r][j] *= f;
              }
            }
            __syncwarp();  // the weights before are read
#pragma unroll
            for (int i = 0; i < NM; ++i) {
              pr[i] = ex2_ftz(pr[i] - (m[i] == -INFINITY ? 0.0f : m[i]));
              l[i] += pr[i];
              sp[key * NR + 4 * i + part] = pr[i];
            }
            __syncwarp();
#pragma unroll
            for (int kx2 = 0; kx2 < 8; ++kx2) {
              float vx[CPL];
              const uint32_t va = sv + chunk_at<C::CH>(8 * kt + kx2, lane * CPL / 4) + (lane * CPL % 4) * 4;
              if constexpr (CPL == 4)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(vx[0]), "=f"(vx[1]), "=f"(vx[2]), "=f"(vx[3])
                             : "r"(va));
              else
                asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(vx[0]), "=f"(vx[1]) : "r"(va));
#pragma unroll
              for (int i = 0; i < NM; ++i) {
                const float4 w4 = *reinterpret_cast<const float4*>(sp + kx2 * NR + 4 * i);
                const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                  for (int j = 0; j < CPL; j += 2)
                    fma2(acc[4 * i + r][j], acc[4 * i + r][j + 1], w[r], w[r], vx[j], vx[j + 1],
                         acc[4 * i + r][j], acc[4 * i + r][j + 1]);
              }
            }
          }
        }
      }
      cu.next(p);
      more = cu.at == at && cu.before(end);
    }

    if (len == 0 && (TREE || t0 != 0)) {
      __syncthreads();  // (sq is free)
      continue;  // the CTA with the first unit of a length past the table stores its zeros (TREE: none)
    }
    // ---------------- the item's units in this CTA are done: join the warps
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < NM; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (lane < 4) sml[warp * MAXR + 8 * (i / 2) + 2 * lane + (i & 1)] = make_float2(m[i], l[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NM; ++i) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if ((lane & 7) == 0) sml[warp * MAXR + 4 * i + (lane >> 3)] = make_float2(m[i], l[i]);
      }
    }
    __syncthreads();
    auto joined = [&](int r, float& M, float& L) {
      M = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sml[w * MAXR + r].x);
      L = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        // (no reference: no token or only scores of -infinity, 0, or NaN, which stays)
        const float2 x = sml[w * MAXR + r];
        L += x.x > -INFINITY ? x.y * exp2f(x.x - M) : x.y;
      }
    };
    // first and last CTA of the item
    const int64_t last = at + begin_of(nt - 1, nt);
    const bool whole = len == 0 || (at >= (int64_t)c * hd.chunk && last < end);
    const int cf = whole ? c : (int)(at / hd.chunk), cl = whole ? c : (int)(last / hd.chunk);
    // part 2 c: the CTA's range begins at or inside the item; 2 c + 1: before it
    auto part_of = [&](int cc) { return 2 * cc + ((int64_t)cc * hd.chunk < at ? 1 : 0); };
    const int my = part_of(c);
    auto lse_at = [&](int r) {  // (in units of heads)
      const int per = it.per_kv(p), kv = it.h / per, first = (it.h - kv * per) * p.rows + r;
      if constexpr (TREE) return (int64_t)(it.q.row + first / p.G) * p.nq + kv * p.G + first % p.G;
      else return (int64_t)it.s * p.nq + kv * p.G + first;
    };
    auto store_o = [&](int r, int col, float4 x) {
      T* o = static_cast<T*>(p.o) + row_at(it, r, p.ld_o) + col;
      if constexpr (BF)
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      else
        *reinterpret_cast<float4*>(o) = x;
    };
#pragma unroll
    for (int r0 = 0; r0 < NR; r0 += C::MR) {
      if (r0 >= rows) break;
      if (r0 > 0) __syncthreads();
      if constexpr (BF) {
        const int ht = r0 / 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * (lane & 3) + i;
          if (r0 + r >= rows) continue;
          float M, L;
          joined(r0 + r, M, L);
          const float mm = m[2 * ht + i], a = mm > -INFINITY ? exp2f(mm - M) : 0.0f;
          float* x = join + (warp * C::MR + r) * C::JS + (lane >> 2);
#pragma unroll
          for (int nn = 0; nn < D / 16; ++nn) {
            x[16 * nn] = acc[nn * HT + ht][i] * a;
            x[16 * nn + 8] = acc[nn * HT + ht][2 + i] * a;
          }
        }
      } else {
#pragma unroll
        for (int rr = 0; rr < C::MR; ++rr) {
          const int r = r0 + rr;
          if (r >= rows) continue;
          float M, L;
          joined(r, M, L);
          const float mr = sml[warp * MAXR + r].x; const float a = mr > -INFINITY ? exp2f(mr - M) : 0.0f;
#pragma unroll
          for (int j = 0; j < CPL; ++j)
            join[(warp * C::MR + rr) * C::JS + lane * CPL + j] = acc[r][j] * a;
        }
      }
      __syncthreads();
      for (int e = tid * 4; e < C::MR * D; e += NT * 4) {
        const int r = r0 + e / D, col = e % D;
        if (r >= rows) break;
        const float* jr = join + (r - r0) * C::JS + col;
        float4 x = *reinterpret_cast<const float4*>(jr);
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(jr + w * C::MR * C::JS);
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        float M, L;
        joined(r, M, L);
        if (whole) {
          const float inv = len > 0 ? 1.0f / L : 0.0f;  // (no token left: 0 / 0)
          store_o(r, col, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
          if (p.lse != nullptr && col == 0)
            p.lse[lse_at(r)] = (M + log2f(L)) * LN2;
        } else {
          *reinterpret_cast<float4*>(p.part + ((int64_t)my * p.rows + r) * D + col) = x;
          if (col == 0) p.ml[(int64_t)my * p.rows + r] = make_float2(M, L);
        }
      }
    }
    if (!whole) {
      // ---- split item: the last CTA to arrive joins the parts in CTA order
      __syncthreads();  // the part is written; thread 0's release covers all of it
      if (tid == 0) {
        uint32_t before;  // acquire and release: the parts before and behind the arrivals
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                     : "=r"(before)
                     : "l"(p.counter + cf), "r"((uint32_t)(cl - cf))
                     : "memory");
        *flag = before == (uint32_t)(cl - cf);
      }
      __syncthreads();
      if (*flag) {
        for (int r = warp; r < rows; r += WARPS) {
          float M = -INFINITY, L = 0.0f, x[CPL] = {};
          for (int cc0 = cf; cc0 <= cl; cc0 += PARTS) {  // PARTS parts requested together
            float z[PARTS][CPL];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
              const int cc = cc0 + i;
#pragma unroll
              for (int j = 0; j < CPL; ++j) z[i][j] = 0.0f;
              if (cc <= cl) {
                const float* y = p.part + ((int64_t)part_of(cc) * p.rows + r) * D + lane * CPL;
                if constexpr (CPL == 4) {
                  const float4 zz = __ldcg(reinterpret_cast<const float4*>(y));
                  z[i][0] = zz.x; z[i][1] = zz.y; z[i][2] = zz.z; z[i][3] = zz.w;
                } else {
                  const float2 zz = __ldcg(reinterpret_cast<const float2*>(y));
                  z[i][0] = zz.x; z[i][1] = zz.y;
                }
              }
            }
            float2 y = make_float2(-INFINITY, 0.0f);  // of part cc0 + lane
            if (lane < PARTS && cc0 + lane <= cl)
              y = __ldcg(&p.ml[(int64_t)part_of(cc0 + lane) * p.rows + r]);
            float mn = y.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mn = fmaxf(mn, M);
            const float base = mn == -INFINITY ? 0.0f : mn;  // (no token so far: every factor is 0)
            const float f = exp2f(M - base), a = exp2f(y.x - base);
            M = mn;
            float lp = y.y * a;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lp += __shfl_xor_sync(0xffffffffu, lp, o);
            L = L * f + lp;
#pragma unroll
            for (int j = 0; j < CPL; ++j) x[j] *= f;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
              const float w = __shfl_sync(0xffffffffu, a, i);
#pragma unroll
              for (int j = 0; j < CPL; ++j) x[j] = fmaf(w, z[i][j], x[j]);
            }
          }
          const float inv = 1.0f / L;
          T* o = static_cast<T*>(p.o) + row_at(it, r, p.ld_o) + lane * CPL;
#pragma unroll
          for (int j = 0; j < CPL; ++j) o[j] = from_f<T>(x[j] * inv);
          if (p.lse != nullptr && lane == 0)
            p.lse[lse_at(r)] = (M + log2f(L)) * LN2;
        }
      }
    }
    __syncthreads();  // the join buffer, sml and sq are free for the next item
  }
  cp_async_wait<0>();
}

}  // namespace
}  // namespace mgb
