// Attention of drafted tokens over a paged cache, bf16, on the tensor cores
// (tcgen05): o = softmax(q K^T / sqrt(d)) V over the cached tokens that a drafted
// token sees, all those before the draft, its ancestors in the tree and itself.
//
// An item's rows are the drafted tokens times the query heads of one KV head, in
// two tiles A and B of 128 (B may be empty). Per 128 keys: S = Q K^T (TMEM), the
// softmax threads (one per row) turn the scores into weights P in place, and O += P V
// with P read from TMEM. Rows share all keys but the drafted ones, so K and V pass
// once through shared memory for up to 256 rows: with few rows HBM is the bound, with
// 256 the tensor core (3072 cycles per 128 keys) comes near it (2800 at 6.7 TB/s).
//
// P multiplies V as the sum of two bf16 parts (off by 2^-16 relative at most): with one
// part the weights' errors would add as much again as the output's own rounding. The
// parts of 16 keys take the 16 columns that their scores had.
//
// K and V come through a ring of slots of 128 keys by 16-byte asynchronous copies of
// four warps, a row per cached token, so any page size and layout works and tokens
// behind the length or of a bad page are never read. The order is K_0, K_1, V_0, K_2,
// V_1, ..: what the products need next.
#include "tree.cuh"

namespace mgb {

namespace {

constexpr int TQ = 128;         // rows per tile (TMEM lanes)
constexpr int TK = TREE_KEYS;   // keys per slot
constexpr int NLOAD = 128;      // producer threads
constexpr int NTHREADS = 32 + NLOAD + 256;  // MMA warp, producers, softmax of A and B
constexpr float LN2 = 0.6931471805599453f;
constexpr float TAU = 8.0f;     // the reference maximum moves in steps above this (log2 units)

template <int D>
struct Cfg {
  static constexpr int NST = D == 64 ? 10 : 5;          // ring slots
  static constexpr int KB = D / 64;                     // 64-wide d boxes
  static constexpr int BOX = 128 * 128;                 // bytes of one [128][64] box
  static constexpr int CH = D / 8;                      // 16-byte chunks of a row
  static constexpr int Q_BYTES = TQ * D * 2;
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int OFF_Q = 0;                       // [tile]
  static constexpr int OFF_R = 2 * Q_BYTES;             // [slot]
  static constexpr int OFF_SEE = OFF_R + NST * KV_BYTES;  // [NSEE][4]: a bit per key that may be seen
  static constexpr int NSEE = 16;
  static constexpr int OFF_BAR = OFF_SEE + NSEE * 16;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;     // barriers, alignment slack
  static constexpr int COL_S = 0;                       // two score buffers
  static constexpr int COL_O = 2 * TK;                  // O_A, then O_B at + D
  static constexpr int TMEM_COLS = 512;
  static_assert(COL_O + 2 * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  // Barriers (8 bytes each). A waiter sees every phase of a barrier, or knows that at
  // most one is outstanding (parity).
  static constexpr int Q_FULL = 0;              // the item's queries copied     (every producer)
  static constexpr int Q_EMPTY = 1;             // the item's last S done        (commit)
  static constexpr int L_FULL = 2;              // [slot] copied                 (every producer)
  static constexpr int L_EMPTY = L_FULL + NST;  // [slot] its products done      (commit)
  static constexpr int S_FULL = L_EMPTY + NST;  // [tile][task & 1] scores       (commit)
  static constexpr int P_FULL = S_FULL + 4;     // [tile][task & 1] weights      (4: one per warp)
  static constexpr int PV_DONE = P_FULL + 4;    // [tile] a task's PV            (commit)
  static constexpr int O_EMPTY = PV_DONE + 2;   // [tile] O read out             (4: one per warp)
  static constexpr int SEE = O_EMPTY + 2;       // [key tile % NSEE] bits there  (4: one per producer warp)
  static constexpr int N_BAR = SEE + NSEE;
  static_assert(N_BAR * 8 <= 480, "barriers");
};

// The slot a key tile's K or V has in the item's order K_0, K_1, V_0, K_2, V_1, ..
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * n - 1; }

// One thread: waits for the phase, for a bounded time and only while no role has given up.
__device__ __forceinline__ bool wait_1(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort != 0) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      record_error(err, kErrTimeout);
      return false;
    }
  }
}
// The same for a whole warp, which goes on together.
__device__ __forceinline__ bool wait_w(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    const bool ok = mbar_try_wait_suspend(bar, parity, 50000u);
    if (__all_sync(0xffffffffu, ok)) return true;
    const bool late = global_ns() - t0 > kWaitLimitNs;
    if (late) record_error(err, kErrTimeout);
    if (__any_sync(0xffffffffu, late || *abort != 0)) return false;
  }
}

// The barrier counts one arrival of this thread when its copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) tree_kernel(const TreeParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t sQ = sb + C::OFF_Q, sR = sb + C::OFF_R;
  constexpr int NST = C::NST;
  auto bar = [&](int which) { return sb + C::OFF_BAR + 8 * which; };
  volatile uint32_t* see = reinterpret_cast<uint32_t*>(smem + C::OFF_SEE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 496);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 500);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();     // everything the call reads may come from the kernel before
  pdl_trigger();  // the join may start up; it waits for this kernel's end
  const int c = blockIdx.x;
  const TreeHeader hd = *p.hdr;
  const TreeStart st = p.start[2 * c];
  const int64_t chunk = 2 * hd.chunk, end = min((c + 1) * chunk, hd.cost);
  TreeSegs sg;
  if (!sg.begin(p, hd, st, end) || st.at + (int64_t)st.t * TREE_UNIT >= end) return;

  if (tid == 0) {
    for (int i = 0; i < C::N_BAR; ++i) {
      int n = 1;
      if (i == C::Q_FULL || (i >= C::L_FULL && i < C::L_EMPTY)) n = NLOAD;
      if ((i >= C::P_FULL && i < C::PV_DONE) || i >= C::O_EMPTY) n = 4;
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
    *abort = 0;
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TreeSeg w;

  if (warp == 0) {
    // ---------------- MMA issuer: one thread
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(TQ, D, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sR, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sR, C::BOX, 1024);
      int nl = 0;              // slots of the items before
      int ns[2] = {0, 0};      // tasks of each tile whose S products are issued
      int np[2] = {0, 0};      // .. whose PV products are issued
      int no[2] = {0, 0};      // items of each tile so far
      bool good = true;
      for (int k = 0; good && sg.next(p, w); ++k) {
        const int nt = w.t1 - w.t0;
        const bool two = w.rows > TQ;
        auto ready = [&](int pos) {
          const int n = nl + pos;
          if (!wait_1(bar(C::L_FULL + n % NST), (n / NST) & 1, p.err, abort)) return false;
          fence_proxy_async();  // the copies were ordinary writes, the tensor core reads
          return true;
        };
        auto release = [&](int pos) { tc_commit(bar(C::L_EMPTY + (nl + pos) % NST)); };
        auto issue_s = [&](int x, int j, int buf) {
          const uint64_t da = dq0 + (uint64_t)((x * C::Q_BYTES) >> 4);
          const uint64_t db = dk0 + (uint64_t)(((nl + pos_k(j)) % NST * C::KV_BYTES) >> 4);
          const uint32_t td = tmem + C::COL_S + buf * TK;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BOX + (kk & 3) * 32;
            tc_mma_f16(td, da + (uint64_t)(off >> 4), db + (uint64_t)(off >> 4), idesc_s, kk > 0);
          }
          tc_commit(bar(C::S_FULL + 2 * x + (ns[x] & 1)));
          ++ns[x];
        };
        // O_X += P_X V_j, the K steps (16 keys) that hold keys of the sequence
        auto issue_pv = [&](int x, int j, int buf) {
          if ((j == 0 && no[x] >= 1 &&
               !wait_1(bar(C::O_EMPTY + x), (no[x] - 1) & 1, p.err, abort)) ||
              !wait_1(bar(C::P_FULL + 2 * x + (np[x] & 1)), (np[x] >> 1) & 1, p.err, abort))
            return false;
          ++np[x];
          tc_fence_after();
          const int left = w.q.len - (w.t0 + j) * TK;
          const int ks = left >= TK ? TK / 16 : (left + 15) / 16;
          const uint64_t db = dv0 + (uint64_t)(((nl + pos_v(j, nt)) % NST * C::KV_BYTES) >> 4);
          const uint32_t ta = tmem + C::COL_S + buf * TK, to = tmem + C::COL_O + x * D;
#pragma unroll 1
          for (int kk = 0; kk < ks; ++kk) {
            const uint64_t dv = db + (uint64_t)((kk * 2048) >> 4);
            tc_mma_f16_ts(to, ta + kk * 16, dv, idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
            tc_mma_f16_ts(to, ta + kk * 16 + 8, dv, idesc_pv, 1u);
          }
          tc_commit(bar(C::PV_DONE + x));
          if (j == nt - 1) ++no[x];
          return true;
        };
        if (!wait_1(bar(C::Q_FULL), k & 1, p.err, abort) || !ready(pos_k(0))) {
          good = false;
          break;
        }
        fence_proxy_async();
        tc_fence_after();
        issue_s(0, 0, 0);
        if (two) issue_s(1, 0, 1);
        release(pos_k(0));
        if (nt == 1) tc_commit(bar(C::Q_EMPTY));
        for (int j = 0; j < nt && good; ++j) {
          if (two) {
            good = (j + 1 == nt || ready(pos_k(j + 1))) && ready(pos_v(j, nt));
            for (int x = 0; x < 2 && good; ++x) {
              good = issue_pv(x, j, x);
              if (good && j + 1 < nt) issue_s(x, j + 1, x);
            }
            if (!good) break;
            if (j + 1 < nt) release(pos_k(j + 1));
          } else {
            // tile A alone: its scores take turns in the two buffers, one task ahead
            if (j + 1 < nt) {
              good = ready(pos_k(j + 1));
              if (!good) break;
              tc_fence_after();
              issue_s(0, j + 1, (j + 1) & 1);
              release(pos_k(j + 1));
            }
            good = ready(pos_v(j, nt)) && issue_pv(0, j, j & 1);
            if (!good) break;
          }
          release(pos_v(j, nt));
          if (j + 2 == nt) tc_commit(bar(C::Q_EMPTY));
        }
        nl += 2 * nt;
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  } else if (warp < 1 + NLOAD / 32) {
    // ---------------- producers: a lane finds one row's place, all copy it
    const int pw = warp - 1;
    int nl = 0, nkey = 0;  // slots, key tiles so far
    bool good = true;
    // 32 rows of D elements, lane r's at base + off (off < 0: zeros), to rows 32 pw .. of a
    // [128][64]-box tile in the 128-byte swizzle
    auto copy = [&](uint32_t dst, const bf16* base, int64_t off) {
#pragma unroll
      for (int i = 0; i < C::CH; ++i) {
        const int r = (i * 32 + lane) / C::CH, ch = (i * 32 + lane) % C::CH;
        const int64_t ro = __shfl_sync(0xffffffffu, off, r);
        const int row = pw * 32 + r;
        cp_async16(dst + (ch >> 3) * C::BOX + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   base + (ro >= 0 ? ro : 0) + ch * 8, ro >= 0);
      }
    };
    for (int k = 0; good && sg.next(p, w); ++k) {
      const int nt = w.t1 - w.t0;
      const int64_t table = (int64_t)w.q.s * p.ld_table;
      // page of this lane's token of unit j, requested one unit ahead
      int pg = 0, slot = 0;
      bool on = false;
      auto peek = [&](int j) {
        const int key = (w.t0 + j) * TK + pw * 32 + lane;  // (lengths end well below 2^31)
        on = j < nt && key < w.q.len;
        if (on) {
          const int i = key / p.page_size;
          slot = key - i * p.page_size;
          pg = p.table[table + i];
        }
      };
      peek(0);
      if (k >= 1 && !wait_w(bar(C::Q_EMPTY), (k - 1) & 1, p.err, abort)) {
        good = false;
        break;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = x * TQ + pw * 32 + lane, rr = w.b * TREE_ROWS + r;
        if (x * TQ + pw * 32 < w.rows) {  // (rows behind the last one of a warp: any values)
          const int t = rr / p.G;
          copy(sQ + x * C::Q_BYTES, static_cast<const bf16*>(p.q),
               r < w.rows ? (w.q.row + t) * p.ld_q + (int64_t)(w.h * p.G + rr - t * p.G) * D : -1);
        }
      }
      cp_async_arrive(bar(C::Q_FULL));
      int64_t before = -1;  // this lane's place of the unit before
      for (int j = 0; j <= nt && good; ++j) {
        int64_t now = -1;
        if (j < nt) {
          const bool ok = on && pg >= 0 && pg < p.n_pages;
          if (on && !ok) record_error(p.err, kErrIndex);
          if (ok) now = pg * p.s_page + slot * p.s_tok + w.h * p.s_head;
          const uint32_t bits = __ballot_sync(0xffffffffu, ok);
          peek(j + 1);
          const int n = nl + pos_k(j), s = n % NST;
          if (n >= NST && !wait_w(bar(C::L_EMPTY + s), (n / NST - 1) & 1, p.err, abort)) {
            good = false;
            break;
          }
          const int at = nkey % C::NSEE;
          if (lane == 0) {
            see[at * 4 + pw] = bits;
            mbar_arrive(bar(C::SEE + at));
          }
          ++nkey;
          copy(sR + s * C::KV_BYTES, static_cast<const bf16*>(p.k), now);
          cp_async_arrive(bar(C::L_FULL + s));
        }
        if (j > 0) {
          const int n = nl + pos_v(j - 1, nt), s = n % NST;
          if (n >= NST && !wait_w(bar(C::L_EMPTY + s), (n / NST - 1) & 1, p.err, abort)) {
            good = false;
            break;
          }
          copy(sR + s * C::KV_BYTES, static_cast<const bf16*>(p.v), before);
          cp_async_arrive(bar(C::L_FULL + s));
        }
        before = now;
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else {
    // ---------------- softmax: a thread per row; warps of tile A, then of tile B
    const int x = (warp - 1 - NLOAD / 32) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_o = tmem + C::COL_O + x * D + lane_base;
    bool good = true;
    int nx = 0;    // tasks of this tile so far
    int nkey = 0;  // key tiles of the items before
    while (good && sg.next(p, w)) {
      const int nt = w.t1 - w.t0, key0 = nkey;
      nkey += nt;
      const bool two = w.rows > TQ;
      if (x == 1 && !two) continue;
      const int row = x * TQ + r;              // of the block
      const bool live = row < w.rows;
      const bool work = x * TQ + quarter * 32 < w.rows;  // the warp has a row
      const int rr = w.b * TREE_ROWS + (live ? row : 0);
      const int tok = rr / p.G, head = w.h * p.G + rr - tok * p.G;
      const uint32_t* mask = p.mask + (int64_t)(w.q.row + tok) * TREE_WORDS;
      const int ctx = w.q.len - w.q.m;         // tokens before the draft
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < nt; ++j, ++nx) {
        const int kv0 = (w.t0 + j) * TK;
        const uint32_t t_s = tmem + C::COL_S + (two ? x : j & 1) * TK + lane_base;
        if (!wait_w(bar(C::S_FULL + 2 * x + (nx & 1)), (nx >> 1) & 1, p.err, abort)) {
          good = false;
          break;
        }
        tc_fence_after();
        if (work) {
          const int at = (key0 + j) % C::NSEE;
          if (!wait_w(bar(C::SEE + at), ((key0 + j) / C::NSEE) & 1, p.err, abort)) {
            good = false;
            break;
          }
          // the keys of the tile that this row sees
          uint32_t vis[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) vis[i] = see[at * 4 + i];
          const bool edge = kv0 + TK > ctx || (vis[0] & vis[1] & vis[2] & vis[3]) != ~0u;
          if (kv0 + TK > ctx)
#pragma unroll
            for (int i = 0; i < 4; ++i) vis[i] &= tree_window(mask, kv0 + 32 * i - ctx);
          // the largest score
          float mx = -INFINITY;
          {
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t s[32];
              tmem_ld32(t_s + i * 32, s);
              tmem_ld_wait();
              tmem_regs_ready(s);
              if (edge)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((vis[i] >> e) & 1u)) s[e] = 0xff800000u;  // -infinity
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            }
            mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
          }
          // scaled before the maximum is subtracted, as the maximum is: one rounding for
          // both, so that the largest weight is 1 for scores of any size
          mx = __fmul_rn(mx, p.sl2);
          const bool up = live && mx > m + TAU;  // the reference moves only when it must
          if (__any_sync(0xffffffffu, up)) {
            const float a = up ? exp2f(m - mx) : 1.0f;
            if (up) m = mx;
            l *= a;
            if (j > 0) {
              // (the task's own PV waits for its weights: at most one phase is outstanding)
              if (!wait_w(bar(C::PV_DONE + x), (nx - 1) & 1, p.err, abort)) *abort = 1;
              tc_fence_after();
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                tmem_ld32(t_o + i * 32, o);
                tmem_ld_wait();
                tmem_regs_ready(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                tmem_st32(t_o + i * 32, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.0f : m;  // (no score so far: every weight is 0)
          float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            uint32_t s[16], h[16];
            tmem_ld16(t_s + g * 16, s);
            tmem_ld_wait();
            tmem_regs_ready(s);
            const uint32_t v = vis[g >> 1] >> ((g & 1) * 16);
            if (edge)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!((v >> e) & 1u)) s[e] = 0xff800000u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float a, b;
              mul2(a, b, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), p.sl2, p.sl2);
              add2(a, b, a, b, -ref, -ref);
              a = ex2_ftz(a);
              b = ex2_ftz(b);
              add2(l0, l1, l0, l1, a, b);
              h[e] = pack_bf16x2(a, b);
              const float2 f = unpack_bf16x2(h[e]);
              h[8 + e] = pack_bf16x2(a - f.x, b - f.y);
            }
            tmem_st16(t_s + g * 16, h);
          }
          l += l0 + l1;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();  // the warp's stores are done: one arrival for the warp
        if (lane == 0) mbar_arrive(bar(C::P_FULL + 2 * x + (nx & 1)));
      }
      if (!good) break;
      // ---- the CTA's units of the item are done
      if (!wait_w(bar(C::PV_DONE + x), (nx - 1) & 1, p.err, abort)) {
        good = false;
        break;
      }
      tc_fence_after();
      if (work) {
        const bool whole = tree_begin(w.nt - 1, w.nt) + w.at < end && w.at >= c * chunk;
        if (whole) {
          const float inv = 1.0f / l;  // (no score: 0 / 0)
          bf16* out = static_cast<bf16*>(p.o) + (w.q.row + tok) * p.ld_o + (int64_t)head * D;
          store_tmem_row<D>(t_o, inv, live ? out : nullptr);
          if (live && p.lse != nullptr)
            p.lse[(int64_t)(w.q.row + tok) * p.nq + head] = (m + log2f(l)) * LN2;
        } else {
          const int64_t at = (int64_t)tree_part(c, chunk, w.at) * p.rows + row;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(t_o + i * 32, o);
            tmem_ld_wait();
            tmem_regs_ready(o);
            if (live)
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(p.part + at * D + i * 32 + e) =
                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          if (live) p.ml[at] = make_float2(m, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::O_EMPTY + x));
    }
    if (!good) *abort = 1;
  }
  __syncthreads();
  if (*abort && tid == 0) spin_10ms();  // let work and copies still in flight finish
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D>
mgb_status launch_d(const TreeParams& p, cudaStream_t st) {
  using C = Cfg<D>;
  auto k = tree_kernel<D>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const mgb_status s = launch_pdl(k, TREE_RANGES / 2, NTHREADS, C::SMEM, st, p);
  return s != MGB_OK ? s : tree_join(p, D, MGB_BF16, TREE_RANGES / 2, 2, st);
}

}  // namespace

mgb_status attention_tree_bf16(const TreeParams& p, int d, cudaStream_t st) {
  return d == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace mgb
