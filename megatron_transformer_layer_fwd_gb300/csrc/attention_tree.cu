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

CUresult tmap_encode_bf16_2d(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer,
                             int64_t ld, uint32_t box_inner, uint32_t box_outer);

namespace {

constexpr int TQ = 128;         // rows per tile (TMEM lanes)
constexpr int TK = TREE_KEYS;   // keys per slot
constexpr int NLOAD = 64;       // threads that copy K and V (without gather), or Q (with it)
constexpr int NTHREADS = 384;   // MMA warp, three loading warps, 2 x 4 softmax warps
constexpr float LN2 = 0.6931471805599453f;
constexpr float TAU = 8.0f;     // the reference maximum moves in steps above this (log2 units)
// Reference (log2 units) up to which the fused scale-and-subtract is off by a factor of
// at most 2, which all weights of a reference share, so that it cancels
constexpr float REF_LIMIT = 16777216.0f;

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
  static constexpr int O_FULL = PV_DONE + 2;    // [tile] the item's last PV     (commit)
  static constexpr int O_EMPTY = O_FULL + 2;    // [tile] O read out             (4: one per warp)
  static constexpr int SEE = O_EMPTY + 2;       // [key tile % NSEE] bits there  (one per producer warp)
  static constexpr int N_BAR = SEE + NSEE;
  static_assert(N_BAR * 8 <= 496, "barriers");
};

// A number for each of the tiles A (0) and B (1); selected, not indexed, so that it stays
// in registers.
struct PerTile {
  int a, b;
  __device__ int operator[](int x) const { return x ? b : a; }
  __device__ void inc(int x) { (x ? b : a) += 1; }
};

// The slot a key tile's K or V has in the item's order K_0, K_1, V_0, K_2, V_1, ..
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * n - 1; }

// The hot loops of all roles share the instruction cache, which they outgrow easily (a
// form with everything unrolled spent 60 % of its cycles waiting for instructions): what is
// rare is kept out of line, copies and score chunks in loops.
//
// One thread: waits for the phase, for a bounded time and only while no role has given up.
__device__ __noinline__ bool wait_1_slow(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
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
__device__ __forceinline__ bool wait_1(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  return mbar_try_wait(bar, parity) || wait_1_slow(bar, parity, err, abort);
}
// The same for a whole warp, which goes on together.
__device__ __noinline__ bool wait_w_slow(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  const uint64_t t0 = global_ns();
  for (;;) {
    const bool ok = mbar_try_wait_suspend(bar, parity, 50000u);
    if (__all_sync(0xffffffffu, ok)) return true;
    const bool late = global_ns() - t0 > kWaitLimitNs;
    if (late) record_error(err, kErrTimeout);
    if (__any_sync(0xffffffffu, late || *abort != 0)) return false;
  }
}
__device__ __forceinline__ bool wait_w(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_w_slow(bar, parity, err, abort);
}

// The barrier counts one arrival of this thread when its copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A warp copies 32 rows of D elements, lane r's at base + off (off < 0: zeros), to rows row0
// .. of a [128][64]-box tile in the 128-byte swizzle.
template <int D>
__device__ __noinline__ void copy_rows(uint32_t dst, int row0, const bf16* base, int64_t off) {
  constexpr int CH = Cfg<D>::CH;
  const int lane = threadIdx.x & 31;
  const int ch = lane % CH, r0 = lane / CH;
  base += ch * 8;
  dst += (ch >> 3) * Cfg<D>::BOX + row0 * 128;
#pragma unroll 8
  for (int i = 0; i < CH; ++i) {
    const int r = i * (32 / CH) + r0;
    const int64_t ro = __shfl_sync(0xffffffffu, off, r);
    cp_async16(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4), base + (ro >= 0 ? ro : 0), ro >= 0);
  }
}

// Queries of the item's rows, groups first, first + step, .. of 32 of them.
template <int D>
__device__ __forceinline__ void copy_q(const TreeParams& p, const TreeSeg& w, uint32_t sQ, int first, int step) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int g = first; g * 32 < w.rows; g += step) {
    const int r = g * 32 + lane, rr = w.b * TREE_ROWS + r, t = rr / p.G;
    copy_rows<D>(sQ + (g >> 2) * Cfg<D>::Q_BYTES, (g & 3) * 32, static_cast<const bf16*>(p.q),
                 r < w.rows ? (w.q.row + t) * p.ld_q + (int64_t)(w.h * p.G + rr - t * p.G) * D : -1);
  }
}

// Scores of 32 keys -> weights 2^(s a + b) in two bf16 parts, per 16 keys the high parts of
// the pairs in the first eight words, the low parts in the others; the sums take them
// whole. The high part is the weight cut off, the low part what that leaves, rounded: off by
// 2^-16 relative at most.
__device__ __forceinline__ void weights(uint32_t (&s)[32], float a, float b, float (&sum)[4]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x, y, u, v;
      fma2(x, y, __uint_as_float(s[16 * g + 2 * e]), __uint_as_float(s[16 * g + 2 * e + 1]), a, a, b, b);
      x = ex2_ftz(x);
      y = ex2_ftz(y);
      float* t = sum + 2 * (e & 1);
      add2(t[0], t[1], t[0], t[1], x, y);
      const uint32_t xu = __float_as_uint(x), yu = __float_as_uint(y);
      hi[e] = __byte_perm(xu, yu, 0x7632);
      add2(u, v, x, y, __uint_as_float((xu & 0xffff0000u) ^ 0x80000000u),
           __uint_as_float((yu & 0xffff0000u) ^ 0x80000000u));
      lo[e] = pack_bf16x2(u, v);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[16 * g + e] = hi[e], s[16 * g + 8 + e] = lo[e];
  }
}

// Where the pools' vectors are as rows of a matrix: vector (page, slot, head) is row page
// r_page + slot + head r_head, column head c_head. Copies take `box` rows (a power of two that
// divides the page size, 8 to 128), which lie in one page.
struct RowMap {
  int r_page, r_head, c_head, rows, box, shift;  // box = 1 << shift
};
struct PoolMaps {
  CUtensorMap k, v, k1, v1;  // boxes of `box` rows; of one row, for gather copies
};

// Four rows of 64 columns from column x on, to 512 bytes of a 128-byte-swizzled tile; a row
// outside the matrix gives zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* tmap, int32_t x, const int (&r)[4],
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

// TMA: the pools are rows of a matrix, and the TMA unit copies
template <int D, bool TMA>
__global__ void __launch_bounds__(NTHREADS, 1)
    tree_kernel(const __grid_constant__ PoolMaps tm, const RowMap rm, const TreeParams p) {
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
      if (i == C::Q_FULL || (!TMA && i >= C::L_FULL && i < C::L_EMPTY)) n = NLOAD;
      if ((i >= C::P_FULL && i < C::PV_DONE) || (i >= C::O_EMPTY && i < C::SEE)) n = 4;
      if (i >= C::SEE) n = TMA ? 1 : NLOAD / 32;
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
      int nl = 0;          // slots of the items before
      PerTile ns{0, 0};    // tasks of each tile whose S products are issued
      PerTile np{0, 0};    // .. whose PV products are issued
      PerTile no{0, 0};    // items of each tile so far
      bool good = true;
      for (int k = 0; good && sg.next(p, w); ++k) {
        const int nt = w.t1 - w.t0;
        const bool two = w.rows > TQ;
        auto ready = [&](int pos) {
          const int n = nl + pos;
          if (!wait_1(bar(C::L_FULL + n % NST), (n / NST) & 1, p.err, abort)) return false;
          fence_proxy_async();  // the copies were ordinary writes, the tensor core reads
          tc_fence_after();
          return true;
        };
        auto release = [&](int pos) { tc_commit(bar(C::L_EMPTY + (nl + pos) % NST)); };
        good = wait_1(bar(C::Q_FULL), k & 1, p.err, abort);
        // Per unit: two tiles take turns, PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1), each in its
        // score buffer; tile A alone has its scores one task ahead, S(j + 1), PV(j), in the
        // two buffers by turns.
#pragma unroll 1
        for (int j = -1; j < nt && good; ++j) {
#pragma unroll 1
          for (int i = 0; i < (two ? 4 : 2) && good; ++i) {
            const int x = i >> 1;
            const bool last = x == 1 || !two;
            if (((i & 1) == 0) != two) {
              if (j + 1 == nt) continue;
              if (x == 0) good = ready(pos_k(j + 1));
              if (!good) break;
              const uint64_t da = dq0 + (uint64_t)((x * C::Q_BYTES) >> 4);
              const uint64_t db = dk0 + (uint64_t)(((nl + pos_k(j + 1)) % NST * C::KV_BYTES) >> 4);
              const uint32_t td = tmem + C::COL_S + (two ? x : (j + 1) & 1) * TK;
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * C::BOX + (kk & 3) * 32;
                tc_mma_f16(td, da + (uint64_t)(off >> 4), db + (uint64_t)(off >> 4), idesc_s, kk > 0);
              }
              tc_commit(bar(C::S_FULL + 2 * x + (ns[x] & 1)));
              ns.inc(x);
              if (last) {
                release(pos_k(j + 1));
                if (j + 2 == nt) tc_commit(bar(C::Q_EMPTY));
              }
            } else {
              if (j < 0) continue;
              // O_X += P_X V_j, the K steps (16 keys) that hold keys of the sequence
              good = (x == 1 || ready(pos_v(j, nt))) &&
                     (j > 0 || no[x] == 0 || wait_1(bar(C::O_EMPTY + x), (no[x] - 1) & 1, p.err, abort)) &&
                     wait_1(bar(C::P_FULL + 2 * x + (np[x] & 1)), (np[x] >> 1) & 1, p.err, abort);
              if (!good) break;
              np.inc(x);
              tc_fence_after();
              const int left = w.q.len - (w.t0 + j) * TK;
              const int ks = left >= TK ? TK / 16 : (left + 15) / 16;
              const uint64_t db = dv0 + (uint64_t)(((nl + pos_v(j, nt)) % NST * C::KV_BYTES) >> 4);
              const uint32_t ta = tmem + C::COL_S + (two ? x : j & 1) * TK, to = tmem + C::COL_O + x * D;
#pragma unroll 4
              for (int kk = 0; kk < ks; ++kk) {
                const uint64_t dv = db + (uint64_t)((kk * 2048) >> 4);
                tc_mma_f16_ts(to, ta + kk * 16, dv, idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
                tc_mma_f16_ts(to, ta + kk * 16 + 8, dv, idesc_pv, 1u);
              }
              tc_commit(bar(C::PV_DONE + x));
              if (j == nt - 1) {
                tc_commit(bar(C::O_FULL + x));
                no.inc(x);
              }
              if (last) release(pos_v(j, nt));
            }
          }
        }
        nl += 2 * nt;
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  } else if (TMA && warp == 1) {
    // ---------------- K and V: a lane finds the page of one box and asks for it
    int nl = 0, nkey = 0;  // slots, key tiles so far
    const int nbox = TK >> rm.shift;
    bool good = true;
    while (good && sg.next(p, w)) {
      const int nt = w.t1 - w.t0, x = w.h * rm.c_head;
      const int32_t* table = p.table + (int64_t)w.q.s * p.ld_table;
      // page of this lane's box of unit j, requested one unit ahead
      int pg = 0, slot = 0;
      bool on = false;
      auto peek = [&](int j) {
        const int key = (w.t0 + j) * TK + (lane << rm.shift);  // (lengths end well below 2^31)
        on = j < nt && lane < nbox && key < w.q.len;
        if (on) {
          const int e = key / p.page_size;
          slot = key - e * p.page_size;
          pg = table[e];
        }
      };
      peek(0);
      int now = rm.rows, before = rm.rows;  // first row of this lane's box of the newest unit, of the one before
#pragma unroll 1
      for (int pos = 0; pos < 2 * nt; ++pos) {
        const bool is_v = pos == 2 * nt - 1 || (pos > 0 && (pos & 1) == 0);
        const int n = nl + pos, s = n % NST;
        const int j = pos == 2 * nt - 1 ? nt - 1 : is_v ? (pos - 2) / 2 : (pos + 1) / 2;
        const int left = w.q.len - (w.t0 + j) * TK;  // keys of the sequence from here on
        uint32_t boxes = 0;
        if (!is_v) {
          const bool ok = on && pg >= 0 && pg < p.n_pages;
          if (on && !ok) record_error(p.err, kErrIndex);
          before = now;
          now = ok ? pg * rm.r_page + slot + w.h * rm.r_head : rm.rows;  // (no row: zeros)
          boxes = __ballot_sync(0xffffffffu, ok);
          peek(j + 1);
        }
        const uint32_t full = bar(C::L_FULL + s);
        if (n >= NST && !wait_w(bar(C::L_EMPTY + s), (n / NST - 1) & 1, p.err, abort)) {
          good = false;
          break;
        }
        if (!is_v) {
          const int at = nkey++ % C::NSEE;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 32 * i + lane;
            const uint32_t bits = __ballot_sync(0xffffffffu, key < left && ((boxes >> (key >> rm.shift)) & 1u));
            if (lane == 0) see[at * 4 + i] = bits;
          }
          if (lane == 0) mbar_arrive(bar(C::SEE + at));
        }
        if (lane == 0) mbar_arrive_expect_tx(full, C::KV_BYTES);
        __syncwarp();
        const int row = !is_v || pos == 2 * nt - 1 ? now : before;
        const uint32_t dst = sR + s * C::KV_BYTES;
        // the box with the sequence's end: row by row, so that slots behind it are zeros
        const int part = left < TK && (left & (rm.box - 1)) ? left >> rm.shift : nbox;
        if (lane < nbox && lane != part)
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(dst + kb * C::BOX + (lane << rm.shift) * 128, is_v ? &tm.v : &tm.k, x + kb * 64, row, full);
        if (part < nbox) {
          const int first = __shfl_sync(0xffffffffu, row, part);
          if ((4 * lane) >> rm.shift == part) {
            int r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              r[i] = first < rm.rows && 4 * lane + i < left ? first + 4 * lane + i - (part << rm.shift) : rm.rows;
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_gather4(dst + kb * C::BOX + lane * 512, is_v ? &tm.v1 : &tm.k1, x + kb * 64, r, full);
          }
        }
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
  } else if (TMA && warp < 4) {
    // ---------------- Q: groups of 32 rows in turn
    bool good = true;
    for (int k = 0; good && sg.next(p, w); ++k) {
      if (k >= 1) good = wait_w(bar(C::Q_EMPTY), (k - 1) & 1, p.err, abort);
      if (good) copy_q<D>(p, w, sQ, warp - 2, 2);
      cp_async_arrive(bar(C::Q_FULL));
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else if (!TMA && warp == 3) {
    // (nothing to do)
  } else if (!TMA && warp < 1 + NLOAD / 32) {
    // ---------------- producers: a lane finds one row's place, all copy it
    const int pw = warp - 1;
    constexpr int NR = TQ / NLOAD;  // rows per lane: 32 (NR pw + i) + lane
    int nl = 0, nkey = 0;  // slots, key tiles so far
    bool good = true;
    for (int k = 0; good && sg.next(p, w); ++k) {
      const int nt = w.t1 - w.t0;
      const int64_t table = (int64_t)w.q.s * p.ld_table;
      // pages of this lane's tokens of unit j, requested one unit ahead
      int pg[NR], slot[NR];
      bool on[NR];
      auto peek = [&](int j) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int key = (w.t0 + j) * TK + (pw * NR + i) * 32 + lane;  // (lengths end well below 2^31)
          on[i] = j < nt && key < w.q.len;
          if (on[i]) {
            const int e = key / p.page_size;
            slot[i] = key - e * p.page_size;
            pg[i] = p.table[table + e];
          }
        }
      };
      peek(0);
      if (k >= 1 && !wait_w(bar(C::Q_EMPTY), (k - 1) & 1, p.err, abort)) {
        good = false;
        break;
      }
      copy_q<D>(p, w, sQ, pw, 2);
      cp_async_arrive(bar(C::Q_FULL));
      int64_t now[NR], before[NR];  // this lane's places of the newest unit and the one before it
#pragma unroll 1
      for (int pos = 0; pos < 2 * nt; ++pos) {
        const bool is_v = pos == 2 * nt - 1 || (pos > 0 && (pos & 1) == 0);
        const int n = nl + pos, s = n % NST;
        uint32_t bits[NR];
        if (!is_v) {
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const bool ok = on[i] && pg[i] >= 0 && pg[i] < p.n_pages;
            if (on[i] && !ok) record_error(p.err, kErrIndex);
            before[i] = now[i];
            now[i] = ok ? pg[i] * p.s_page + slot[i] * p.s_tok + w.h * p.s_head : -1;
            bits[i] = __ballot_sync(0xffffffffu, ok);
          }
          peek((pos + 1) / 2 + 1);
        }
        if (n >= NST && !wait_w(bar(C::L_EMPTY + s), (n / NST - 1) & 1, p.err, abort)) {
          good = false;
          break;
        }
        if (!is_v) {
          const int at = nkey++ % C::NSEE;
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < NR; ++i) see[at * 4 + pw * NR + i] = bits[i];
            mbar_arrive(bar(C::SEE + at));
          }
        }
        const bool newest = !is_v || pos == 2 * nt - 1;
#pragma unroll
        for (int i = 0; i < NR; ++i)
          copy_rows<D>(sR + s * C::KV_BYTES, (pw * NR + i) * 32,
                       static_cast<const bf16*>(is_v ? p.v : p.k), newest ? now[i] : before[i]);
        cp_async_arrive(bar(C::L_FULL + s));
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else {
    // ---------------- softmax: a thread per row; warps of tile A, then of tile B
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_o = tmem + C::COL_O + x * D + lane_base;
    bool good = true;
    int nx = 0;    // tasks of this tile so far
    int ko = 0;    // items of this tile so far
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
          // Few tiles have hidden keys: their scores are overwritten first.
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = vis[i];
              if (__all_sync(0xffffffffu, v == ~0u)) continue;
              uint32_t s[32];
              tmem_ld32(t_s + i * 32, s);
              tmem_ld_wait();
              tmem_regs_ready(s);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((v >> e) & 1u)) s[e] = 0xff800000u;  // -infinity
              tmem_st32(t_s + i * 32, s);
            }
            tmem_st_wait();
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int i = 0; i < 4; i += 2) {
            uint32_t s[2][32];
            tmem_ld32(t_s + i * 32, s[0]);
            tmem_ld32(t_s + i * 32 + 32, s[1]);
            tmem_ld_wait();
            tmem_regs_ready(s[0]);
            tmem_regs_ready(s[1]);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                m4[y] = fmax3(m4[y], __uint_as_float(s[y & 1][e + (y & 2)]),
                              __uint_as_float(s[y & 1][e + (y & 2) + 1]));
          }
          const float mx = __fmul_rn(fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]), p.sl2);
          const bool up = live && mx > m + TAU;  // the reference moves only when it must
          if (__any_sync(0xffffffffu, up)) {
            const float a = up ? exp2f(m - mx) : 1.0f;
            if (up) m = mx;
            l *= a;
            if (j > 0) {
              // (the scores were formed behind the PV before the last, and the task's own PV waits for
              // its weights: at most one phase is outstanding)
              if (!wait_w(bar(C::PV_DONE + x), (nx - 1) & 1, p.err, abort)) *abort = 1;
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                uint32_t o[16];
                tmem_ld16(t_o + i * 16, o);
                tmem_ld_wait();
                tmem_regs_ready(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                tmem_st16(t_o + i * 16, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.0f : m;  // (no score so far: every weight is 0)
          float shift = -ref;
          if (__any_sync(0xffffffffu, fabsf(ref) > REF_LIMIT)) {
            // scores scaled and rounded as the maximum was before it is subtracted, so that the
            // largest weight is 1; the differences take the scores' place
            shift = 0.0f;
            const float back = 1.0f / p.sl2;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              uint32_t s[16];
              tmem_ld16(t_s + i * 16, s);
              tmem_ld_wait();
              tmem_regs_ready(s);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                s[e] = __float_as_uint((__fmul_rn(__uint_as_float(s[e]), p.sl2) - ref) * back);
              tmem_st16(t_s + i * 16, s);
            }
            tmem_st_wait();
          }
          float sum[4] = {};
#pragma unroll 1
          for (int i = 0; i < 4; i += 2) {  // (no load is under way from one round to the next)
            uint32_t s[2][32];
            tmem_ld32(t_s + i * 32, s[0]);
            tmem_ld32(t_s + i * 32 + 32, s[1]);
            tmem_ld_wait();
            tmem_regs_ready(s[0]);
            tmem_regs_ready(s[1]);
            weights(s[0], p.sl2, shift, sum);
            tmem_st32(t_s + i * 32, s[0]);
            weights(s[1], p.sl2, shift, sum);
            tmem_st32(t_s + i * 32 + 32, s[1]);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();  // the warp's stores are done: one arrival for the warp
        if (lane == 0) mbar_arrive(bar(C::P_FULL + 2 * x + (nx & 1)));
      }
      if (!good) break;
      // ---- the CTA's units of the item are done
      if (!wait_w(bar(C::O_FULL + x), ko++ & 1, p.err, abort)) {
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

// Whether the TMA unit can copy: pages of a multiple of 8 slots, and vectors one stride apart
// over slots, pages and heads (or heads next to each other in a row).
bool row_map(const TreeParams& p, int d, RowMap& m, int64_t& ld, int64_t& width) {
  m.shift = __builtin_ctz((unsigned)p.page_size);
  if (m.shift < 3) return false;
  if (m.shift > 7) m.shift = 7;
  m.box = 1 << m.shift;
  ld = p.s_tok;
  if (p.n_pages > 1 && p.s_page % ld) return false;
  const int64_t across = (p.nkv - 1) * p.s_head + d;
  const bool in_row = across <= ld;
  if (!in_row && p.s_head % ld) return false;
  width = in_row ? across : d;
  const int64_t r_page = p.n_pages > 1 ? p.s_page / ld : 0, r_head = in_row ? 0 : p.s_head / ld;
  const int64_t rows = (p.n_pages - 1) * r_page + p.page_size + (p.nkv - 1) * r_head;
  if (rows >= (int64_t)1 << 31 || width >= (int64_t)1 << 31) return false;
  m.r_page = (int)r_page; m.r_head = (int)r_head; m.c_head = in_row && p.nkv > 1 ? (int)p.s_head : 0;
  m.rows = (int)rows;
  return true;
}

template <int D, bool TMA>
mgb_status launch_k(const TreeParams& p, const PoolMaps& tm, const RowMap& rm, cudaStream_t st) {
  using C = Cfg<D>;
  auto k = tree_kernel<D, TMA>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const mgb_status s = launch_pdl(k, TREE_RANGES / 2, NTHREADS, C::SMEM, st, tm, rm, p);
  return s != MGB_OK ? s : tree_join(p, D, MGB_BF16, TREE_RANGES / 2, 2, st);
}

template <int D>
mgb_status launch_d(const TreeParams& p, cudaStream_t st) {
  PoolMaps tm{};
  RowMap rm{};
  int64_t ld, w;
  if (!row_map(p, D, rm, ld, w)) return launch_k<D, false>(p, tm, rm, st);
  const uint64_t n = (uint64_t)rm.rows;
  if (tmap_encode_bf16_2d(&tm.k, p.k, w, n, ld, 64, rm.box) != CUDA_SUCCESS ||
      tmap_encode_bf16_2d(&tm.v, p.v, w, n, ld, 64, rm.box) != CUDA_SUCCESS ||
      tmap_encode_bf16_2d(&tm.k1, p.k, w, n, ld, 64, 1) != CUDA_SUCCESS ||
      tmap_encode_bf16_2d(&tm.v1, p.v, w, n, ld, 64, 1) != CUDA_SUCCESS)
    return MGB_ERR_CUDA;
  return launch_k<D, true>(p, tm, rm, st);
}

}  // namespace

mgb_status attention_tree_bf16(const TreeParams& p, int d, cudaStream_t st) {
  return d == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace mgb
