// Attention of drafted tokens over a paged cache, bf16, on the tensor cores
// (tcgen05): o = softmax(q K^T / sqrt(d)) V over the cached tokens that a drafted
// token sees, all those before the draft, its ancestors in the tree and itself.
//
// An item's rows are the drafted tokens times the query heads of one KV head. K and V
// pass once through shared memory for up to 256 rows. Two streams A and B of 128 rows
// take turns on the tensor core: with more than 128 rows they are the two halves of the
// rows, each with all units of 128 keys; with fewer both are the same rows, A with the
// even units, B with the odd ones, joined at the end. Per unit and stream: S = Q K^T
// (TMEM), the softmax threads (one per row) turn the scores into weights P in place, and
// O += P V with P read from TMEM. One thread issues PV and the next S of one stream while the
// other's softmax is at work. (A thread per stream was slower, 156 us against 143 with 244 rows
// over 131001 tokens: the streams' products mix, and their softmaxes fall together.)
//
// P multiplies V as the sum of two bf16 parts (off by 2^-16 relative at most): with one
// part the weights' errors would add as much again as the output's own rounding. The
// parts of 16 keys take the 16 columns that their scores had.
//
// K and V come through a ring of slots of 128 keys in the order in which the products need
// them: K_0, V_0, K_1, .., or, where the streams take the units in turn, K_0, K_1, V_0, K_2, V_1,
// .. Pages of a multiple of 8 slots are copied by the TMA unit, a box of up to 128 slots of one
// page at a time (V by threads where the unit alone is too slow, see SPLIT_COST); others row by
// row with 16-byte asynchronous copies. A wait for a
// place n to be free tells its laps apart by a parity, so whoever waits has to know that the place's lap
// before, n - 2 NST, is free. It does: one thread frees the places in their order, and of those that a
// role waits for (all; where V has threads of its own, those of K or of V) each is at most RING_GAP
// <= NST behind the one before, whose wait has shown everything up to n - RING_GAP - NST free. V of
// tokens behind the length, and K and V of those of a bad page, are not read: zeros stand in their
// place; a bit per key says that no row sees them.
//
// Measured, 32 query and 8 KV heads of 128: one sequence of 131001 tokens, 244 rows 125 to 131
// us, 1000 to 1045 TFLOP/s with each product counted once (P's second part makes it half as much
// again), 64 rows 90 to 94 us, 5.7 to 6.0 TB/s; 32 sequences of 33 to 16000 tokens, 8 to 96 rows 58 us, 4.5 TB/s; two of 7000 to
// 9000 with 1024 rows each 69 us. Bound: with two halves of rows the tensor cores, 101 of the
// 125 us at the rate of a large product (start and join 10); with one the HBM.
#include <cudaTypedefs.h>

#include "tree.cuh"

namespace mgb {

namespace {

constexpr int TQ = 128;         // rows per stream (TMEM lanes)
constexpr int TK = CutTc::KEYS;   // keys per slot
constexpr int NLOAD = 64;       // threads that copy K, V and Q without TMA
constexpr int NFILL = 33;       // arrivals at a slot that TMA fills: the bytes' one, and a warp's
constexpr int NTHREADS = 384;   // warp 0: products; 1 to 3: loads; 2 x 4: softmax
constexpr float LN2 = 0.6931471805599453f;
constexpr float TAU = 8.0f;     // the reference maximum moves in steps above this (log2 units)
// Reference (log2 units) up to which the fused scale-and-subtract is off by a factor of
// at most 2, which all weights of a reference share, so that it cancels
constexpr float REF_LIMIT = 16777216.0f;

template <int D>
struct Cfg {
  static constexpr int NST = D == 64 ? 10 : 5;          // ring slots
  // Two K, or two V, that follow each other in the ring are at most this many places apart: an item's
  // last K, V, V and the next item's K; an item's last V and the next item's K, K, V.
  static constexpr int RING_GAP = 3;
  static_assert(RING_GAP <= NST, "a wait could take a lap long past for its own");
  static constexpr int KB = D / 64;                     // 64-wide d blocks
  static constexpr int CH = D / 8;                      // 16-byte chunks of a row
  // A tile of 128 rows: groups of 8 rows, in a group the d blocks, in a block 8 rows of 128
  // bytes in the 128-byte swizzle; so a TMA box of whole rows is a run of groups.
  static constexpr int GROUP = KB * 1024;
  static constexpr int TILE = 16 * GROUP;
  // (Q: the d blocks of all 128 rows one behind the other)
  static constexpr int OFF_Q = 0;                       // [tile] 128 rows: an item's halves, or items in turn
  static constexpr int OFF_R = 2 * TILE;                // [slot]
  static constexpr int OFF_SEE = OFF_R + NST * TILE;    // [NSEE][4]: a bit per key that may be seen
  static constexpr int NSEE = 16;
  static constexpr int OFF_ML = OFF_SEE + NSEE * 16;    // [128] maximum and row sum of stream B
  static constexpr int OFF_BAR = OFF_ML + TQ * 8;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;     // barriers, alignment slack
  static constexpr int COL_S = 0;                       // scores of A, of B
  static constexpr int COL_O = 2 * TK;                  // O_A, then O_B at + D
  static constexpr int TMEM_COLS = 512;
  static_assert(COL_O + 2 * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  // Barriers (8 bytes each). A waiter sees every phase of a barrier, or knows that its
  // phase is complete (parity).
  static constexpr int Q_FULL = 0;              // [tile] 128 rows of queries    (tx, or the copying threads)
  static constexpr int Q_EMPTY = 2;             // [tile] the item's last S done (commit)
  static constexpr int L_FULL = 4;              // [slot] copied                 (tx and NFILL or NLOAD threads)
  static constexpr int L_EMPTY = L_FULL + NST;  // [slot] its products done      (commit)
  static constexpr int S_FULL = L_EMPTY + NST;  // [stream] scores, and the PV before  (commit)
  static constexpr int O_FULL = S_FULL + 2;     // [stream] the item's last PV   (commit)
  static constexpr int P_HALF = O_FULL + 2;     // [stream] weights of 64 keys   (4: one per warp)
  static constexpr int P_FULL = P_HALF + 2;     // [stream] of all               (4: one per warp)
  static constexpr int O_EMPTY = P_FULL + 2;    // [stream] O read out           (4: one per warp)
  static constexpr int ML = O_EMPTY + 2;        // B's maxima and sums are there (4: one per warp)
  static constexpr int SEE = ML + 1;            // [unit % NSEE] bits are there  (one per loading warp)
  static constexpr int N_BAR = SEE + NSEE;
  static_assert(N_BAR * 8 <= 496, "barriers");
};

// A number for each of the streams A (0) and B (1); selected, not indexed, so that it stays
// in registers.
struct PerStream {
  int a, b;
  __device__ int operator[](int x) const { return x ? b : a; }
  __device__ void inc(int x) { (x ? b : a) += 1; }
};

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
// .. of a tile whose groups of 8 rows and d blocks lie `group` and `block` bytes apart.
template <int D>
__device__ __noinline__ void copy_rows(uint32_t dst, int row0, const bf16* base, int64_t off, int group, int block) {
  constexpr int CH = Cfg<D>::CH;
  const int lane = threadIdx.x & 31;
  const int ch = lane % CH, r0 = lane / CH;
  base += ch * 8;
  dst += (row0 >> 3) * group + (ch >> 3) * block;
#pragma unroll 8
  for (int i = 0; i < CH; ++i) {
    const int r = i * (32 / CH) + r0;
    const int64_t ro = __shfl_sync(0xffffffffu, off, r);
    cp_async16(dst + (r >> 3) * group + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4),
               base + (ro >= 0 ? ro : 0), ro >= 0);
  }
}

// A loading warp's groups of 32 of the item's queries (first, first + step, .. of four per
// tile), into the next one or two tiles (nq so far).
template <int D>
__device__ __forceinline__ bool copy_q(const TreeParams& p, const TreeSeg& w, uint32_t sb, int first, int step,
                                       int& nq, volatile int* abort) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int x = 0; x * TQ < w.rows; ++x, ++nq) {
    const int tile = nq & 1;
    if (nq >= 2 && !wait_w(sb + C::OFF_BAR + 8 * (C::Q_EMPTY + tile), ((nq >> 1) - 1) & 1, p.err, abort)) return false;
#pragma unroll 1
    for (int g = 4 * x + first; g < 4 * x + 4 && g * 32 < w.rows; g += step) {
      const int r = g * 32 + lane, rr = w.b * CutTc::ROWS + r, t = rr / p.G;
      copy_rows<D>(sb + C::OFF_Q + tile * C::TILE, (g & 3) * 32, static_cast<const bf16*>(p.q),
                   r < w.rows ? (w.q.row + t) * p.ld_q + (int64_t)(w.h * p.G + rr - t * p.G) * D : -1, 1024, 16384);
    }
    cp_async_arrive(sb + C::OFF_BAR + 8 * (C::Q_FULL + tile));
  }
  return true;
}

// The steps of the weights in an order that the compiler keeps (volatile).
__device__ __forceinline__ void v_fma2(float& r0, float& r1, uint32_t a0, uint32_t a1, float b, float c) {
  asm volatile(
      "{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " mov.b64 c, {%5, %5};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r0), "=f"(r1)
      : "r"(a0), "r"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void v_ex2(float& x) { asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x)); }
__device__ __forceinline__ void v_add2(float& r0, float& r1, float a0, float a1, float b0, float b1) {
  asm volatile(
      "{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ uint32_t v_pack(float lo, float hi) {
  uint32_t r;
  asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// what a pair of bf16 leaves of the two numbers that it was rounded from (exact)
__device__ __forceinline__ void v_rest(float& r0, float& r1, float x0, float x1, uint32_t pair) {
  asm volatile(
      "{\n .reg .b16 a, b, m;\n mov.b32 {a, b}, %4;\n mov.b16 m, 0xBF80;\n"
      " fma.rn.f32.bf16 %0, a, m, %2;\n fma.rn.f32.bf16 %1, b, m, %3;\n}\n"
      : "=f"(r0), "=f"(r1)
      : "f"(x0), "f"(x1), "r"(pair));
}

// Scores of 64 keys -> weights 2^(s a + b) in two bf16 parts, per 16 keys the high parts of
// the pairs in the first eight words, the low parts in the others; the sums take them
// whole. The high part is the weight rounded, the low part what that leaves, rounded: off by
// 2^-16 relative at most. Groups of four keys: the exponentials of one between the sums and
// parts of the second before (whose exponentials are done by then) and the scaling of the
// second next. (The exponential unit takes 4 cycles per instruction; conversions, masks and
// permutes 2 like the paired products and sums, which they hold up; so what the high part leaves
// comes from a mixed fused product of the FMA pipe, not from masks and a paired sum.)
__device__ __forceinline__ void weights(uint32_t (&s)[2][32], float a, float b, float (&sum)[4]) {
  float t[8][4];
  auto scale = [&](int g) {
    const uint32_t* z = s[g >> 3] + (g & 7) * 4;
    v_fma2(t[g & 7][0], t[g & 7][1], z[0], z[1], a, b);
    v_fma2(t[g & 7][2], t[g & 7][3], z[2], z[3], a, b);
  };
  scale(0);
  scale(1);
  uint32_t out[2][32];
#pragma unroll
  for (int g = 0; g < 16 + 2; ++g) {
    float* y = t[g & 7];
    const int h = g - 2;
    const float* u = t[h & 7];
    uint32_t* o = h >= 0 ? out[h >> 3] + (h & 4) * 4 + (h & 3) * 2 : nullptr;
    float r0, r1, r2, r3;
    if (g < 16) v_ex2(y[0]);
    if (h >= 0) {
      o[0] = v_pack(u[0], u[1]);
      v_add2(sum[0], sum[1], sum[0], sum[1], u[0], u[1]);
    }
    if (g < 16) v_ex2(y[1]);
    if (h >= 0) {
      o[1] = v_pack(u[2], u[3]);
      v_add2(sum[2], sum[3], sum[2], sum[3], u[2], u[3]);
    }
    if (g < 16) v_ex2(y[2]);
    if (h >= 0) v_rest(r0, r1, u[0], u[1], o[0]);
    if (g + 2 < 16) scale(g + 2);
    if (g < 16) v_ex2(y[3]);
    if (h >= 0) {
      v_rest(r2, r3, u[2], u[3], o[1]);
      o[8] = v_pack(r0, r1);
      o[9] = v_pack(r2, r3);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 32; ++e) s[i][e] = out[i][e];
}

// How the TMA unit finds a pool's vectors: an element of a head's vector, row of 8 slots, d
// block, group of 8 slots, page.
struct PoolMaps {
  CUtensorMap k, v[2];     // boxes of `box` slots; of 8
  CUtensorMap q;           // an element of a head's vector, query head of a KV head, token, d block
  int shift;               // box = 1 << shift slots: 8 to 128, in one page
  int q_tma;               // q is used: heads of a group divide 128
  int split;               // V of long sequences comes by threads
};
// rows of a unit's V that its products read: those with keys of the sequence, to the K step's end
__device__ __forceinline__ int used_rows(int left) { return min(TK, (left + 15) & ~15); }
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int head, int token, int kb,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(head), "r"(token), "r"(kb), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int x, int row, int kb, int group,
                                            int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(row), "r"(kb), "r"(group), "r"(page), "r"(bar)
      : "memory");
}

// Whether V comes by two warps, row by row, beside K by the TMA unit: the unit needs 100 to 150
// cycles per box and 4 to 5 per row of 128 bytes, so with small boxes, and at head dim 64, it
// alone is slower than the memory. One choice for a launch. Sequences that average 1000 tokens or
// more (8 units of up to 128 rows) gain, 64 of 2000 tokens: head dim 64, pages of 8, 16, 32 and
// 64, 231, 177, 152 and 140 us with V by TMA, 150, 131, 131 and 132 by threads; head dim 128 143,
// 115, 103 and 98 and 105, 103, 103 and 103. Short ones wait longer for a V by threads (200
// of 100 to 600 tokens, pages of 16, 78 us and 104), and with items of more than 128 rows the
// tensor cores are the bound (64 of 2000 tokens, 256 rows, 156 us and 169).
constexpr int SPLIT_COST = 8 * CutTc::C1 + CutTc::ITEM;

template <int D, bool TMA>
__global__ void __launch_bounds__(NTHREADS, 1)
    tree_kernel(const __grid_constant__ PoolMaps tm, const TreeParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t sQ = sb + C::OFF_Q, sR = sb + C::OFF_R;
  constexpr int NST = C::NST;
  auto bar = [&](int which) { return sb + C::OFF_BAR + 8 * which; };
  volatile uint32_t* see = reinterpret_cast<uint32_t*>(smem + C::OFF_SEE);
  volatile float* sml = reinterpret_cast<float*>(smem + C::OFF_ML);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 496);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 500);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (shared memory and TMEM while the kernel before may still run)
  if (tid < C::N_BAR) {
    int n = 1;
    if (tid < C::Q_EMPTY) n = !TMA ? NLOAD : tm.q_tma ? 1 : 32;
    else if (tid >= C::L_FULL && tid < C::L_EMPTY) n = !TMA || tm.split ? NLOAD : NFILL;
    if (tid >= C::P_HALF && tid <= C::ML) n = 4;
    if (!TMA && tid >= C::SEE) n = NLOAD / 32;
    mbar_init(bar(tid), n);
    fence_mbar_init();
  }
  if (tid == 0) *abort = 0;
  if (TMA && tid >= 64 && tid < 68) tma_prefetch_desc(tid < 66 ? &tm.v[tid - 64] : tid < 67 ? &tm.k : &tm.q);
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();     // everything the call reads may come from the kernel before
  pdl_trigger();  // the join may start up; it waits for this kernel's end
  const int c = blockIdx.x;
  TreeSeg w;
  TreeSegs<CutTc> sg;
  sg.begin(p, c);  // (without work the roles find nothing)
  const bool split = TMA && tm.split && p.hdr->cost >= p.hdr->live * (int64_t)p.nkv * SPLIT_COST;

  if (warp == 0) {
    // ---------------- products: one thread
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(TQ, D, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sR, 16, C::GROUP);
      const uint64_t dv0 = smem_desc_sw128(sR, 1024, C::GROUP);
      int slot = 0, phase = 0;  // of the next place in the ring
      int nq = 0;               // query tiles of the items before
      PerStream np{0, 0};       // weights of each stream so far
      PerStream no{0, 0};       // items of each stream so far
      // the next slot of the ring, once it is loaded
      auto next_slot = [&](int& at) {
        at = slot;
        if (!wait_1(bar(C::L_FULL + at), phase, p.err, abort)) return false;
        if (!TMA || tm.split) fence_proxy_async();  // what was copied by ordinary writes is read by the tensor core
        if (++slot == NST) slot = 0, phase ^= 1;
        return true;
      };
      // S_X = Q_tile K^T, K in slot `at`
      auto issue_s = [&](int x, int tile, int at) {
        const uint64_t da = dq0 + (uint64_t)((tile * C::TILE) >> 4), db = dk0 + (uint64_t)((at * C::TILE) >> 4);
        const uint32_t td = tmem + C::COL_S + x * TK;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_f16(td, da + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                     db + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
        tc_commit(bar(C::S_FULL + x));
      };
      // O_X += P_X V, V in slot `at`; the K steps (16 keys) that hold keys of the sequence, of
      // which `left` are left; fresh: the stream's first unit of the item, last: its last one
      auto issue_pv = [&](int x, int at, int left, bool fresh, bool last) {
        const int n = np[x];
        if ((fresh && no[x] > 0 && !wait_1(bar(C::O_EMPTY + x), (no[x] - 1) & 1, p.err, abort)) ||
            !wait_1(bar(C::P_HALF + x), n & 1, p.err, abort))
          return false;
        np.inc(x);
        const int ks = left >= TK ? TK / 16 : (left + 15) / 16;
        const uint64_t db = dv0 + (uint64_t)((at * C::TILE) >> 4);
        const uint32_t ta = tmem + C::COL_S + x * TK, to = tmem + C::COL_O + x * D;
        if (TMA && left < TK) fence_proxy_async();  // (the slots about the end may be ordinary writes)
        // (the first half's products run while the other half's weights are formed)
#pragma unroll 1
        for (int k0 = 0; k0 < TK / 16; k0 += TK / 32) {
          if (k0 > 0 && !wait_1(bar(C::P_FULL + x), n & 1, p.err, abort)) return false;
          tc_fence_after();
#pragma unroll 4
          for (int kk = k0; kk < min(ks, k0 + TK / 32); ++kk) {
            const uint64_t dv = db + (uint64_t)((kk * 2 * C::GROUP) >> 4);
            tc_mma_f16_ts(to, ta + kk * 16, dv, idesc_pv, (!fresh || kk > 0) ? 1u : 0u);
            tc_mma_f16_ts(to, ta + kk * 16 + 8, dv, idesc_pv, 1u);
          }
        }
        if (last) {
          tc_commit(bar(C::O_FULL + x));
          no.inc(x);
        }
        return true;
      };
      auto free_slot = [&](int at) { tc_commit(bar(C::L_EMPTY + at)); };
      bool good = true;
      while (good && sg.next(p, w)) {
        const int nt = w.t1 - w.t0, len = w.q.len - w.t0 * TK;
        const bool two = w.rows > TQ;
        const int ta = nq & 1, tb = two ? ta ^ 1 : ta;  // the streams' query tiles
        for (int i = 0; i < (two ? 2 : 1) && good; ++i, ++nq)
          good = wait_1(bar(C::Q_FULL + (nq & 1)), (nq >> 1) & 1, p.err, abort);
        if (!TMA || !tm.q_tma) fence_proxy_async();
        tc_fence_after();
        int k, v;
        if (two) {
          // halves of the rows: PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1)
          good = good && next_slot(k);
          if (!good) break;
          issue_s(0, ta, k);
          issue_s(1, tb, k);
          free_slot(k);
          auto free_queries = [&]() {
            tc_commit(bar(C::Q_EMPTY + ta));
            tc_commit(bar(C::Q_EMPTY + tb));
          };
          if (nt == 1) free_queries();
#pragma unroll 1
          for (int j = 0; j < nt; ++j) {
            const bool more = j + 1 < nt;
            good = next_slot(v) && issue_pv(0, v, len - j * TK, j == 0, !more) && (!more || next_slot(k));
            if (!good) break;
            if (more) issue_s(0, ta, k);
            good = issue_pv(1, v, len - j * TK, j == 0, !more);
            if (!good) break;
            free_slot(v);
            if (more) {
              issue_s(1, tb, k);
              free_slot(k);
              if (j + 2 == nt) free_queries();
            }
          }
        } else {
          // units in turn: S_A(0), S_B(1), PV_A(0), S_A(2), PV_B(1), S_B(3), ..
#pragma unroll 1
          for (int i = 0; i < nt + 2 && good; ++i) {
            const int x = i & 1;
            if (i >= 2) {
              good = next_slot(v) && issue_pv(x, v, len - (i - 2) * TK, i < 4, i >= nt);
              if (!good) break;
              free_slot(v);
            }
            if (i < nt) {
              good = next_slot(k);
              if (!good) break;
              issue_s(x, ta, k);
              free_slot(k);
              if (i == nt - 1) tc_commit(bar(C::Q_EMPTY + ta));
            }
          }
        }
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  } else if (TMA && warp == 1) {
    // ---------------- K and V: a lane finds the page of one box and asks for it
    int nl = 0, nkey = 0;  // slots, units so far
    const int nbox = TK >> tm.shift;
    bool good = true;
    while (good && sg.next(p, w)) {
      const int nt = w.t1 - w.t0, x = w.h * (int)p.s_head;
      const bool two = w.rows > TQ;
      const int32_t* table = p.table + (int64_t)w.q.s * p.ld_table;
      // page and slot of this lane's box of unit j, requested one unit ahead
      int pg = 0, slot = 0;
      bool on = false;
      auto peek = [&](int j) {
        const int key = (w.t0 + j) * TK + (lane << tm.shift);  // (lengths end well below 2^31)
        on = j < nt && lane < nbox && key < w.q.len;
        if (on) {
          const int e = key / p.page_size;
          slot = key - e * p.page_size;
          pg = table[e];
        }
      };
      peek(0);
      // place of this lane's box of the newest unit, of the one before; page n_pages: zeros
      int2 now = make_int2(p.n_pages, 0), before = now;
#pragma unroll 1
      for (int pos = 0; pos < 2 * nt; ++pos) {
        const bool newest = two || pos == 2 * nt - 1;  // of V: of the newest unit
        const bool is_v = two ? pos & 1 : newest || (pos > 0 && (pos & 1) == 0);
        if (is_v && split) continue;
        const int n = nl + pos, s = n % NST;
        const int j = newest ? pos / 2 : is_v ? (pos - 2) / 2 : (pos + 1) / 2;
        const int left = w.q.len - (w.t0 + j) * TK;  // keys of the sequence from here on
        uint32_t boxes = 0;
        if (!is_v) {
          const bool ok = on && pg >= 0 && pg < p.n_pages;
          if (on && !ok) record_error(p.err, kErrIndex);
          before = now;
          now = ok ? make_int2(pg, slot >> 3) : make_int2(p.n_pages, 0);
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
            const uint32_t bits = __ballot_sync(0xffffffffu, key < left && ((boxes >> (key >> tm.shift)) & 1u));
            if (lane == 0) see[at * 4 + i] = bits;
          }
          if (lane == 0) mbar_arrive(bar(C::SEE + at));
        }
        // K: the boxes with keys of the sequence, whole (its scores behind the end are overwritten).
        // V: as far as its products read, zeros behind the end (a NaN there would not be masked by a
        // weight of 0): the box with the end 8 slots at a time, the 8 with the end by threads.
        const int box = 1 << tm.shift, used = is_v ? used_rows(left) : min(TK, left);
        const bool cut = is_v && left < TK && (left & 7);  // the end is inside of 8 slots
        if (lane == 0) {
          const int others = (tm.split ? NLOAD : NFILL) - 1 - (cut ? 32 : 0);
          if (others > 0) mbar_arrive_n(full, others);
          const int rows = is_v ? used - (cut ? 8 : 0) : min(TK, (left + box - 1) & -box);
          mbar_arrive_expect_tx(full, (uint32_t)(rows * D * 2));
        }
        __syncwarp();
        const int2 b = !is_v || newest ? now : before;
        const uint32_t dst = sR + s * C::TILE;
        const int part = is_v && left < TK && (left & (box - 1)) ? left >> tm.shift : nbox;
        if ((lane << tm.shift) < used && lane != part)
          tma_load_5d(dst + ((lane << tm.shift) >> 3) * C::GROUP, is_v ? &tm.v[0] : &tm.k, x, 0, 0, b.y, b.x, full);
        if (part < nbox) {
          const int pb = __shfl_sync(0xffffffffu, b.x, part), gb = __shfl_sync(0xffffffffu, b.y, part);
          const int g0 = part << (tm.shift - 3);  // the box's first group of the tile
          const int edge = left >> 3;             // the group with the end, if it is inside one
          const int g = g0 + lane;
          if (lane < (box >> 3) && g * 8 < used && !(cut && g == edge))
            tma_load_5d(dst + g * C::GROUP, &tm.v[1], x, 0, 0, gb + lane, g < edge ? pb : p.n_pages, full);
          if (cut) {
#pragma unroll
            for (int i = 0; i < C::CH / 4; ++i) {
              const int r = (i * 32 + lane) / C::CH, ch = lane % C::CH;
              const bool ok = pb < p.n_pages && edge * 8 + r < left;
              const int64_t from = ok ? pb * p.s_page + ((gb + edge - g0) * 8 + r) * p.s_tok + x + ch * 8 : 0;
              cp_async16(dst + edge * C::GROUP + (ch >> 3) * 1024 + r * 128 + (((ch & 7) ^ r) << 4),
                         static_cast<const bf16*>(p.v) + from, ok);
            }
            cp_async_arrive(full);
          }
        }
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else if (TMA && warp < 4 && (warp == 3 || split)) {
    // ---------------- Q, and V row by row
    const int pw = warp - 2;
    constexpr int NR = TQ / NLOAD;  // rows per lane: 32 (NR pw + i) + lane
    bool good = true;
    int nq = 0, nl = 0;  // query tiles, slots so far
    while (good && sg.next(p, w)) {
      if (warp == 3 && !tm.q_tma) good = copy_q<D>(p, w, sb, 0, 1, nq, abort);
      // (rows behind the item's last one: any queries)
      for (int x = 0; warp == 3 && tm.q_tma && x * TQ < w.rows && good; ++x, ++nq) {
        const int tile = nq & 1;
        good = nq < 2 || wait_w(bar(C::Q_EMPTY + tile), ((nq >> 1) - 1) & 1, p.err, abort);
        if (good && lane == 0) {
          mbar_arrive_expect_tx(bar(C::Q_FULL + tile), C::TILE);
          tma_load_4d(sQ + tile * C::TILE, &tm.q, w.h * p.G * D, 0,
                      w.q.row + (w.b * CutTc::ROWS + x * TQ) / p.G, 0, bar(C::Q_FULL + tile));
        }
        __syncwarp();
      }
      if (!split) continue;
      const int nt = w.t1 - w.t0, ahead = w.rows > TQ ? 1 : min(2, nt);
      const int64_t table = (int64_t)w.q.s * p.ld_table;
      // places of this lane's tokens of a unit, requested one unit ahead
      int64_t off[NR];
      auto find = [&](int j) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int key = (w.t0 + j) * TK + (pw * NR + i) * 32 + lane;  // (lengths end well below 2^31)
          off[i] = -1;
          if (j < nt && key < w.q.len) {
            const int e = key / p.page_size, page = p.table[table + e];  // (a bad one is reported with K)
            if (page >= 0 && page < p.n_pages)
              off[i] = page * p.s_page + (key - e * p.page_size) * p.s_tok + w.h * p.s_head;
          }
        }
      };
      find(0);
#pragma unroll 1
      for (int j = 0; j < nt && good; ++j) {
        const int n = nl + (j < nt - ahead ? ahead + 2 * j : nt + j), s = n % NST;  // V_j's place
        good = n < NST || wait_w(bar(C::L_EMPTY + s), (n / NST - 1) & 1, p.err, abort);
        if (!good) break;
        int64_t now[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) now[i] = off[i];
        find(j + 1);
#pragma unroll
        for (int i = 0; i < NR; ++i)
          copy_rows<D>(sR + s * C::TILE, (pw * NR + i) * 32, static_cast<const bf16*>(p.v), now[i], C::GROUP, 1024);
        cp_async_arrive(bar(C::L_FULL + s));
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else if (!TMA && warp < 4 && (warp & 1)) {
    // ---------------- Q, K and V row by row: a lane finds one row's place, all copy it
    const int pw = warp >> 1;
    constexpr int NR = TQ / NLOAD;  // rows per lane: 32 (NR pw + i) + lane
    int nl = 0, nkey = 0, nq = 0;  // slots, units, query tiles so far
    bool good = true;
    while (good && sg.next(p, w)) {
      const int nt = w.t1 - w.t0;
      const bool two = w.rows > TQ;
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
      good = copy_q<D>(p, w, sb, pw, 2, nq, abort);
      if (!good) break;
      int64_t now[NR] = {}, before[NR] = {};  // this lane's places of the newest unit and the one before it
#pragma unroll 1
      for (int pos = 0; pos < 2 * nt; ++pos) {
        const bool newest = two || pos == 2 * nt - 1;  // of V: of the newest unit
        const bool is_v = two ? pos & 1 : newest || (pos > 0 && (pos & 1) == 0);
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
          peek((two ? pos / 2 : (pos + 1) / 2) + 1);
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
#pragma unroll
        for (int i = 0; i < NR; ++i)
          copy_rows<D>(sR + s * C::TILE, (pw * NR + i) * 32, static_cast<const bf16*>(is_v ? p.v : p.k),
                       !is_v || newest ? now[i] : before[i], C::GROUP, 1024);
        cp_async_arrive(bar(C::L_FULL + s));
      }
      nl += 2 * nt;
    }
    if (!good) *abort = 1;
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp >= 4) {
    // ---------------- softmax: a thread per row; warps of stream A, then of stream B
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the stream
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + C::COL_S + x * TK + lane_base, t_o = tmem + C::COL_O + x * D + lane_base;
    bool good = true;
    int nx = 0;    // units of this stream so far
    int ko = 0;    // items of this stream so far
    int km = 0;    // items joined from both streams so far
    int nkey = 0;  // units of the items before
    while (good && sg.next(p, w)) {
      const int nt = w.t1 - w.t0, key0 = nkey;
      nkey += nt;
      const bool two = w.rows > TQ;
      if (x == 1 && !two && nt < 2) continue;
      const int row = (two ? x * TQ : 0) + r;  // of the block
      const bool live = row < w.rows;
      const bool work = row - lane < w.rows;   // the warp has a row
      const int rr = w.b * CutTc::ROWS + (live ? row : 0);
      const int tok = rr / p.G, head = w.h * p.G + rr - tok * p.G;
      const uint32_t* mask = p.mask + (int64_t)(w.q.row + tok) * TREE_WORDS;
      const int ctx = w.q.len - w.q.m;         // tokens before the draft
      float m = -INFINITY, l = 0.0f;
      const int j0 = two ? 0 : x;
      for (int j = j0; j < nt; j += two ? 1 : 2, ++nx) {
        const int kv0 = (w.t0 + j) * TK;
        if (!wait_w(bar(C::S_FULL + x), nx & 1, p.err, abort)) {
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
          // the keys of the unit that this row sees
          uint32_t vis[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) vis[i] = see[at * 4 + i];
          if (kv0 + TK > ctx || (vis[0] & vis[1] & vis[2] & vis[3]) != ~0u) {
            // Few units have hidden keys: their scores are overwritten first.
            if (kv0 + TK > ctx)
#pragma unroll
              for (int i = 0; i < 4; ++i) vis[i] &= tree_window(mask, kv0 + 32 * i - ctx);
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
            if (j > j0) {  // (the PV before is complete: the scores were formed behind it)
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
            weights(s, p.sl2, shift, sum);
            tmem_st32(t_s + i * 32, s[0]);
            tmem_st32(t_s + i * 32 + 32, s[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();  // the warp's stores are done: one arrival for the warp
            if (lane == 0) mbar_arrive(bar((i == 0 ? C::P_HALF : C::P_FULL) + x));
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        } else if (lane == 0) {
          mbar_arrive(bar(C::P_HALF + x));
          mbar_arrive(bar(C::P_FULL + x));
        }
        __syncwarp();
      }
      if (!good) break;
      // ---- the CTA's units of the item are done
      if (!wait_w(bar(C::O_FULL + x), ko++ & 1, p.err, abort)) {
        good = false;
        break;
      }
      tc_fence_after();
      const bool join = !two && nt > 1;  // B's sums go to A
      if (join && x == 1) {
        sml[2 * r] = m;
        sml[2 * r + 1] = l;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::ML));
        continue;
      }
      float fa = 1.0f, fb = 0.0f;
      if (join) {
        if (!wait_w(bar(C::ML), km++ & 1, p.err, abort)) {
          good = false;
          break;
        }
        tc_fence_after();
        const float mb = sml[2 * r], lb = sml[2 * r + 1], M = fmaxf(m, mb);
        // (no reference: no key or only scores of -infinity, sum 0, or NaN, which stays)
        fa = m > -INFINITY ? exp2f(m - M) : 1.0f;
        fb = mb > -INFINITY ? exp2f(mb - M) : 1.0f;
        l = l * fa + lb * fb;
        m = M;
      }
      if (work) {
        const bool whole = sg.whole(w);
        const float inv = whole ? 1.0f / l : 1.0f;  // (no score: 0 / 0)
        fa *= inv;
        fb *= inv;
        bf16* out = static_cast<bf16*>(p.o) + (w.q.row + tok) * p.ld_o + (int64_t)head * D;
        const int part = tree_part(c, sg.begin_at, w.at);
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i) {
          uint32_t o[16], o2[16];
          tmem_ld16(t_o + i * 16, o);
          if (join) tmem_ld16(t_o + D + i * 16, o2);
          tmem_ld_wait();
          tmem_regs_ready(o);
          tmem_regs_ready(o2);
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            f[e] = __uint_as_float(o[e]) * fa;
            if (join) f[e] = fmaf(__uint_as_float(o2[e]), fb, f[e]);
          }
          if (live && whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(out + i * 16 + e) =
                  make_uint4(pack_bf16x2(f[e], f[e + 1]), pack_bf16x2(f[e + 2], f[e + 3]),
                             pack_bf16x2(f[e + 4], f[e + 5]), pack_bf16x2(f[e + 6], f[e + 7]));
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *tree_part_at(p, part, D, (i * 16 + e) / 4, row) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          }
          __syncwarp();  // (the loads are the whole warp's)
        }
        if (live && whole && p.lse != nullptr)
          p.lse[(int64_t)(w.q.row + tok) * p.nq + head] = (m + log2f(l)) * LN2;
        if (live && !whole) p.ml[(int64_t)part * p.rows + row] = make_float2(m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::O_EMPTY + x));
        if (join) mbar_arrive(bar(C::O_EMPTY + 1));
      }
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  return fn;
}

// bf16 tensor map with 128-byte swizzle and zero fill; strides (bytes) of the dimensions behind
// the first.
bool encode_map(CUtensorMap* tm, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const uint32_t es[5] = {1, 1, 1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the TMA unit can copy: pages of a multiple of 8 slots (and sizes that its numbers hold).
bool tma_ok(const TreeParams& p, int d) {
  const int64_t most = (int64_t)1 << 31;
  return p.page_size % 8 == 0 && (p.nkv - 1) * p.s_head + d < most && p.s_page < most * 128 &&
         8 * p.s_tok < most * 128;
}

bool encode_pool(CUtensorMap* tm, const void* pool, const TreeParams& p, int d, int shift) {
  const uint64_t es = 2;
  const uint64_t dims[5] = {(uint64_t)((p.nkv - 1) * p.s_head + 64), 8, (uint64_t)(d / 64),
                            (uint64_t)(p.page_size / 8), (uint64_t)p.n_pages};
  const uint64_t strides[4] = {(uint64_t)p.s_tok * es, 64 * es, 8 * (uint64_t)p.s_tok * es,
                               (uint64_t)(p.n_pages > 1 ? p.s_page : 8) * es};
  const uint32_t box[5] = {64, 8, (uint32_t)(d / 64), 1u << (shift - 3), 1};
  return encode_map(tm, pool, 5, dims, strides, box);
}

template <int D, bool TMA>
mgb_status launch_k(const TreeParams& p, const PoolMaps& tm, cudaStream_t st) {
  using C = Cfg<D>;
  auto k = tree_kernel<D, TMA>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const mgb_status s = launch_pdl(k, CutTc::RANGES, NTHREADS, C::SMEM, st, tm, p);
  return s != MGB_OK ? s : tree_join<bf16, D>(p, CutTc::RANGES, st);
}

template <int D>
mgb_status launch_d(const TreeParams& p, cudaStream_t st) {
  PoolMaps tm{};
  if (!tma_ok(p, D)) return launch_k<D, false>(p, tm, st);
  // queries: the heads of a group next to each other, tokens ld_q apart; 128 rows are whole tokens
  tm.q_tma = 128 % p.G == 0;
  if (tm.q_tma) {
    const uint64_t dims[4] = {(uint64_t)(p.nkv - 1) * p.G * D + 64, (uint64_t)p.G, (uint64_t)p.tokens, D / 64};
    const uint64_t strides[3] = {2 * D, 2 * (uint64_t)(p.tokens > 1 ? p.ld_q : p.nq * D), 128};
    const uint32_t box[4] = {64, (uint32_t)p.G, (uint32_t)(128 / p.G), D / 64};
    if (!encode_map(&tm.q, p.q, 4, dims, strides, box)) return MGB_ERR_CUDA;
  }
  while (tm.shift < 7 && p.page_size % (2 << tm.shift) == 0) ++tm.shift;
  tm.split = tm.shift <= (D == 64 ? 6 : 4) && (int64_t)p.tokens * p.G <= (int64_t)p.n * TQ;
  if (!encode_pool(&tm.k, p.k, p, D, tm.shift) || !encode_pool(&tm.v[0], p.v, p, D, tm.shift) ||
      !encode_pool(&tm.v[1], p.v, p, D, 3))
    return MGB_ERR_CUDA;
  return launch_k<D, true>(p, tm, st);
}

}  // namespace

mgb_status attention_tree_bf16(const TreeParams& p, int d, cudaStream_t st) {
  return d == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace mgb
