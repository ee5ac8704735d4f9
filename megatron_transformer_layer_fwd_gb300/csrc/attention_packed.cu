// Attention over packed sequences of different lengths, bf16, on the tensor
// cores (tcgen05): O_h = softmax(Q_h K_g^T / sqrt(d)) V_g within each sequence,
// optionally causal, and its log-sum-exp.
//
// A work item is 256 query rows of one (sequence, head), in two tiles A and B
// of 128 that take turns on the tensor core. Per 128 keys the MMA thread issues
// PV_A(j), S_A(j+1), PV_B(j), S_B(j+1); while tile A's scores are turned into
// weights, tile B's two products run. TMEM (512 columns) holds the scores and O_A,
// O_B; a tile's weights P (bf16 pairs) overwrite scores already read and are
// read from there by PV.
//
// Each tile goes round a chain: scores complete - softmax - weights ready -
// PV and the next scores (16 products of 64 cycles) - scores complete. Two
// tiles cover the tensor core only as far as that chain is short (measured at
// D = 128, in cycles: softmax 1040, to the MMA thread 170, products 1270; the
// tensor core is busy for 2048 of the 2500). What shortens it:
//   - the row maximum is not on it: weights are formed in log2 units with the
//     reference maximum so far, and only if a row's then sum to more than
//     SUM_LIMIT (each is at most the sum) does its warp take the maximum, move the
//     reference, rescale the sums and the O rows, and form the weights again;
//   - one thread issues all products: the waits and votes of a whole warp
//     between two tiles' products took 900 cycles in which the tensor core ran
//     dry; and a ring stage holds V_j and K_{j+1}, which the same round needs, so
//     a round has one wait and one release for both;
//   - the exponentials are spread between the other steps in a fixed order
//     (form() below: 1340 -> 1020 cycles), as only one warp per scheduler is
//     at work on a tile. (Two threads per row, 16 softmax warps, took 1070 and a
//     barrier.)
// Where TMEM has room the next scores are formed before the weights are done,
// which takes the products off the chain: at D = 64 in three score buffers that
// the tasks of both tiles take in turn, and for an item whose tile B is empty
// in the two buffers by turns.
//
// Measured in a captured graph (causal but the last): two sequences of 4012 and 4165
// tokens, 32 / 8 heads: D = 128 180 us, 1530 TFLOP/s (called one by one from the
// host 192 us, 1430); 2 x 4096, D = 64 120 us, 1150 TFLOP/s; 8 x 1024, D = 128, no
// mask 96 us, 1440 TFLOP/s.
//
// Items come from a list that the prepare kernel derives from the row offsets
// (longest first, so that the snake order of item_index evens the CTAs out);
// lengths stay on the device. Every layer of a model uses the same list.
//
// Tiles that reach past their sequence's end hold rows of the next sequence,
// whose values must not change a result. A key there is masked before the
// softmax (by selection, so NaN scores vanish too) and a query row's products
// stay in its own TMEM lane, which is not stored; but a weight of zero times a
// NaN value is NaN. So the PV product of the last tile takes only the K steps
// (16 keys) that hold keys of the sequence, and the softmax warps clear the up
// to 15 value rows behind the end of the last step in shared memory first.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mgb {

CUresult tmap_encode_bf16_2d(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer,
                             int64_t ld, uint32_t box_inner, uint32_t box_outer);

namespace {

constexpr int TQ = 128;         // query rows per tile (TMEM lanes)
constexpr int TK = 128;         // keys per KV tile
constexpr int NSOFTW = 4;       // softmax warps per tile
constexpr int NTHREADS = 320;   // MMA warp, producer warp, 2 x 4 softmax warps
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float SUM_LIMIT = 8192.0f;  // of a row's weights in a tile
// Reference (log2 units) up to which the fused scale-and-subtract is off by a factor of
// at most 2, which all weights of a reference share, so that it cancels
constexpr float REF_LIMIT = 16777216.0f;

template <int D>
struct Cfg2 {
  static constexpr int NB = D == 64 ? 3 : 2;            // score buffers in TMEM
  static constexpr int NST = D == 64 ? 4 : 2;           // ring stages: V_j and K_{j+1}
  static constexpr int KB = D / 64;                     // 64-wide d boxes
  static constexpr int BOX = 128 * 128;                 // bytes of one [128][64] box
  static constexpr int Q_BYTES = TQ * D * 2;
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int OFF_Q = 0;                       // [tile]
  static constexpr int OFF_K = 2 * Q_BYTES;             // [stage]
  static constexpr int OFF_V = OFF_K + NST * KV_BYTES;  // [stage]
  static constexpr int OFF_BAR = OFF_V + NST * KV_BYTES;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;     // barriers, alignment slack
  static constexpr int COL_S = 0;                       // score buffers
  static constexpr int COL_O = NB * TK;                 // O_A, then O_B at + D
  static constexpr int TMEM_COLS = 512;
  static_assert(COL_O + 2 * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  // Barriers (8 bytes each). A waiter sees every phase of a barrier or knows that
  // at most one is outstanding (parity). Up to two tasks of a tile are under way,
  // so the barriers of scores and weights take turns by the tile's task count.
  static constexpr int Q_FULL = 0;              // the item's Q tiles loaded          (tx)
  static constexpr int Q_EMPTY = 1;             // the item's last S product done     (commit)
  static constexpr int L_FULL = 2;              // [stage] loaded                    (tx)
  static constexpr int L_EMPTY = L_FULL + NST;  // [stage] products with it done     (commit)
  static constexpr int S_FULL = L_EMPTY + NST;  // [tile][task & 1] scores complete  (commit)
  static constexpr int P_FULL = S_FULL + 4;     // [tile][task & 1] weights written  (4: one per warp)
  static constexpr int O_FULL = P_FULL + 4;     // [tile] the item's last PV done     (commit)
  static constexpr int O_EMPTY = O_FULL + 2;    // [tile] O read out                 (4: one per warp)
  static constexpr int N_BAR = O_EMPTY + 2;
  static_assert(N_BAR * 8 <= 232, "barriers");
};

struct Params {
  int nq, causal, tokens;
  uint64_t m_nq, m_group;  // div_by of nq and of the group size nq / nkv
  const PackedHeader* hdr;
  const int4* list;  // entries of 256 rows
  bf16* o;
  int64_t ld_o;
  int wide;  // o's rows are 32-byte aligned
  float* lse;
  int* err;
  float sl2;  // log2(e) / sqrt(d)
};

// A number for each of the tiles A (0) and B (1); selected, not indexed, so that
// it stays in registers.
struct PerTile {
  int a, b;
  __device__ int operator[](int x) const { return x ? b : a; }
  __device__ void inc(int x) { (x ? b : a) += 1; }
};

// An item: 256 query rows of one (sequence, head).
struct Job {
  int a, len;    // the sequence's first row and length
  int q, h;      // first query row in it (tile B: + 128), head
  PerTile n;     // key tiles (B 0, or at least A's)
};

// i / d for i < 2^31 by one high product; `m` = 2^64 / d rounded up, 0 for d = 1.
__device__ __forceinline__ int div_by(int i, uint64_t m) {
  return m == 0 ? i : (int)__umul64hi((uint64_t)(uint32_t)i, m);
}

// The item a CTA takes in its k-th round: snake order over the list, as in the
// dense forward.
__device__ __forceinline__ int item_index(int k) {
  const int g = (int)gridDim.x, c = (int)blockIdx.x;
  return k * g + ((k & 1) ? g - 1 - c : c);
}

// A CTA's items in order, the same for every role: item i is entry i / nq of the
// list and head i % nq (the heads of a group next to each other share their keys
// and values in L2). The next item's entry is requested one item ahead.
struct Jobs {
  int k, n_items;
  int i, h;  // next item, its head
  int4 e;    // its entry
  Job w;
  __device__ void fetch(const Params& p) {
    i = item_index(k++);
    if (i < n_items) {
      const int u = div_by(i, p.m_nq);
      h = i - u * p.nq;
      e = p.list[u];
    }
  }
  __device__ bool begin(int items, const Params& p) {
    n_items = items;
    k = 0;
    fetch(p);
    return next(p);
  }
  // false: no more items
  __device__ bool next(const Params& p) {
    if (i >= n_items) return false;
    w.a = e.x;
    w.len = e.y;
    w.q = e.z;
    w.h = h;
    auto tiles = [&](int q0) {
      const int end = p.causal ? min(w.len, q0 + TQ) : w.len;
      return q0 < w.len ? (end + TK - 1) / TK : 0;
    };
    w.n = {tiles(w.q), tiles(w.q + TQ)};
    fetch(p);
    return true;
  }
};

// The steps of the weights in an order that the compiler keeps (volatile): see
// the softmax warps.
__device__ __forceinline__ void v_fma2(float& r0, float& r1, uint32_t a0, uint32_t a1, float b, float c) {
  asm volatile(
      "{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " mov.b64 c, {%5, %5};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r0), "=f"(r1)
      : "r"(a0), "r"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void v_ex2(float& x) {
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
}
__device__ __forceinline__ void v_add2(float& r0, float& r1, float a0, float a1) {
  asm volatile(
      "{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "+f"(r0), "+f"(r1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint32_t v_pack(float lo, float hi) {
  uint32_t r;
  asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 bytes to a 32-byte aligned address: a whole sector by one store.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Whole warp: waits for the phase, for a bounded time and only while no role has
// given up; the same result in every lane. The usual case, a phase already
// complete, is one try and one vote.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, int* err,
                                           volatile int* abort) {
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

// The same for one thread.
__device__ __forceinline__ bool wait_phase_1(uint32_t bar, uint32_t parity, int* err,
                                             volatile int* abort) {
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

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg2<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t sQ = sb + C::OFF_Q, sK = sb + C::OFF_K, sV = sb + C::OFF_V;
  constexpr int NB = C::NB, NST = C::NST;
  auto bar = [&](int which) { return sb + C::OFF_BAR + 8 * which; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 240);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 244);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // the list and the inputs may come from the kernel before
  const int n_items = p.hdr->entries * p.nq;
  if ((int)blockIdx.x >= n_items) return;

  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < C::N_BAR; ++i)
      mbar_init(bar(i), (i >= C::P_FULL && i < C::O_FULL) || i >= C::O_EMPTY ? NSOFTW : 1);
    fence_mbar_init();
    *abort = 0;
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 1) {
    // ---------------- producer (one thread): per item the Q tiles, then the
    // stages (K_0), (V_0, K_1), .., (V_last)
    if (elect_one()) {
      int nl = 0;  // stages loaded so far
      int k = 0;   // items so far
      bool good = true;
      Jobs js;
      for (bool more = js.begin(n_items, p); more && good; more = js.next(p), ++k) {
        const Job& w = js.w;
        const int xkv = div_by(w.h, p.m_group) * D;
        // the item lies in the tensors (TMA x coordinates are multiples of 64)
        if (!dcheck(w.a >= 0 && w.q >= 0 && w.q < w.len && w.len <= p.tokens - w.a && w.h < p.nq,
                    p.err) ||
            (k >= 1 && !wait_phase_1(bar(C::Q_EMPTY), (k - 1) & 1, p.err, abort))) {
          good = false;
          break;
        }
        mbar_arrive_expect_tx(bar(C::Q_FULL), (w.n[1] > 0 ? 2 : 1) * C::Q_BYTES);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (w.n[x] > 0)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_2d(sQ + x * C::Q_BYTES + kb * C::BOX, &tmQ, w.h * D + kb * 64, w.a + w.q + x * TQ,
                          bar(C::Q_FULL));
        const int nt = max(w.n[0], w.n[1]);
        for (int j = 0; j <= nt && good; ++j, ++nl) {
          const int s = nl % NST;
          if (nl >= NST && !wait_phase_1(bar(C::L_EMPTY + s), ((nl - NST) / NST) & 1, p.err, abort)) {
            good = false;
            break;
          }
          const uint32_t full = bar(C::L_FULL + s), dk = sK + s * C::KV_BYTES,
                         dv = sV + s * C::KV_BYTES;
          mbar_arrive_expect_tx(full, (j > 0 && j < nt ? 2 : 1) * C::KV_BYTES);
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb) {
            if (j > 0) tma_load_2d(dv + kb * C::BOX, &tmV, xkv + kb * 64, w.a + (j - 1) * TK, full);
            if (j < nt) tma_load_2d(dk + kb * C::BOX, &tmK, xkv + kb * 64, w.a + j * TK, full);
          }
        }
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------- MMA issuer: one thread
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(TQ, D, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sK, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sV, C::BOX, 1024);
      int nl = 0;             // stages consumed so far
      PerTile nt_ = {0, 0};   // tasks of each tile whose PV products are issued
      PerTile ns = {0, 0};    // .. whose S products are issued
      PerTile no = {0, 0};    // items of each tile so far
      bool good = true;
      Jobs js;
      int k = 0;
      for (bool more = js.begin(n_items, p); more && good; more = js.next(p), ++k) {
        const Job& w = js.w;
        const int n0 = w.n[0], n1 = w.n[1], nt = max(n0, n1), st0 = nl;
        // S_X(j) = Q_X K_j^T into score buffer buf (stage st)
        auto issue_s = [&](int x, int st, int buf) {
          const uint64_t da = dq0 + (x ? (uint64_t)(C::Q_BYTES >> 4) : 0);
          const uint64_t db = dk0 + (uint64_t)((st % NST * C::KV_BYTES) >> 4);
          const uint32_t td = tmem + C::COL_S + buf * TK;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::BOX + (kk & 3) * 32;
            tc_mma_f16(td, da + (uint64_t)(off >> 4), db + (uint64_t)(off >> 4), idesc_s, kk > 0);
          }
          tc_commit(bar(C::S_FULL + 2 * x + (ns[x] & 1)));
          ns.inc(x);
        };
        // O_X += P_X V_j, the K steps (16 keys) that hold keys of the sequence
        auto issue_pv = [&](int x, int j, int st, int buf) {
          // O_X of the item before read out before this item's first PV_X
          if ((j == 0 && no[x] >= 1 &&
               !wait_phase_1(bar(C::O_EMPTY + x), (no[x] - 1) & 1, p.err, abort)) ||
              !wait_phase_1(bar(C::P_FULL + 2 * x + (nt_[x] & 1)), (nt_[x] >> 1) & 1, p.err, abort))
            return false;
          nt_.inc(x);
          tc_fence_after();
          const int left = w.len - j * TK;
          const int ks = left >= TK ? TK / 16 : (left + 15) / 16;
          const uint64_t db = dv0 + (uint64_t)((st % NST * C::KV_BYTES) >> 4);
          const uint32_t ta = tmem + C::COL_S + buf * TK, to = tmem + C::COL_O + x * D;
          if (ks == TK / 16) {
#pragma unroll
            for (int kk = 0; kk < TK / 16; ++kk)
              tc_mma_f16_ts(to, ta + kk * 8, db + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                            (j > 0 || kk > 0) ? 1u : 0u);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < ks; ++kk)
              tc_mma_f16_ts(to, ta + kk * 8, db + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                            (j > 0 || kk > 0) ? 1u : 0u);
          }
          if (j == w.n[x] - 1) {
            tc_commit(bar(C::O_FULL + x));
            no.inc(x);
          }
          return true;
        };
        // stage of K_j and V_{j-1}, once loaded
        auto ready = [&](int j) {
          return wait_phase_1(bar(C::L_FULL + (st0 + j) % NST), ((st0 + j) / NST) & 1, p.err, abort);
        };
        auto release = [&](int j) { tc_commit(bar(C::L_EMPTY + (st0 + j) % NST)); };
        nl += nt + 1;
        if (!wait_phase_1(bar(C::Q_FULL), k & 1, p.err, abort) || !ready(0)) {
          good = false;
          break;
        }
        tc_fence_after();
        if (n1 == 0) {
          // tile A alone: its scores take turns in buffers 0 and 1, one task ahead
          issue_s(0, st0, 0);
          release(0);
          if (nt == 1) tc_commit(bar(C::Q_EMPTY));
          for (int j = 0; j < nt; ++j) {
            if (!ready(j + 1)) {
              good = false;
              break;
            }
            if (j + 1 < nt) {
              tc_fence_after();
              issue_s(0, st0 + j + 1, (j + 1) & 1);
              if (j + 2 == nt) tc_commit(bar(C::Q_EMPTY));
            }
            if (!issue_pv(0, j, st0 + j + 1, j & 1)) {
              good = false;
              break;
            }
            release(j + 1);
          }
        } else if (NB == 2) {
          issue_s(0, st0, 0);
          issue_s(1, st0, 1);
          release(0);
          if (nt == 1) tc_commit(bar(C::Q_EMPTY));
          for (int j = 0; j < nt; ++j) {
            if (!ready(j + 1)) {
              good = false;
              break;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!good || j >= w.n[x]) continue;
              good = issue_pv(x, j, st0 + j + 1, x);
              if (good && j + 1 < w.n[x]) issue_s(x, st0 + j + 1, x);
            }
            if (!good) break;
            release(j + 1);
            if (j + 2 == nt) tc_commit(bar(C::Q_EMPTY));
          }
        } else {
          // Three buffers in turn: the scores of task t + 3 follow task t's PV, so
          // a tile's next scores are there when its weights are written. After
          // PV_A(j) that is S_B(j + 1), after PV_B(j) S_A(j + 2), or, if A ends
          // one step before B, the last S_B.
          issue_s(0, st0, 0);
          issue_s(1, st0, 1);
          release(0);
          if (nt == 1) tc_commit(bar(C::Q_EMPTY));
          if (nt > 1) {
            good = ready(1);
            tc_fence_after();
            if (good) issue_s(n0 > 1 ? 0 : 1, st0 + 1, 2);
            if (n0 == 1) tc_commit(bar(C::Q_EMPTY));
          }
          int b0 = 0, b1 = 1, b2 = 2;  // buffers of tasks t, t + 1, t + 2
          for (int j = 0; j < nt && good; ++j) {
            if (j + 1 == nt && !ready(nt)) {  // (earlier stages: before their S products)
              good = false;
              break;
            }
            if (j < n0) {
              good = issue_pv(0, j, st0 + j + 1, b0);
              if (!good) break;
              if (j + 1 < n0) {
                issue_s(1, st0 + j + 1, b0);
                if (j + 1 == n1 - 1) tc_commit(bar(C::Q_EMPTY));
              }
              const int b = b0;
              b0 = b1; b1 = b2; b2 = b;
            }
            good = issue_pv(1, j, st0 + j + 1, b0);
            if (!good) break;
            release(j + 1);
            if (j + 2 < n0 || (j + 2 == n0 && n1 > n0)) {
              good = ready(j + 2);
              if (!good) break;
              tc_fence_after();
              if (j + 2 < n0) {
                issue_s(0, st0 + j + 2, b0);
              } else {
                issue_s(1, st0 + j + 2, b0);
                tc_commit(bar(C::Q_EMPTY));
              }
            }
            const int b = b0;
            b0 = b1; b1 = b2; b2 = b;
          }
        }
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  } else {
    // ---------------- softmax: warps 2-5 tile A, 6-9 tile B, a thread per row
    const int x = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;                // row of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_o = tmem + C::COL_O + x * D + lane_base;
    bool good = true;
    int nx = 0;     // tasks of this tile so far
    int ko = 0;     // items of this tile so far
    int stage = 0;  // ring stages of the items before
    Jobs js;
    for (bool more = js.begin(n_items, p); more && good; more = js.next(p)) {
      const Job& w = js.w;
      const int stage_job = stage, both = min(w.n[0], w.n[1]);
      stage += max(w.n[0], w.n[1]) + 1;
      if (w.n[x] == 0) continue;
      const int row0 = w.q + x * TQ;  // first row of the tile
      const int row = row0 + r;
      float m_ref = -INFINITY, l = 0.0f;
      for (int j = 0; j < w.n[x]; ++j, ++nx) {
        const int kv0 = j * TK;
        const int buf = w.n[1] == 0 ? j & 1 : NB == 2 ? x : (j < both ? 2 * j + x : both + j) % 3;
        const uint32_t t_s = tmem + C::COL_S + buf * TK + lane_base;  // scores, then P
        if (!wait_phase(bar(C::S_FULL + 2 * x + (nx & 1)), (nx >> 1) & 1, p.err, abort)) {
          good = false;
          break;
        }
        tc_fence_after();
        // visible keys of the tile: kv0 .. kv0 + see - 1
        const bool edge = kv0 + TK > w.len || (p.causal && kv0 + TK - 1 > row0);
        const int see = min(w.len, p.causal ? row + 1 : w.len) - kv0;
        // the maximum of the 32 scores of chunk c, or m0 if it is larger
        auto chunk_max = [&](int c, float m0) {
          uint32_t q[32];
          tmem_ld32(t_s + c * 32, q);
          tmem_ld_wait();
          tmem_regs_ready(q);
          float m4[4] = {m0, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = edge && c * 32 + e >= see ? -INFINITY : __uint_as_float(q[e]);
            const float b = edge && c * 32 + e + 1 >= see ? -INFINITY : __uint_as_float(q[e + 1]);
            m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], a, b);
          }
          return fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
        };
        // P = 2^(s log2e / sqrt(d) - m_ref) as bf16 pairs (the row sum takes them
        // unrounded): off by 2^-8 relative at most per weight. Averaging shrinks these
        // errors as it shrinks the result, so they add about as much as the output's
        // own rounding: relative error against 64 bits 0.0021 on long prompts, 0.0016
        // without. A second bf16 part for what the first leaves, as in the decode kernel,
        // would add half as many tensor cycles again (512 per tile to 1024) where the
        // tensor core is the bound; the layer's dense forward rounds alike.
        uint32_t pk[64];
        float sum = 0.0f;
        auto form = [&](auto masked) {
          // One warp per scheduler has to keep the exponential unit (4 cycles
          // per instruction) busy by itself: groups of four keys, the exponentials of
          // one between the sums and packing of the one before and the scaling
          // of the second next, scores of the next 16 keys on their way.
          // (past REF_LIMIT: below)
          const float nref = fabsf(m_ref) <= REF_LIMIT ? -m_ref : 0.0f;
          float r0 = 0.0f, r1 = 0.0f, r2 = 0.0f, r3 = 0.0f;
          uint32_t q[2][16];
          float t[4][4];
          auto scale = [&](int g) {
            uint32_t z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[e] = q[(g >> 2) & 1][(g & 3) * 4 + e];
              if constexpr (decltype(masked)::value)
                if (4 * g + e >= see) z[e] = 0xff800000u;  // -infinity
            }
            v_fma2(t[g & 3][0], t[g & 3][1], z[0], z[1], p.sl2, nref);
            v_fma2(t[g & 3][2], t[g & 3][3], z[2], z[3], p.sl2, nref);
          };
          tmem_ld16(t_s, q[0]);
          tmem_ld_wait();
          tmem_regs_ready(q[0]);
          tmem_ld16(t_s + 16, q[1]);
          scale(0);
          scale(1);
#pragma unroll
          for (int g = 0; g < 32; ++g) {
            float* y = t[g & 3];
            const float* u = t[(g + 3) & 3];  // group g - 1
            v_ex2(y[0]);
            if (g > 0) v_add2(r0, r1, u[0], u[1]);
            v_ex2(y[1]);
            if (g > 0) pk[2 * g - 2] = v_pack(u[0], u[1]);
            v_ex2(y[2]);
            if (g > 0) v_add2(r2, r3, u[2], u[3]);
            v_ex2(y[3]);
            if (g > 0) pk[2 * g - 1] = v_pack(u[2], u[3]);
            if (g + 2 < 32) {
              if (((g + 2) & 3) == 0) {
                const int c = (g + 2) >> 2;
                tmem_ld_wait();
                tmem_regs_ready(q[c & 1]);
                if (c < 7) tmem_ld16(t_s + (c + 1) * 16, q[(c + 1) & 1]);
              }
              scale(g + 2);
            }
          }
          v_add2(r0, r1, t[3][0], t[3][1]);
          v_add2(r2, r3, t[3][2], t[3][3]);
          pk[62] = v_pack(t[3][0], t[3][1]);
          pk[63] = v_pack(t[3][2], t[3][3]);
          sum = (r0 + r1) + (r2 + r3);
        };
        // The first reference is the maximum of the first 32 keys (key 0 is
        // visible to every row): at most the row's, so the sum is at least 1, and
        // far below it only if the sum shows it.
        if (j == 0) m_ref = __fmul_rn(chunk_max(0, -INFINITY), p.sl2);
        if (edge) form(std::true_type{});
        else form(std::false_type{});
        // (NaN too; and a reference past REF_LIMIT, or none, as all first scores were
        // -infinity, whose weights were not formed with it.) Rows behind the end hold
        // other sequences' queries and have no say; nor does a row move its reference
        // because another one must, so that its bits are its own. The branch is the
        // whole warp's, as the TMEM loads inside must be.
        bool need = !(sum <= SUM_LIMIT) || fabsf(m_ref) > REF_LIMIT;
        if (__any_sync(0xffffffffu, need) && __any_sync(0xffffffffu, need &= row < w.len)) {
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) mx = chunk_max(c, mx);
          mx = __fmul_rn(mx, p.sl2);  // (rounded: not fused into what follows)
          float alpha = 1.0f;
          if (need && mx > m_ref) {
            alpha = exp2f(m_ref - mx);
            m_ref = mx;
            l *= alpha;
          }
          if (j > 0) {
            // rescale the O_X row once PV_X(j - 1) is complete: the stage of
            // V_{j-1} has been released (and not been filled and released again,
            // which takes this task's weights)
            const int st = stage_job + j;
            if (!wait_phase(bar(C::L_EMPTY + st % NST), (st / NST) & 1, p.err, abort)) *abort = 1;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ro[32];
              tmem_ld32(t_o + c * 32, ro);
              tmem_ld_wait();
              tmem_regs_ready(ro);
#pragma unroll
              for (int e = 0; e < 32; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha);
              tmem_st32(t_o + c * 32, ro);
            }
          }
          const bool apart = fabsf(m_ref) > REF_LIMIT && m_ref > -INFINITY;
          if (__any_sync(0xffffffffu, apart)) {
            // The reference is subtracted from scores scaled and rounded as it was, so that
            // equal scores leave exactly 0; the differences take the scores' place.
            const float back = 1.0f / p.sl2;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t q[32];
              tmem_ld32(t_s + c * 32, q);
              tmem_ld_wait();
              tmem_regs_ready(q);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (apart)
                  q[e] = __float_as_uint((__fmul_rn(__uint_as_float(q[e]), p.sl2) - m_ref) * back);
              tmem_st32(t_s + c * 32, q);
            }
            tmem_st_wait();
          }
          form(std::true_type{});  // (masks nothing inside)
        }
        l += sum;
        {
          uint32_t h[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int e = 0; e < 32; ++e) h[e] = pk[c * 32 + e];
            tmem_st32(t_s + c * 32, h);
          }
        }
        const int left = w.len - j * TK;  // keys of the sequence from this tile on
        if (left < TK && (left & 15) && (x == 0 || j >= w.n[0])) {
          // clear the value rows behind the end, up to the K step's last (8
          // chunks per 64-column box); j is the item's last step
          const int st = stage_job + j + 1, rows = 16 - (left & 15);
          if (!wait_phase(bar(C::L_FULL + st % NST), (st / NST) & 1, p.err, abort)) *abort = 1;
          const uint32_t dv = sV + (st % NST) * C::KV_BYTES;
          for (int c = r; c < rows * 8 * C::KB; c += TQ) {
            const int kb = c / (rows * 8), rc = c - kb * (rows * 8);
            st_shared_v4u(dv + kb * C::BOX + (left + rc / 8) * 128 + (rc % 8) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async();  // before the tensor core reads them
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();  // the warp's P stores are done: one arrival for the warp
        if (lane == 0) mbar_arrive(bar(C::P_FULL + 2 * x + (nx & 1)));
      }
      if (!good) break;
      // ---- tile done: O / l and LSE
      if (!wait_phase(bar(C::O_FULL + x), ko & 1, p.err, abort)) {
        good = false;
        break;
      }
      ++ko;
      tc_fence_after();
      const float inv = 1.0f / l;  // (l = 0: every score is -infinity, 0 / 0)
      const bool row_ok = row < w.len;
      bf16* out = p.o + (int64_t)(w.a + row) * p.ld_o + w.h * D;
      if (p.wide) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t q[32], h[16];
          tmem_ld32(t_o + c * 32, q);
          tmem_ld_wait();
          tmem_regs_ready(q);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            h[e] = pack_bf16x2(__uint_as_float(q[2 * e]) * inv, __uint_as_float(q[2 * e + 1]) * inv);
          if (row_ok) {
            st_global_32(out + c * 32, h);
            st_global_32(out + c * 32 + 16, h + 8);
          }
        }
      } else {
        store_tmem_row<D>(t_o, inv, row_ok ? out : nullptr);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::O_EMPTY + x));
      if (row_ok && p.lse != nullptr)
        p.lse[(int64_t)w.h * p.tokens + w.a + row] = (m_ref + log2f(l)) * LN2;
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
mgb_status fwd_d(const PackedArgs& a, cudaStream_t st) {
  using C = Cfg2<D>;
  CUtensorMap tq, tk, tv;
  const uint64_t T = (uint64_t)a.tokens;
  if (tmap_encode_bf16_2d(&tq, a.q, (uint64_t)a.nq * D, T, a.ld_q, 64, TQ) != CUDA_SUCCESS ||
      tmap_encode_bf16_2d(&tk, a.k, (uint64_t)a.nkv * D, T, a.ld_kv, 64, TK) != CUDA_SUCCESS ||
      tmap_encode_bf16_2d(&tv, a.v, (uint64_t)a.nkv * D, T, a.ld_kv, 64, TK) != CUDA_SUCCESS)
    return MGB_ERR_CUDA;
  Params p{};
  auto magic = [](int d) { return d == 1 ? 0 : ~(uint64_t)0 / (uint64_t)d + 1; };
  p.nq = a.nq; p.m_nq = magic(a.nq); p.m_group = magic(a.nq / a.nkv); p.causal = a.causal; p.tokens = a.tokens;
  p.hdr = a.hdr256; p.list = a.list256;
  p.o = static_cast<bf16*>(a.o); p.ld_o = a.ld_o; p.lse = a.lse;
  p.wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0 && a.ld_o % 16 == 0;
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  p.sl2 = LOG2E / sqrtf((float)D);
  auto k = packed_fwd_kernel<D>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const int64_t most = a.max256 * a.nq;
  const int grid = most < device_sm_count() ? (int)most : device_sm_count();
  return launch_pdl(k, grid, NTHREADS, C::SMEM, st, tq, tk, tv, p);
}

}  // namespace

mgb_status attention_packed_bf16(const PackedArgs& a, cudaStream_t st) {
  return a.d == 64 ? fwd_d<64>(a, st) : fwd_d<128>(a, st);
}

}  // namespace mgb
