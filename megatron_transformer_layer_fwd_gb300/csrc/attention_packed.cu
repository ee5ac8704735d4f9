// Attention over packed sequences of different lengths, bf16, on the tensor
// cores (tcgen05): O_h = softmax(Q_h K_g^T / sqrt(d)) V_g within each sequence,
// optionally causal, and its log-sum-exp.
//
// A work item is 256 query rows of one (sequence, head), in two tiles A and B
// of 128 that take turns on the tensor core. Per 128 keys the MMA warp issues
// PV_A(j), S_A(j+1), PV_B(j), S_B(j+1); while tile A's scores are turned into
// weights, tile B's two products run. TMEM (512 columns) holds S_A, S_B, O_A, O_B; a
// tile's weights P (bf16 pairs) overwrite scores already read and are read from
// there by PV.
//
// Each tile goes round a chain: scores complete - softmax - weights ready -
// PV and the next scores (16 products of 64 cycles) - scores complete. Two
// tiles cover the tensor core only as far as that chain is short (measured at
// D = 128, in cycles: softmax 1020, to the MMA warp 220, products 1270; the
// tensor core is busy for 2048 of the 2515). What shortens it:
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
// 8177 tokens in two sequences, 32 / 8 heads, D = 128, causal: 184 us, 1490
// TFLOP/s.
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
constexpr int NST = 2;          // ring stages, each a K tile and the V tile before it
constexpr int NSOFTW = 4;       // softmax warps per tile
constexpr int NTHREADS = 320;   // MMA warp, producer warp, 2 x 4 softmax warps
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float SUM_LIMIT = 8192.0f;  // of a row's weights in a tile

template <int D>
struct Cfg2 {
  static constexpr int KB = D / 64;                     // 64-wide d boxes
  static constexpr int BOX = 128 * 128;                 // bytes of one [128][64] box
  static constexpr int Q_BYTES = TQ * D * 2;
  static constexpr int KV_BYTES = TK * D * 2;
  static constexpr int OFF_QA = 0;
  static constexpr int OFF_QB = Q_BYTES;
  static constexpr int OFF_K = 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NST * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + NST * KV_BYTES;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;     // barriers, alignment slack
  static constexpr int COL_S = 0;                       // S_A at 0, S_B at TK
  static constexpr int COL_O = 2 * TK;                  // O_A, then O_B at + D
  static constexpr int TMEM_COLS = 512;
  static_assert(COL_O + 2 * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct Params {
  int nq, group, causal, tokens;
  const PackedHeader* hdr;
  const int4* list;  // entries of 256 rows
  bf16* o;
  int64_t ld_o;
  int wide;  // o's rows are 32-byte aligned
  float* lse;
  int* err;
  float sl2;  // log2(e) / sqrt(d)
};

struct Item {
  int a, len, q0, h, n[2];  // sequence's first row and length; first query row in it; head;
                            // key tiles of tile A and B
};

// Item i: entry i / nq, head i % nq (the heads of a group next to each other
// share their keys and values in L2).
__device__ __forceinline__ Item item_of(int i, const Params& p) {
  const int4 e = p.list[i / p.nq];
  Item it;
  it.a = e.x;
  it.len = e.y;
  it.q0 = e.z;
  it.h = i % p.nq;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r0 = it.q0 + x * TQ;
    const int end = p.causal ? min(it.len, r0 + TQ) : it.len;
    it.n[x] = r0 < it.len ? (end + TK - 1) / TK : 0;
  }
  return it;
}

// The item a CTA takes in its k-th round: snake order over the list, as in the
// dense forward.
__device__ __forceinline__ int item_index(int k) {
  const int g = (int)gridDim.x, c = (int)blockIdx.x;
  return k * g + ((k & 1) ? g - 1 - c : c);
}

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
  const uint32_t sQ[2] = {sb + C::OFF_QA, sb + C::OFF_QB};
  const uint32_t sK = sb + C::OFF_K, sV = sb + C::OFF_V;
  const uint32_t bar = sb + C::OFF_BAR;
  const uint32_t q_full = bar;         // both Q tiles loaded                   (tx)
  const uint32_t q_empty = bar + 8;    // the item's last S product done        (commit)
  const uint32_t l_full0 = bar + 16;   // [2] stage loaded                      (tx)
  const uint32_t l_empty0 = bar + 32;  // [2] products with it done             (commit)
  const uint32_t s_full0 = bar + 80;   // [tile] S_X(j) complete                (commit)
  const uint32_t p_full0 = bar + 96;   // [tile] P_X(j) written, O_X rescaled   (4: one per warp)
  const uint32_t o_full0 = bar + 112;  // [tile] the item's last PV_X done      (commit)
  const uint32_t o_empty0 = bar + 128; // [tile] O_X read out                   (4: one per warp)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 240);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 244);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_items = p.hdr->entries * p.nq;
  if ((int)blockIdx.x >= n_items) return;

  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(l_full0 + 8 * i, 1);
      mbar_init(l_empty0 + 8 * i, 1);
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(p_full0 + 8 * i, NSOFTW);
      mbar_init(o_full0 + 8 * i, 1);
      mbar_init(o_empty0 + 8 * i, NSOFTW);
    }
    fence_mbar_init();
    *abort = 0;
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 2) {
  if (warp == 1) {
    // ---------------- producer: per item Q_A, Q_B, then the stages (K_0),
    // (V_0, K_1), (V_1, K_2), .., (V_last)
    if (lane == 0) {
      int nl = 0;  // stages loaded so far
      for (int k = 0, i = item_index(0); i < n_items && !*abort; ++k, i = item_index(k)) {
        const Item w = item_of(i, p);
        const int xcol = (w.h / p.group) * D;
        // the item lies in the tensors and the TMA x coordinates are 16-byte
        // multiples (head columns: multiples of 64)
        if (!dcheck(w.a >= 0 && w.q0 >= 0 && w.q0 < w.len && w.len <= p.tokens - w.a &&
                        w.h < p.nq && (xcol & 7) == 0 && ((w.h * D) & 7) == 0,
                    p.err)) {
          *abort = 1;
          break;
        }
        if (k >= 1 && !mbar_wait(q_empty, (k - 1) & 1, p.err)) {
          *abort = 1;
          break;
        }
        mbar_arrive_expect_tx(q_full, (w.n[1] > 0 ? 2 : 1) * C::Q_BYTES);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (w.n[x] == 0) continue;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(sQ[x] + kb * C::BOX, &tmQ, w.h * D + kb * 64, w.a + w.q0 + x * TQ, q_full);
        }
        const int nt = max(w.n[0], w.n[1]);
        bool good = true;
        for (int j = 0; j <= nt; ++j, ++nl) {
          const int s = nl % NST;
          if (nl >= NST && !mbar_wait(l_empty0 + 8 * s, ((nl - NST) / NST) & 1, p.err)) {
            good = false;
            break;
          }
          mbar_arrive_expect_tx(l_full0 + 8 * s, (j > 0 && j < nt ? 2 : 1) * C::KV_BYTES);
          if (j > 0)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_2d(sV + s * C::KV_BYTES + kb * C::BOX, &tmV, xcol + kb * 64,
                          w.a + (j - 1) * TK, l_full0 + 8 * s);
          if (j < nt)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_2d(sK + s * C::KV_BYTES + kb * C::BOX, &tmK, xcol + kb * 64, w.a + j * TK,
                          l_full0 + 8 * s);
        }
        if (!good) {
          *abort = 1;
          break;
        }
      }
    }
  } else if (warp == 0) {
    // ---------------- MMA issuer: one thread
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(TQ, TK, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(TQ, D, 0, 1);
      const uint64_t dq0[2] = {smem_desc_sw128(sQ[0], 16, 1024), smem_desc_sw128(sQ[1], 16, 1024)};
      const uint64_t dk0 = smem_desc_sw128(sK, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sV, C::BOX, 1024);
      int nl = 0;             // stages consumed so far
      int np[2] = {0, 0};     // PV products of each tile so far (p_full phases)
      int no[2] = {0, 0};     // items with a non-empty tile X so far (o_full / o_empty phases)
      bool good = true;
      // S_X = Q_X K^T into tile X's score columns (K stage sk)
      auto issue_s = [&](int x, int sk) {
        const uint64_t db = dk0 + (uint64_t)((sk * C::KV_BYTES) >> 4);
        const uint32_t td = tmem + C::COL_S + x * TK;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::BOX + (kk & 3) * 32;
          tc_mma_f16(td, dq0[x] + (uint64_t)(off >> 4), db + (uint64_t)(off >> 4), idesc_s, kk > 0);
        }
        tc_commit(s_full0 + 8 * x);
      };
      for (int k = 0, i = item_index(0); i < n_items && good; ++k, i = item_index(k)) {
        const Item w = item_of(i, p);
        const int nt = max(w.n[0], w.n[1]);
        const int s0 = nl % NST;
        if (!wait_phase_1(q_full, k & 1, p.err, abort) ||
            !wait_phase_1(l_full0 + 8 * s0, (nl / NST) & 1, p.err, abort)) {
          good = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (w.n[x] > 0) issue_s(x, s0);
        tc_commit(l_empty0 + 8 * s0);
        if (nt == 1) tc_commit(q_empty);
        ++nl;
        for (int j = 0; j < nt && good; ++j) {
          const int s = nl % NST;  // V_j, K_{j+1}
          if (!wait_phase_1(l_full0 + 8 * s, (nl / NST) & 1, p.err, abort)) {
            good = false;
            break;
          }
          const int left = w.len - j * TK;  // keys of the sequence from this tile on
          const int steps = left >= TK ? TK / 16 : (left + 15) / 16;
          const uint64_t db = dv0 + (uint64_t)((s * C::KV_BYTES) >> 4);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!good || j >= w.n[x]) continue;
            // O_X of the previous item read out before this item's first PV_X
            if ((j == 0 && no[x] >= 1 &&
                 !wait_phase_1(o_empty0 + 8 * x, (no[x] - 1) & 1, p.err, abort)) ||
                !wait_phase_1(p_full0 + 8 * x, np[x] & 1, p.err, abort)) {
              good = false;
              continue;
            }
            tc_fence_after();
            const uint32_t ta = tmem + C::COL_S + x * TK, to = tmem + C::COL_O + x * D;
            if (steps == TK / 16) {
#pragma unroll
              for (int kk = 0; kk < TK / 16; ++kk)
                tc_mma_f16_ts(to, ta + kk * 8, db + (uint64_t)((kk * 2048) >> 4),
                              idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < steps; ++kk)
                tc_mma_f16_ts(to, ta + kk * 8, db + (uint64_t)((kk * 2048) >> 4),
                              idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
            }
            ++np[x];
            if (j == w.n[x] - 1) {
              tc_commit(o_full0 + 8 * x);
              ++no[x];
            } else {
              issue_s(x, s);
            }
          }
          if (!good) break;
          tc_commit(l_empty0 + 8 * s);
          ++nl;
          // the item's last score product has been issued once j + 1 == nt - 1
          if (j + 2 == nt) tc_commit(q_empty);
        }
      }
      if (!good) *abort = 1;
    }
    __syncwarp();
  }
  } else {
    // ---------------- softmax: warps 2-5 tile A, 6-9 tile B, a thread per row
    const int x = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;                // row of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + C::COL_S + x * TK + lane_base;  // scores, then P
    const uint32_t t_o = tmem + C::COL_O + x * D + lane_base;
    const uint32_t sfull = s_full0 + 8 * x, pfull = p_full0 + 8 * x;
    const uint32_t ofull = o_full0 + 8 * x, oempty = o_empty0 + 8 * x;
    bool good = true;
    int n = 0;   // S_X products consumed so far
    int ko = 0;  // items with a non-empty tile X so far
    int nl = 0;  // ring stages of the items before
    for (int k = 0, i = item_index(0); i < n_items && good; ++k, i = item_index(k)) {
      const Item w = item_of(i, p);
      const int nt = max(w.n[0], w.n[1]), nl0 = nl;
      nl += nt + 1;
      if (w.n[x] == 0) continue;  // tile past the sequence end: nothing to do
      const int row0 = w.q0 + x * TQ;  // first row of the tile
      const int row = row0 + r;
      float m_ref = -INFINITY, l = 0.0f;
      for (int j = 0; j < w.n[x]; ++j, ++n) {
        const int kv0 = j * TK;
        if (!wait_phase(sfull, n & 1, p.err, abort)) {
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
        // unrounded): a relative error of at most 2^-8 per weight, below the
        // output's own rounding after averaging
        uint32_t pk[64];
        float sum = 0.0f;
        auto form = [&](auto masked) {
          // One warp per scheduler has to keep the exponential unit (4 cycles
          // per instruction) busy by itself: groups of four keys, the exponentials of
          // one between the sums and packing of the one before and the scaling
          // of the second next, scores of the next 16 keys on their way.
          const float nref = m_ref == -INFINITY ? 0.0f : -m_ref;
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
        if (j == 0) m_ref = chunk_max(0, -INFINITY) * p.sl2;
        if (edge) form(std::true_type{});
        else form(std::false_type{});
        // (NaN too; no reference: all first scores were -infinity)
        if (__any_sync(0xffffffffu, !(sum <= SUM_LIMIT) || m_ref == -INFINITY)) {
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) mx = chunk_max(c, mx);
          mx *= p.sl2;
          float alpha = 1.0f;
          if (mx > m_ref) {
            alpha = exp2f(m_ref - mx);
            m_ref = mx;
            l *= alpha;
          }
          if (j > 0) {
            // rescale the O_X row (PV_X(j - 1) completed before S_X(j) did)
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
          // chunks per 64-column box); j is the item's last tile
          const int v = nl0 + j + 1, rows = 16 - (left & 15);
          if (!wait_phase(l_full0 + 8 * (v % NST), (v / NST) & 1, p.err, abort)) *abort = 1;
          for (int c = r; c < rows * 8 * C::KB; c += TQ) {
            const int kb = c / (rows * 8), rc = c - kb * (rows * 8);
            st_shared_v4u(sV + (v % NST) * C::KV_BYTES + kb * C::BOX + (left + rc / 8) * 128 +
                              (rc % 8) * 16,
                          0, 0, 0, 0);
          }
          fence_proxy_async();  // before the tensor core reads them
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();  // the warp's P stores are done: one arrival for the warp
        if (lane == 0) mbar_arrive(pfull);
      }
      if (!good) break;
      // ---- tile done: O / l and LSE
      if (!wait_phase(ofull, ko & 1, p.err, abort)) {
        good = false;
        break;
      }
      ++ko;
      tc_fence_after();
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
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
      if (lane == 0) mbar_arrive(oempty);
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
  p.nq = a.nq; p.group = a.nq / a.nkv; p.causal = a.causal; p.tokens = a.tokens;
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
  k<<<grid, NTHREADS, C::SMEM, st>>>(tq, tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? MGB_OK : MGB_ERR_CUDA;
}

}  // namespace

mgb_status attention_packed_bf16(const PackedArgs& a, cudaStream_t st) {
  return a.d == 64 ? fwd_d<64>(a, st) : fwd_d<128>(a, st);
}

}  // namespace mgb
