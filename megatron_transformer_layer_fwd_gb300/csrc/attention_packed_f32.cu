// Attention over packed sequences, float32, on the CUDA cores: O_h =
// softmax(Q_h K_g^T / sqrt(d)) V_g within each sequence, optionally causal, and
// its log-sum-exp. Exact float32 products (no TF32), online softmax.
//
// A block of 128 threads takes 64 query rows of one (sequence, head) and walks
// key tiles of BN. Thread (ty, tx) of an 8 x 16 grid holds rows 8 ty .. + 7 and
// keys tx + 16 c of the score tile, then the same rows and columns 4 tx + 64 c ..
// + 3 of the output: per 4 (inner) steps the scores take 8 + BN / 16 16-byte
// shared-memory reads for 2 BN FMAs (two per instruction), the output product
// 8 + 4 D / 64 for 2 D, so the FMA pipe is the bound (8 x 1000 tokens, 16 heads:
// 35 TFLOP/s at either head dim). K of the next tile is copied while the softmax and
// the second product run, V of this one while the scores are formed. Three
// (D = 64) or two blocks per SM fill each other's barriers and softmax.
// Rows behind the sequence are zeros in shared memory (never read).
#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mgb {

namespace {

constexpr int NT = 128;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

template <int D, int RPT>
struct Cfg {
  static constexpr int BM = 8 * RPT;              // query rows per block
  static constexpr int BN = D == 64 ? 64 : 32;    // keys per tile
  static constexpr int BLOCKS = D == 64 ? 3 : 2;  // per SM
  static constexpr int PS = BN + 4;               // row stride of P (floats)
  static constexpr int RS = D + 4;  // row stride of Q, K, V (floats): 16 rows' float4 hit all banks
  static constexpr int OFF_K = BM * RS;
  static constexpr int OFF_V = OFF_K + BN * RS;
  static constexpr int OFF_P = OFF_V + BN * RS;
  static constexpr int SMEM = (OFF_P + BM * PS) * 4;
  static_assert((SMEM + 1024) * BLOCKS <= 228 * 1024, "blocks per SM");
};

struct Params {
  int nq, group, causal, tokens;
  const PackedHeader* hdr;
  const int4* list;
  const float *q, *k, *v;
  int64_t ld_q, ld_kv;
  float* o;
  int64_t ld_o;
  float* lse;
  float sl2;
};

// RPT: query rows per thread
template <int D, int RPT>
__global__ void __launch_bounds__(NT, Cfg<D, RPT>::BLOCKS) packed_f32_kernel(const Params p) {
  using C = Cfg<D, RPT>;
  constexpr int RS = C::RS, PS = C::PS, BN = C::BN, BM = C::BM, PARTS = 128 / BM;
  constexpr int OC = D / 64, KC = BN / 16;  // 4-column groups, keys per thread
  extern __shared__ __align__(16) float sh[];
  float *sq = sh, *sk = sh + C::OFF_K, *sv = sh + C::OFF_V, *sp = sh + C::OFF_P;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n_items = p.hdr->entries * PARTS * p.nq;  // an entry is 128 rows
  const uint32_t bq = smem_u32(sq), bk = smem_u32(sk), bv = smem_u32(sv);

  // snake order over the list (longest first), as in the bf16 kernel
  auto item_index = [&](int turn) {
    const int g = (int)gridDim.x, c = (int)blockIdx.x;
    return turn * g + ((turn & 1) ? g - 1 - c : c);
  };
  for (int turn = 0, i = item_index(0); i < n_items; ++turn, i = item_index(turn)) {
    const int4 e = p.list[i / (PARTS * p.nq)];
    const int h = i % p.nq, len = e.y, q0 = e.z + (i / p.nq % PARTS) * BM;
    if (q0 >= len) continue;
    const float* Q = p.q + (int64_t)(e.x + q0) * p.ld_q + (int64_t)h * D;
    const float* K = p.k + (int64_t)e.x * p.ld_kv + (int64_t)(h / p.group) * D;
    const float* V = p.v + (int64_t)e.x * p.ld_kv + (int64_t)(h / p.group) * D;
    const int rows = min(BM, len - q0);
    const int nt = ((p.causal ? min(len, q0 + BM) : len) + BN - 1) / BN;
    // rows r0 .. of x (stride ld), those at or behind `valid` as zeros
    auto copy = [&](uint32_t dst, const float* x, int64_t ld, int n, int valid) {
      for (int c = tid; c < n * (D / 4); c += NT) {
        const int r = c / (D / 4), f = c % (D / 4) * 4;
        const bool on = r < valid;
        cp_async16(dst + (r * RS + f) * 4, x + (on ? (int64_t)r * ld + f : 0), on);
      }
    };
    __syncthreads();  // the previous item is done with shared memory
    copy(bq, Q, p.ld_q, BM, rows);
    copy(bk, K, p.ld_kv, BN, len);
    cp_async_commit();
    float acc[RPT][4 * OC], m[RPT], l[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
#pragma unroll
      for (int c = 0; c < 4 * OC; ++c) acc[r][c] = 0.0f;
    }
    for (int j = 0; j < nt; ++j) {
      const int k0 = j * BN;
      __syncthreads();  // V and P of the tile before are read
      copy(bv, V + (int64_t)k0 * p.ld_kv, p.ld_kv, BN, len - k0);
      cp_async_commit();
      cp_async_wait<1>();  // Q and this tile's K
      __syncthreads();
      float s[RPT][KC] = {}, s2[RPT][KC] = {};  // sums over even and odd inner indices
#pragma unroll 4
      for (int f = 0; f < D; f += 4) {
        float4 kk[KC];
#pragma unroll
        for (int c = 0; c < KC; ++c) kk[c] = *reinterpret_cast<const float4*>(sk + (tx + 16 * c) * RS + f);
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const float4 qq = *reinterpret_cast<const float4*>(sq + (RPT * ty + r) * RS + f);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            fma2(s[r][c], s2[r][c], qq.x, qq.y, kk[c].x, kk[c].y, s[r][c], s2[r][c]);
            fma2(s[r][c], s2[r][c], qq.z, qq.w, kk[c].z, kk[c].w, s[r][c], s2[r][c]);
          }
        }
      }
      const bool edge = k0 + BN > len || (p.causal && k0 + BN - 1 > q0);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const int key = k0 + tx + 16 * c;
          // (rounded before the maximum and the subtraction: the largest weight is 1)
          s[r][c] = __fmul_rn(s[r][c] + s2[r][c], p.sl2);
          if (edge && (key >= len || (p.causal && key > q0 + RPT * ty + r))) s[r][c] = -INFINITY;
          mx = fmaxf(mx, s[r][c]);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx > m[r]) {
          const float a = exp2f(m[r] - mx);
          m[r] = mx;
          l[r] *= a;
#pragma unroll
          for (int c = 0; c < 4 * OC; ++c) acc[r][c] *= a;
        }
        const float mr = m[r] == -INFINITY ? 0.0f : m[r];  // -infinity: every score so far is
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          s[r][c] = exp2f(s[r][c] - mr);
          l[r] += s[r][c];
          sp[(RPT * ty + r) * PS + tx + 16 * c] = s[r][c];
        }
      }
      __syncthreads();  // K is read, P written
      if (j + 1 < nt) copy(bk, K + (int64_t)(k0 + BN) * p.ld_kv, p.ld_kv, BN, len - k0 - BN);
      cp_async_commit();
      cp_async_wait<1>();  // V
      __syncthreads();
#pragma unroll 2
      for (int f = 0; f < BN; f += 4) {
        float4 vv[4][OC];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int c = 0; c < OC; ++c)
            vv[g][c] = *reinterpret_cast<const float4*>(sv + (f + g) * RS + 4 * tx + 64 * c);
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(sp + (RPT * ty + r) * PS + f);
          const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int c = 0; c < OC; ++c) {
              float* o = acc[r] + 4 * c;
              fma2(o[0], o[1], ww[g], ww[g], vv[g][c].x, vv[g][c].y, o[0], o[1]);
              fma2(o[2], o[3], ww[g], ww[g], vv[g][c].z, vv[g][c].w, o[2], o[3]);
            }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      const int row = RPT * ty + r;
      if (row >= rows) continue;
      const float inv = 1.0f / l[r];  // (l = 0: every score is -infinity, 0 / 0)
      float* o = p.o + (int64_t)(e.x + q0 + row) * p.ld_o + (int64_t)h * D;
#pragma unroll
      for (int c = 0; c < OC; ++c)
        *reinterpret_cast<float4*>(o + 4 * tx + 64 * c) =
            make_float4(acc[r][4 * c] * inv, acc[r][4 * c + 1] * inv, acc[r][4 * c + 2] * inv,
                        acc[r][4 * c + 3] * inv);
      if (tx == 0 && p.lse != nullptr)
        p.lse[(int64_t)h * p.tokens + e.x + q0 + row] = (m[r] + log2f(l[r])) * LN2;
    }
  }
  cp_async_wait<0>();
}

template <int D, int RPT>
mgb_status launch(const Params& p, int64_t most, cudaStream_t st) {
  using C = Cfg<D, RPT>;
  auto k = packed_f32_kernel<D, RPT>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const int64_t items = most * (128 / C::BM), slots = (int64_t)device_sm_count() * C::BLOCKS;
  k<<<(int)(items < slots ? items : slots), NT, C::SMEM, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? MGB_OK : MGB_ERR_CUDA;
}

// 64 query rows per block, or 32 while 64 would leave less than three blocks per
// slot (`most`: 128-row entries x heads at most): D = 64, 32 heads, 3 x 900
// tokens (3.2 per slot) 358 us against 369, 2 x 600 (1.4) 211 against 198.
template <int D>
mgb_status launch_d(const Params& p, int64_t most, cudaStream_t st) {
  return 2 * most < 3 * (int64_t)device_sm_count() * Cfg<D, 8>::BLOCKS ? launch<D, 4>(p, most, st)
                                                                     : launch<D, 8>(p, most, st);
}

}  // namespace

mgb_status attention_packed_f32(const PackedArgs& a, cudaStream_t st) {
  Params p{};
  p.nq = a.nq; p.group = a.nq / a.nkv; p.causal = a.causal; p.tokens = a.tokens;
  p.hdr = a.hdr128; p.list = a.list128;
  p.q = static_cast<const float*>(a.q); p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.ld_q = a.ld_q; p.ld_kv = a.ld_kv;
  p.o = static_cast<float*>(a.o); p.ld_o = a.ld_o; p.lse = a.lse;
  p.sl2 = LOG2E / sqrtf((float)a.d);
  return a.d == 64 ? launch_d<64>(p, a.max128 * a.nq, st) : launch_d<128>(p, a.max128 * a.nq, st);
}

}  // namespace mgb
