// Attention over packed sequences, float32, on the CUDA cores: O_h =
// softmax(Q_h K_g^T / sqrt(d)) V_g within each sequence, optionally causal, and
// its log-sum-exp. Exact float32 products (no TF32), online softmax.
//
// A block of 256 threads takes 128 query rows of one (sequence, head) and walks
// key tiles of 64. Thread (ty, tx) of a 16 x 16 grid holds rows 8 ty .. + 7 and
// keys tx + 16 c of the score tile, then the same rows and columns 4 tx + 64 c ..
// + 3 of the output: per 4 (inner) steps the scores take 12 16-byte
// shared-memory reads for 128 FMAs, the output product 8 + 8 for 256 (D = 128),
// so the FMA pipe is the bound. K of the next tile is copied while the softmax
// and the second product run, V of this one while the scores are formed.
// Rows behind the sequence are zeros in shared memory (never read).
#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mgb {

namespace {

constexpr int BM = 128, BN = 64, NT = 256;
constexpr int PS = BN + 4;  // row stride of P (floats)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int RS = D + 4;  // row stride of Q, K, V (floats): 16 rows' float4 hit all banks
  static constexpr int OFF_K = BM * RS;
  static constexpr int OFF_V = OFF_K + BN * RS;
  static constexpr int OFF_P = OFF_V + BN * RS;
  static constexpr int SMEM = (OFF_P + BM * PS) * 4;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(NT, D == 64 ? 2 : 1) packed_f32_kernel(const Params p) {
  using C = Cfg<D>;
  constexpr int RS = C::RS, OC = D / 64;  // 4-column groups per thread
  extern __shared__ __align__(16) float sh[];
  float *sq = sh, *sk = sh + C::OFF_K, *sv = sh + C::OFF_V, *sp = sh + C::OFF_P;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n_items = p.hdr->entries * p.nq;
  const uint32_t bq = smem_u32(sq), bk = smem_u32(sk), bv = smem_u32(sv);

  for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
    const int4 e = p.list[i / p.nq];
    const int h = i % p.nq, len = e.y, q0 = e.z;
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
    float acc[8][4 * OC], m[8], l[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
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
      float s[8][4] = {};
#pragma unroll 4
      for (int f = 0; f < D; f += 4) {
        float4 kk[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) kk[c] = *reinterpret_cast<const float4*>(sk + (tx + 16 * c) * RS + f);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float4 qq = *reinterpret_cast<const float4*>(sq + (8 * ty + r) * RS + f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s[r][c] = fmaf(qq.x, kk[c].x, s[r][c]);
            s[r][c] = fmaf(qq.y, kk[c].y, s[r][c]);
            s[r][c] = fmaf(qq.z, kk[c].z, s[r][c]);
            s[r][c] = fmaf(qq.w, kk[c].w, s[r][c]);
          }
        }
      }
      const bool edge = k0 + BN > len || (p.causal && k0 + BN - 1 > q0);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = k0 + tx + 16 * c;
          s[r][c] *= p.sl2;
          if (edge && (key >= len || (p.causal && key > q0 + 8 * ty + r))) s[r][c] = -INFINITY;
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
        for (int c = 0; c < 4; ++c) {
          s[r][c] = exp2f(s[r][c] - mr);
          l[r] += s[r][c];
          sp[(8 * ty + r) * PS + tx + 16 * c] = s[r][c];
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
        for (int r = 0; r < 8; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(sp + (8 * ty + r) * PS + f);
          const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int c = 0; c < OC; ++c) {
              acc[r][4 * c] = fmaf(ww[g], vv[g][c].x, acc[r][4 * c]);
              acc[r][4 * c + 1] = fmaf(ww[g], vv[g][c].y, acc[r][4 * c + 1]);
              acc[r][4 * c + 2] = fmaf(ww[g], vv[g][c].z, acc[r][4 * c + 2]);
              acc[r][4 * c + 3] = fmaf(ww[g], vv[g][c].w, acc[r][4 * c + 3]);
            }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      const int row = 8 * ty + r;
      if (row >= rows) continue;
      const float inv = l[r] > 0.0f ? 1.0f / l[r] : 0.0f;
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

template <int D>
mgb_status launch(const Params& p, int64_t most, cudaStream_t st) {
  auto k = packed_f32_kernel<D>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const int64_t slots = (int64_t)device_sm_count() * (D == 64 ? 2 : 1);
  k<<<(int)(most < slots ? most : slots), NT, Cfg<D>::SMEM, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? MGB_OK : MGB_ERR_CUDA;
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
  return a.d == 64 ? launch<64>(p, a.max128 * a.nq, st) : launch<128>(p, a.max128 * a.nq, st);
}

}  // namespace mgb
