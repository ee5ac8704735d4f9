// Attention of drafted tokens over a paged cache, float32, on the CUDA cores:
// exact float32 products, online softmax.
//
// A block of 128 threads takes BM rows of an item (all of them in turn) and walks its
// units in key tiles of BN. Thread (ty, tx) of an 8 x 16 grid holds rows RPT ty .. and
// keys tx + 16 c of the score tile, then the same rows and columns 4 tx + 64 c .. of
// the output, two FMAs per instruction. K of the next tile is copied while the softmax
// and the second product run, V of this one while the scores are formed. Tokens of a
// bad page and behind the length are zeros in shared memory (never read) and hidden.
//
// Bound: the 16-byte reads of Q, K, V and P from shared memory, one per 2 to 8 paired FMAs. 8 sequences to 3000 tokens, 16 query and 4 KV heads of
// 128, 12 to 80 rows 29 us (HBM 5); 64 of 2000, 20 rows 281 us; one of 20000, 240 rows 301 us, 33
// TFLOP/s. (K and V in two buffers each, one block per SM: no gain.)
#include "tree.cuh"

namespace mgb {

namespace {

constexpr int NT = 128;
constexpr float LN2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int BM = 64;                   // rows per block at most
  static constexpr int BN = D == 64 ? 64 : 32;    // keys per tile
  static constexpr int PS = BN + 4;               // row stride of P (floats)
  static constexpr int RS = D + 4;  // row stride of Q, K, V (floats): 16 rows' float4 hit all banks
  static constexpr int OFF_K = BM * RS;
  static constexpr int OFF_V = OFF_K + BN * RS;
  static constexpr int OFF_P = OFF_V + BN * RS;
  static constexpr int OFF_AT = OFF_P + BM * PS;  // [2][BN] int64: places of the tile's tokens
  static constexpr int SMEM = OFF_AT * 4 + 2 * BN * 8;
  static_assert((SMEM + 1024) * 2 <= 228 * 1024, "two blocks per SM");
  static_assert(OFF_AT % 2 == 0 && BN == CutF32<D>::KEYS && BM == CutF32<D>::ROWS, "layout");
};

// The rows of a segment, RPT per thread.
template <int D, int RPT>
__device__ __forceinline__ void run_rows(const TreeParams& p, const TreeSeg& w, bool whole,
                                         int part, float* sh) {
  using C = Cfg<D>;
  constexpr int RS = C::RS, PS = C::PS, BN = C::BN, BM = 8 * RPT;
  constexpr int OC = D / 64, KC = BN / 16;  // 4-column groups, keys per thread
  float *sq = sh, *sk = sh + C::OFF_K, *sv = sh + C::OFF_V, *sp = sh + C::OFF_P;
  int64_t* sat = reinterpret_cast<int64_t*>(sh + C::OFF_AT);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const uint32_t bq = smem_u32(sq), bk = smem_u32(sk), bv = smem_u32(sv);
  const int rows = w.rows, first = w.b * CutF32<D>::ROWS;
  const int len = w.q.len, ctx = len - w.q.m;
  const int k_first = w.t0 * BN, k_end = min(len, w.t1 * BN);
  const int nt = (k_end - k_first + BN - 1) / BN;
  const int32_t* table = p.table + (int64_t)w.q.s * p.ld_table;
  // the place of this thread's token (tid < BN) of tile j, or -1
  auto find = [&](int j) {
    const int key = k_first + j * BN + tid;
    if (tid >= BN || j >= nt || key >= k_end) return (int64_t)-1;
    const int i = key / p.page_size, page = table[i];
    if (page < 0 || page >= p.n_pages) {
      record_error(p.err, kErrIndex);
      return (int64_t)-1;
    }
    return page * p.s_page + (key - i * p.page_size) * p.s_tok + w.h * p.s_head;
  };
  auto copy = [&](uint32_t dst, const void* x, const int64_t* at) {
    for (int c = tid; c < BN * (D / 4); c += NT) {
      const int r = c / (D / 4), f = c % (D / 4) * 4;
      const int64_t o = at[r];
      cp_async16(dst + (r * RS + f) * 4, static_cast<const float*>(x) + (o >= 0 ? o + f : 0), o >= 0);
    }
  };
  __syncthreads();  // what came before is done with shared memory
  if (tid < BN) sat[tid] = find(0);
  for (int c = tid; c < BM * (D / 4); c += NT) {
    const int r = c / (D / 4), f = c % (D / 4) * 4, t = (first + r) / p.G;
    const bool on = r < rows;
    const float* x = static_cast<const float*>(p.q);
    if (on) x += (w.q.row + t) * p.ld_q + (int64_t)(w.h * p.G + first + r - t * p.G) * D + f;
    cp_async16(bq + (r * RS + f) * 4, x, on);
  }
  __syncthreads();
  copy(bk, p.k, sat);
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
    const int k0 = k_first + j * BN;
    const int64_t* at = sat + (j & 1) * BN;
    const int64_t next = find(j + 1);
    __syncthreads();  // V, P and places of the tile before are read
    copy(bv, p.v, at);
    cp_async_commit();
    if (tid < BN) sat[((j + 1) & 1) * BN + tid] = next;
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
    bool hidden[KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) hidden[c] = at[tx + 16 * c] < 0;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int row = RPT * ty + r;
      const uint32_t* mask = p.mask + (int64_t)(w.q.row + (first + min(row, rows - 1)) / p.G) * TREE_WORDS;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int d = k0 + tx + 16 * c - ctx;  // drafted token
        // (rounded before the maximum and the subtraction: the largest weight is 1)
        s[r][c] = __fmul_rn(s[r][c] + s2[r][c], p.sl2);
        if (hidden[c] || (d >= 0 && !((mask[d >> 5] >> (d & 31)) & 1u))) s[r][c] = -INFINITY;
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
        sp[row * PS + tx + 16 * c] = s[r][c];
      }
    }
    __syncthreads();  // K is read, P written
    if (j + 1 < nt) copy(bk, p.k, sat + ((j + 1) & 1) * BN);
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
        const float4 wv = *reinterpret_cast<const float4*>(sp + (RPT * ty + r) * PS + f);
        const float ww[4] = {wv.x, wv.y, wv.z, wv.w};
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
    if (whole) {
      const int t = (first + row) / p.G, head = w.h * p.G + first + row - t * p.G;
      const float inv = 1.0f / l[r];  // (l = 0: no score, 0 / 0)
      float* out = static_cast<float*>(p.o) + (w.q.row + t) * p.ld_o + (int64_t)head * D;
      if (tx == 0 && p.lse != nullptr)
        p.lse[(int64_t)(w.q.row + t) * p.nq + head] = (m[r] + log2f(l[r])) * LN2;
#pragma unroll
      for (int c = 0; c < OC; ++c)
        *reinterpret_cast<float4*>(out + 4 * tx + 64 * c) =
            make_float4(acc[r][4 * c] * inv, acc[r][4 * c + 1] * inv, acc[r][4 * c + 2] * inv,
                        acc[r][4 * c + 3] * inv);
    } else {
      if (tx == 0) p.ml[(int64_t)part * p.rows + row] = make_float2(m[r], l[r]);
#pragma unroll
      for (int c = 0; c < OC; ++c)
        *tree_part_at(p, part, D, tx + 16 * c, row) =
            make_float4(acc[r][4 * c], acc[r][4 * c + 1], acc[r][4 * c + 2], acc[r][4 * c + 3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(NT, 2) tree_f32_kernel(const TreeParams p) {
  extern __shared__ __align__(16) float sh[];
  pdl_wait();     // everything the call reads may come from the kernel before
  pdl_trigger();  // the join may start up; it waits for this kernel's end
  TreeSegs<CutF32<D>> sg;
  if (!sg.begin(p, blockIdx.x)) return;
  TreeSeg w;
  while (sg.next(p, w)) {
    const bool whole = sg.whole(w);
    const int part = tree_part(blockIdx.x, sg.begin_at, w.at);
    // the smallest form that holds the rows
    if (w.rows <= 16) run_rows<D, 2>(p, w, whole, part, sh);
    else if (w.rows <= 32) run_rows<D, 4>(p, w, whole, part, sh);
    else run_rows<D, 8>(p, w, whole, part, sh);
  }
  cp_async_wait<0>();
}

template <int D>
mgb_status launch_d(const TreeParams& p, cudaStream_t st) {
  using C = Cfg<D>;
  auto k = tree_f32_kernel<D>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  const mgb_status s = launch_pdl(k, CutF32<D>::RANGES, NT, C::SMEM, st, p);
  return s != MGB_OK ? s : tree_join<float, D>(p, CutF32<D>::RANGES, st);
}

}  // namespace

mgb_status attention_tree_f32(const TreeParams& p, int d, cudaStream_t st) {
  return d == 64 ? launch_d<64>(p, st) : launch_d<128>(p, st);
}

}  // namespace mgb
