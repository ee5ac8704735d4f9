// Appending a step's keys and values to a paged cache, with the rotary
// rotation of queries and keys on the way.
//
// Row t of sequence s (rows cu[s] .. cu[s+1] - 1, length len[s] after the
// step) has position p = len[s] - (cu[s+1] - cu[s]) + t - cu[s]. The first
// rot elements of each q and k head rotate in pairs, a' = a c - b s,
// b' = a s + b c with (c, s) = rope[p][j]; k' and v go to slot p % page_size of
// page table[s][p / page_size].
//
// Bound: HBM (each element read once; q' once, k' twice, v once written; the
// table's row is 4 bytes per rotated element and stays in L2 for the heads of
// one token). A thread owns a unit: the two 16-byte vectors of one head whose
// elements pair up (half split: vectors u and u + rot / (2 VN), so the pair
// partners sit at the same place of the two vectors; interleaved: vectors 2u
// and 2u + 1). Both read the same 2 VN floats of the table row, VN u onwards.
// The owner both reads and writes its unit, so the output may be the input.
//
// Each group of threads of a block (threadIdx.y) takes one token. A thread
// requests UB of its units before it needs to know where they go; meanwhile
// the group's first warp finds the token's sequence, position and page (a
// 32-way search over cu, then two dependent loads).
#include "common.cuh"
#include "internal.h"

namespace mgb {

namespace {

constexpr int MAX_GROUPS = 8;       // tokens per block
constexpr int FEW_THREADS = 512;    // of a block at most, with few tokens
constexpr int MANY_THREADS = 128;   // .. with many

struct AppendParams {
  int tokens, n_seqs, nq, nkv, rot;
  int units_head;              // units per head
  uint32_t m_head;             // 2^32 / units_head, rounded up; 0 for one unit
  int units;                   // per token: (nq + 2 nkv) heads (0 q heads without q_out)
  int page_size, n_pages, d;
  const int32_t *cu, *lens, *table;
  int64_t ld_table, s_page, s_tok, s_head;
  const float* rope;
  const char *q, *k, *v;
  char *q_out, *k_out, *k_pool, *v_pool;
  int64_t ld_q, ld_kv, ld_qo, ld_ko;
  int whole;                   // lengths are the rows' numbers (or 0)
  int cap;                     // positions below this: the table's and the rotary table's
  unsigned check_blocks;       // the last blocks, which check cu
  int* err;
};

// The largest s in [0, n] with s == 0 or cu[s] <= t (whole warp, same result in
// every lane). Reads cu[1 .. n] only, whatever they hold.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool le = i <= hi && cu[i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <typename T>
struct Vec {
  static constexpr int VN = 16 / sizeof(T);
  __device__ static void unpack(const uint4& w, float (&f)[VN]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        const float2 p = unpack_bf16x2(u[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      } else {
        f[i] = __uint_as_float(u[i]);
      }
    }
  }
  __device__ static uint4 pack(const float (&f)[VN]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) u[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      else u[i] = __float_as_uint(f[i]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Rotates the unit's VN pairs; cs = the unit's 2 VN table floats.
template <typename T, bool INTER>
__device__ __forceinline__ void rotate(uint4& w0, uint4& w1,
                                       const float4 (&cs)[Vec<T>::VN / 2]) {
  constexpr int VN = Vec<T>::VN;
  float x[VN], y[VN];
  Vec<T>::unpack(w0, x);
  Vec<T>::unpack(w1, y);
#pragma unroll
  for (int i = 0; i < VN / 2; ++i) {
    const float4 t = cs[i];  // (c, s) of pairs 2i and 2i + 1
    const float c[2] = {t.x, t.z}, s[2] = {t.y, t.w};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * i + e;
      // the pair's two elements: (x[j], y[j]), or neighbours of one vector
      float* v = j < VN / 2 ? x : y;
      float& a = INTER ? v[(2 * j) % VN] : x[j];
      float& b = INTER ? v[(2 * j + 1) % VN] : y[j];
      const float a0 = a, b0 = b;
      a = fmaf(a0, c[e], -(b0 * s[e]));
      b = fmaf(a0, s[e], b0 * c[e]);
    }
  }
  w0 = Vec<T>::pack(x);
  w1 = Vec<T>::pack(y);
}

template <typename T, int UB, bool INTER>
__global__ void __launch_bounds__(UB == 1 ? FEW_THREADS : MANY_THREADS, UB == 1 ? 1 : 8)
    kv_append_kernel(const AppendParams p) {
  constexpr int VN = Vec<T>::VN;
  __shared__ int s_pos[MAX_GROUPS];       // -1: nothing to do for the token
  __shared__ int64_t s_slot[MAX_GROUPS];  // element offset in the pools, head 0
  const int g = threadIdx.y;
  const int t = blockIdx.x * blockDim.y + g;
  const int rot_units = p.rot / (2 * VN);

  // the unit's two vectors in its row, for q / k / v of token t
  auto locate = [&](int u, int& head, int& e0, int& e1, int& ju) {
    head = p.m_head == 0 ? u : (int)__umulhi((uint32_t)u, p.m_head);  // u / units_head
    const int w = u - head * p.units_head;
    ju = w < rot_units ? w * VN : -1;  // first table pair of the unit
    if (INTER || ju < 0) {
      e0 = 2 * w * VN;
      e1 = e0 + VN;
    } else {
      e0 = w * VN;
      e1 = e0 + p.rot / 2;
    }
  };
  const int q_heads = p.q_out != nullptr ? p.nq : 0;
  auto src = [&](int head) -> const T* {
    if (head < q_heads) return reinterpret_cast<const T*>(p.q) + t * p.ld_q + (int64_t)head * p.d;
    head -= q_heads;
    if (head < p.nkv) return reinterpret_cast<const T*>(p.k) + t * p.ld_kv + (int64_t)head * p.d;
    return reinterpret_cast<const T*>(p.v) + t * p.ld_kv + (int64_t)(head - p.nkv) * p.d;
  };
  uint4 a[UB], b[UB];
  auto load = [&](int u0) {  // units u0, u0 + blockDim.x, ..
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const int u = u0 + i * blockDim.x;
      if (u < p.units && t < p.tokens) {
        int head, e0, e1, ju;
        locate(u, head, e0, e1, ju);
        const T* x = src(head);
        a[i] = *reinterpret_cast<const uint4*>(x + e0);
        b[i] = *reinterpret_cast<const uint4*>(x + e1);
      }
    }
  };
  pdl_wait();  // everything the call reads may come from the kernel before
  load(threadIdx.x);

  const unsigned back = gridDim.x - 1 - blockIdx.x;
  if (back < p.check_blocks) {
    // Every offset is checked once, by the grid's last threads (which start last and,
    // in a call of one block, are not the warp that looks its token up): whatever
    // sequence the search below finds in offsets that are not sorted, the call
    // reports them.
    const int nt = blockDim.x * blockDim.y;
    for (int64_t i = (int64_t)back * nt + nt - 1 - (g * blockDim.x + threadIdx.x); i < p.n_seqs;
         i += (int64_t)p.check_blocks * nt) {
      const int c0 = p.cu[i], c1 = p.cu[i + 1];
      if (c0 < 0 || c1 < c0 || c1 > p.tokens || (i == 0 && c0 != 0)) record_error(p.err, kErrIndex);
    }
  }
  if (threadIdx.x < 32 && t < p.tokens) {
    int s = t, first = t, behind = t + 1;  // the sequence's rows first .. behind - 1
    int before = 0;                        // offset of the sequence before
    if (p.cu != nullptr) {
      s = find_seq(p.cu, p.n_seqs, t);
      if (s < p.n_seqs) {
        if (s > 0) before = p.cu[s - 1];
        first = p.cu[s];
        behind = p.cu[s + 1];
      }
    }
    int pos = -1;
    int64_t slot = 0;
    const int len = s < p.n_seqs ? p.lens[s] : 0;
    if (len != 0) {  // else padding, or behind the last sequence
      // (a row outside its sequence's, by bad offsets, would go over cached tokens or
      // behind the sequence's length)
      const bool in = first >= max(before, 0) && first <= t && t < behind && behind <= p.tokens &&
                      (!p.whole || len == behind - first);
      const int at = in ? max(len, 0) - (behind - t) : -1;
      bool ok = at >= 0 && at < p.cap;
      if (ok) {
        const int pg = at / p.page_size;
        const int page = p.table[s * p.ld_table + pg];
        ok = page >= 0 && page < p.n_pages;
        slot = page * p.s_page + (at - pg * p.page_size) * p.s_tok;
      }
      if (ok) pos = at;
      else if (threadIdx.x == 0) record_error(p.err, kErrIndex);
    }
    if (threadIdx.x == 0) {
      s_pos[g] = pos;
      s_slot[g] = slot;
    }
  }
  __syncthreads();

  if (t >= p.tokens) return;
  const int pos = s_pos[g];
  if (pos < 0) return;
  const int64_t slot = s_slot[g];
  // the table floats of the pairs cs_at ..: the same for all of a thread's units
  // when the group's threads are a multiple of a head's units
  float4 cs[VN / 2];
  int cs_at = -1;
  for (int u0 = threadIdx.x; u0 < p.units; u0 += UB * blockDim.x) {
    if (u0 != threadIdx.x) load(u0);
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const int u = u0 + i * blockDim.x;
      if (u >= p.units) break;
      int head, e0, e1, ju;
      locate(u, head, e0, e1, ju);
      const bool is_q = head < q_heads;
      const int kh = head - q_heads;  // k heads, then v heads
      const bool is_k = !is_q && kh < p.nkv;
      if (ju >= 0 && (is_q || is_k)) {
        if (ju != cs_at) {
          const float4* x = reinterpret_cast<const float4*>(p.rope + (int64_t)pos * p.rot + 2 * ju);
#pragma unroll
          for (int j = 0; j < VN / 2; ++j) cs[j] = x[j];
          cs_at = ju;
        }
        rotate<T, INTER>(a[i], b[i], cs);
      }
      if (is_q || (is_k && p.k_out != nullptr)) {
        T* o = is_q ? reinterpret_cast<T*>(p.q_out) + t * p.ld_qo + (int64_t)head * p.d
                    : reinterpret_cast<T*>(p.k_out) + t * p.ld_ko + (int64_t)kh * p.d;
        *reinterpret_cast<uint4*>(o + e0) = a[i];
        *reinterpret_cast<uint4*>(o + e1) = b[i];
      }
      if (!is_q) {
        T* o = is_k ? reinterpret_cast<T*>(p.k_pool) + kh * p.s_head
                    : reinterpret_cast<T*>(p.v_pool) + (kh - p.nkv) * p.s_head;
        o += slot;
        *reinterpret_cast<uint4*>(o + e0) = a[i];
        *reinterpret_cast<uint4*>(o + e1) = b[i];
      }
    }
  }
}

template <typename T, int UB>
mgb_status launch(AppendParams p, bool inter, int most, cudaStream_t st) {
  // threads along a token's units (whole warps, up to `most`), and groups of
  // them until a block has about 128
  const int x = p.units >= most ? most : (p.units + 31) / 32 * 32;
  int y = x >= 128 ? 1 : 128 / x;
  if (y > MAX_GROUPS) y = MAX_GROUPS;
  if (y > p.tokens) y = p.tokens;
  const int grid = (int)(((int64_t)p.tokens + y - 1) / y);
  if (p.cu != nullptr) {
    const int64_t all = ((int64_t)p.n_seqs + x * y - 1) / (x * y);
    p.check_blocks = (unsigned)(all < grid ? all : grid);
  }
  LaunchScope scope(PROF_KV_APPEND, st);
  return launch_pdl(inter ? kv_append_kernel<T, UB, true> : kv_append_kernel<T, UB, false>, grid,
                    dim3(x, y), 0, st, p);
}

template <typename T>
mgb_status launch_t(const AppendParams& p, bool inter, cudaStream_t st) {
  // Few tokens: as many threads as units, one each (one token 3.0 us; 0.5 us more
  // with 128 threads), while all blocks are resident at once: one token per sequence,
  // bf16 and 384 units, 304 tokens 3.7 us (the other form 4.0), 456 tokens 6.3 (4.3),
  // 912 9.4 (5.4); float32 and 192 units 2.9 (3.2), 3.1 (3.4), 3.8 (3.9).
  // Many: small blocks with three units per thread, eight per SM (4699 tokens of 384
  // units, 127 MB, 23.7 us, 5.4 TB/s; 1.6 more with six, 24 and more with blocks of 192
  // threads and two units, 30 with 384 and one). There the chain cu, length, page of
  // each token is the bound, not DRAM (41 % busy). Groups that take runs of tokens and
  // find their places together need 27 us: too few of them are left to hide the rest.
  return p.tokens <= 2 * device_sm_count() ? launch<T, 1>(p, inter, FEW_THREADS, st)
                                           : launch<T, 3>(p, inter, MANY_THREADS, st);
}

}  // namespace

mgb_status check_kv_cache(const mgb_kv_cache* c, int n_seqs) {
  if (c == nullptr) return MGB_ERR_INVALID_ARG;
  if (c->dtype != MGB_BF16 && c->dtype != MGB_F32) return MGB_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->n_kv_heads < 1 ||
      c->head_dim < 1 || c->stride_page < 0 || c->stride_token < 0 || c->stride_head < 0 ||
      (n_seqs > 1 && c->ld_table < c->max_pages))
    return MGB_ERR_INVALID_ARG;
  if (!c->k || !c->v || (n_seqs > 0 && !c->block_table)) return MGB_ERR_INVALID_ARG;
  const int vn = c->dtype == MGB_BF16 ? 8 : 4;
  if (!is_aligned16(c->k) || !is_aligned16(c->v) || c->stride_page % vn || c->stride_token % vn ||
      c->stride_head % vn || (reinterpret_cast<uintptr_t>(c->block_table) & 3u))
    return MGB_ERR_MISALIGNED;
  // slots and heads of a page do not overlap
  if ((c->page_size > 1 && c->stride_token < c->head_dim) ||
      (c->n_kv_heads > 1 && c->stride_head < c->head_dim) ||
      (c->n_pages > 1 && c->stride_page < c->head_dim))
    return MGB_ERR_INVALID_ARG;
  return MGB_OK;
}

}  // namespace mgb

using namespace mgb;

extern "C" mgb_status mgb_kv_append(const mgb_kv_append_desc* d, const mgb_kv_cache* c,
                                    const int32_t* cu_seqlens, const int32_t* seq_lens,
                                    const float* rope, const void* q, const void* k, const void* v,
                                    int64_t ld_q, int64_t ld_kv, void* q_out, int64_t ld_qo,
                                    void* k_out, int64_t ld_ko, void* stream) {
  if (fault_injected()) return MGB_ERR_INVALID_ARG;
  if (d == nullptr || d->tokens < 0 || d->n_seqs < 0 || d->rot_dim < 0 || d->rope_len < 0 ||
      (d->interleaved & ~1) || (d->whole & ~1))
    return MGB_ERR_INVALID_ARG;
  mgb_status s = check_kv_cache(c, d->n_seqs);
  if (s != MGB_OK) return s;
  const int vn = c->dtype == MGB_BF16 ? 8 : 4;
  if (c->head_dim > 256 || c->head_dim % (2 * vn) || d->rot_dim % (2 * vn))
    return MGB_ERR_UNSUPPORTED;
  if (d->rot_dim > c->head_dim || (d->rot_dim > 0 && (d->rope_len < 1 || rope == nullptr)))
    return MGB_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && d->tokens != d->n_seqs) return MGB_ERR_INVALID_ARG;
  if (q_out != nullptr && (d->n_q_heads < 1 || q == nullptr)) return MGB_ERR_INVALID_ARG;
  if (d->tokens > 0 && (!k || !v || (d->n_seqs > 0 && !seq_lens))) return MGB_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)d->n_q_heads * c->head_dim, wk = (int64_t)c->n_kv_heads * c->head_dim;
  // (units x units per head stays below 2^32, for the division by multiplication)
  if (wk >= ((int64_t)1 << 28) || (q_out != nullptr && wq >= ((int64_t)1 << 28)))
    return MGB_ERR_INVALID_ARG;
  if (ld_kv < wk || (k_out != nullptr && ld_ko < wk) ||
      (q_out != nullptr && (ld_q < wq || ld_qo < wq)))
    return MGB_ERR_INVALID_ARG;
  if ((q_out != nullptr && q_out == q && ld_qo != ld_q) ||
      (k_out != nullptr && k_out == k && ld_ko != ld_kv))
    return MGB_ERR_INVALID_ARG;
  const void* ps[] = {k, v, k_out, q_out, rope, q_out ? q : nullptr};
  for (const void* x : ps)
    if (!is_aligned16(x)) return MGB_ERR_MISALIGNED;
  if (ld_kv % vn || (k_out && ld_ko % vn) || (q_out && (ld_q % vn || ld_qo % vn)) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return MGB_ERR_MISALIGNED;
  s = check_arch();
  if (s != MGB_OK) return s;
  if (d->tokens == 0 || d->n_seqs == 0) return MGB_OK;
  AppendParams p{};
  p.tokens = d->tokens; p.n_seqs = d->n_seqs; p.nq = d->n_q_heads; p.nkv = c->n_kv_heads;
  p.rot = d->rot_dim; p.whole = d->whole; p.d = c->head_dim;
  p.units_head = c->head_dim / (2 * vn);
  p.m_head = p.units_head == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + p.units_head - 1) / p.units_head);
  p.units = ((q_out ? p.nq : 0) + 2 * p.nkv) * p.units_head;
  int64_t cap = (int64_t)c->max_pages * c->page_size;
  if (d->rot_dim > 0 && cap > d->rope_len) cap = d->rope_len;
  p.cap = (int)(cap < INT32_MAX ? cap : INT32_MAX);
  p.page_size = c->page_size; p.n_pages = c->n_pages;
  p.cu = cu_seqlens; p.lens = seq_lens; p.table = c->block_table; p.ld_table = c->ld_table;
  p.s_page = c->stride_page; p.s_tok = c->stride_token; p.s_head = c->stride_head;
  p.rope = rope;
  p.q = static_cast<const char*>(q); p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.q_out = static_cast<char*>(q_out); p.k_out = static_cast<char*>(k_out);
  p.k_pool = static_cast<char*>(c->k); p.v_pool = static_cast<char*>(c->v);
  p.ld_q = ld_q; p.ld_kv = ld_kv; p.ld_qo = ld_qo; p.ld_ko = ld_ko;
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return c->dtype == MGB_BF16 ? launch_t<bf16>(p, d->interleaved != 0, st)
                              : launch_t<float>(p, d->interleaved != 0, st);
}
