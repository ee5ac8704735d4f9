// Cached tokens moved inside the cache: an accepted path to the front of its
// draft's slots, and slots of pages to other pages. Bound: HBM (every byte read and
// written once), and for the few slots of a path the launch and the reads of where
// they are.
#include "tree.cuh"

namespace mgb {

namespace {

constexpr int NT = 128;

struct MoveParams {
  char *k, *v;
  const int32_t* table;
  int64_t s_page, s_tok, s_head, ld_table;  // strides in 16-byte vectors but ld_table
  int n_pages, page_size, nkv, ch, cap;     // ch: vectors of a head
  int* err;
};

// ---------------------------------------------------------------- accept
// Block (s, y): NT of the sequence's 2 nkv ch columns of vectors (keys, then values). The
// i-th token of the path has index a_i >= i in the draft, growing with i, so a thread
// that moves its column's vectors in order, BATCH reads and then their writes, never
// reads a slot it has written: the writes end at i + BATCH - 1 < a_{i + BATCH}. 200 sequences of 8 to
// 61 drafted tokens 2.6 us, one 2.3: launch, and the reads of where the slots are.
constexpr int BATCH = 8;

__global__ void __launch_bounds__(NT) kv_accept_kernel(const MoveParams p, const TreeSeq* seq,
                                                       const uint32_t* mask, const int32_t* accepted,
                                                       int32_t* new_lens) {
  __shared__ int path[TREE_MAX];
  __shared__ int64_t from[TREE_MAX], to[TREE_MAX];  // vectors; from -1: stays
  pdl_wait();
  const int s = blockIdx.x, tid = threadIdx.x;
  const TreeSeq q = seq[s];
  const int ctx = q.len - q.m;
  int leaf = accepted[s];
  if (leaf < -1 || leaf >= q.m) {
    // (no drafted tokens: padding, or a sequence that the prepare has reported)
    if (blockIdx.y == 0 && tid == 0 && q.m > 0) record_error(p.err, kErrIndex);
    leaf = -1;
  }
  uint32_t words[TREE_WORDS];
  int n = 0, at[TREE_WORDS];
  if (leaf >= 0) {
#pragma unroll
    for (int i = 0; i < TREE_WORDS; ++i) words[i] = mask[(int64_t)(q.row + leaf) * TREE_WORDS + i];
#pragma unroll
    for (int i = 0; i < TREE_WORDS; ++i) {
      at[i] = n;
      n += __popc(words[i]);
    }
  }
  const bool fits = q.len <= p.cap;
  if (blockIdx.y == 0 && tid == 0) {
    if (new_lens != nullptr) new_lens[s] = q.m > 0 ? ctx + n : q.len;
    if (q.m > 0 && !fits) record_error(p.err, kErrIndex);
  }
  if (n == 0 || !fits) return;  // (the same for the whole block)
#pragma unroll
  for (int w = 0; w < TREE_WORDS; ++w)
    if (tid < 32 && ((words[w] >> tid) & 1u)) path[at[w] + __popc(words[w] & ((1u << tid) - 1u))] = 32 * w + tid;
  __syncthreads();
  const int32_t* table = p.table + (int64_t)s * p.ld_table;
  auto place = [&](int slot, int64_t& x) {
    const int i = slot / p.page_size, page = table[i];
    x = page * p.s_page + (slot - i * p.page_size) * p.s_tok;
    return page >= 0 && page < p.n_pages;
  };
  for (int i = tid; i < n; i += NT) {
    int64_t a = -1, b = 0;
    if (path[i] != i) {
      const bool ok_a = place(ctx + path[i], a), ok_b = place(ctx + i, b);
      if (!ok_a || !ok_b) {
        record_error(p.err, kErrIndex);
        a = -1;
      }
    }
    from[i] = a;
    to[i] = b;
  }
  __syncthreads();
  const int col = blockIdx.y * NT + tid, half = p.nkv * p.ch;
  if (col >= 2 * half) return;
  const int hc = col < half ? col : col - half, head = hc / p.ch;
  uint4* x = reinterpret_cast<uint4*>(col < half ? p.k : p.v) + head * p.s_head + (hc - head * p.ch);
  for (int i0 = 0; i0 < n; i0 += BATCH) {
    uint4 y[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < n && from[i0 + i] >= 0) y[i] = x[from[i0 + i]];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < n && from[i0 + i] >= 0) x[to[i0 + i]] = y[i];
  }
}

// ---------------------------------------------------------------- copy
// A block takes COPY_VECS vectors of one page's keys or values at a time, COPY_PER per
// thread, all requested before the first is stored. 1000 pages of 256 KB (524 MB read and
// written) 84 us, 6.2 TB/s, 0.93 of a plain copy; three pages 2.4 us. (256 threads and 8 vectors
// 91 and 4.0, 8 blocks per SM 86, one vector 112 and 1.8.)
constexpr int CT = 128, COPY_PER = 4, COPY_BLOCKS = 24, COPY_VECS = CT * COPY_PER;  // blocks per SM

__global__ void __launch_bounds__(CT) kv_copy_kernel(const MoveParams p, int n, int parts, int slot_inner,
                                                     const int32_t* src, const int32_t* dst,
                                                     const int32_t* slots) {
  pdl_wait();
  const int64_t all = (int64_t)n * 2 * parts;
  for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
    const int part = (int)(u % parts);
    const int64_t pv = u / parts;
    const int i = (int)(pv >> 1);
    const int a = src[i], b = dst[i], c = slots != nullptr ? slots[i] : p.page_size;
    if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages || c < 0 || c > p.page_size) {
      if (threadIdx.x == 0) record_error(p.err, kErrIndex);
      continue;
    }
    if (a == b) continue;
    uint4* x = reinterpret_cast<uint4*>((pv & 1) ? p.v : p.k);
    const int64_t vecs = (int64_t)c * p.nkv * p.ch;
    uint4 y[COPY_PER];
    int64_t off[COPY_PER];
#pragma unroll
    for (int j = 0; j < COPY_PER; ++j) {
      const int64_t e = (int64_t)part * COPY_VECS + j * CT + threadIdx.x;
      off[j] = -1;
      if (e < vecs) {
        const int64_t row = e / p.ch;
        const int64_t outer = row / (slot_inner ? c : p.nkv), inner = row - outer * (slot_inner ? c : p.nkv);
        const int64_t slot = slot_inner ? inner : outer, head = slot_inner ? outer : inner;
        off[j] = slot * p.s_tok + head * p.s_head + (e - row * p.ch);
        y[j] = x[a * p.s_page + off[j]];
      }
    }
#pragma unroll
    for (int j = 0; j < COPY_PER; ++j)
      if (off[j] >= 0) x[b * p.s_page + off[j]] = y[j];
  }
}

// 32-bit numbers in units of 16 bytes; false: head rows are not whole vectors.
bool move_params(const mgb_kv_cache* c, MoveParams& p) {
  const int vn = c->dtype == MGB_BF16 ? 8 : 4;
  if (c->head_dim % vn) return false;
  p.k = static_cast<char*>(c->k);
  p.v = static_cast<char*>(c->v);
  p.table = c->block_table;
  p.s_page = c->stride_page / vn; p.s_tok = c->stride_token / vn; p.s_head = c->stride_head / vn;
  p.ld_table = c->ld_table;
  p.n_pages = c->n_pages; p.page_size = c->page_size; p.nkv = c->n_kv_heads; p.ch = c->head_dim / vn;
  const int64_t cap = (int64_t)c->max_pages * c->page_size;
  p.cap = cap < TREE_LONGEST ? (int)cap : TREE_LONGEST;
  return true;
}

}  // namespace
}  // namespace mgb

using namespace mgb;

extern "C" {

mgb_status mgb_kv_accept(const mgb_attention_tree_plan* plan, const mgb_kv_cache* c,
                         const int32_t* accepted, int32_t* new_lens, void* stream) {
  if (fault_injected()) return MGB_ERR_INVALID_ARG;
  mgb_status s = check_tree_plan(plan);
  if (s != MGB_OK) return s;
  s = check_kv_cache(c, plan->n_seqs);
  if (s != MGB_OK) return s;
  if (c->n_kv_heads != plan->n_kv_heads || c->head_dim != plan->head_dim ||
      (plan->n_seqs > 0 && accepted == nullptr))
    return MGB_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(accepted) & 3u) || (reinterpret_cast<uintptr_t>(new_lens) & 3u))
    return MGB_ERR_MISALIGNED;
  // (a block per sequence: one would write what another has yet to read)
  const uintptr_t from = reinterpret_cast<uintptr_t>(accepted), to = reinterpret_cast<uintptr_t>(new_lens);
  const uintptr_t size = sizeof(int32_t) * (uintptr_t)plan->n_seqs;
  if (new_lens != nullptr && from < to + size && to < from + size) return MGB_ERR_INVALID_ARG;
  MoveParams p{};
  if (!move_params(c, p)) return MGB_ERR_UNSUPPORTED;
  const int64_t blocks = ((int64_t)2 * p.nkv * p.ch + NT - 1) / NT;
  if (blocks > 65535) return MGB_ERR_UNSUPPORTED;
  s = check_arch();
  if (s != MGB_OK) return s;
  if (plan->n_seqs == 0) return MGB_OK;
  const TreeLayout l =
      tree_layout(plan->n_seqs, plan->tokens, plan->n_q_heads, plan->n_kv_heads, plan->head_dim);
  const char* b = static_cast<const char*>(plan->ws);
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(PROF_KV_MOVE, st);
  return launch_pdl(kv_accept_kernel, dim3((unsigned)plan->n_seqs, (unsigned)blocks), dim3(NT), 0, st, p,
                    reinterpret_cast<const TreeSeq*>(b + l.seq),
                    reinterpret_cast<const uint32_t*>(b + l.mask), accepted, new_lens);
}

mgb_status mgb_kv_copy_pages(const mgb_kv_cache* c, int32_t n_copies, const int32_t* src,
                             const int32_t* dst, const int32_t* slots, void* stream) {
  if (fault_injected() || n_copies < 0) return MGB_ERR_INVALID_ARG;
  mgb_status s = check_kv_cache(c, 0);
  if (s != MGB_OK) return s;
  if (n_copies > 0 && (src == nullptr || dst == nullptr)) return MGB_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(src) & 3u) || (reinterpret_cast<uintptr_t>(dst) & 3u) ||
      (reinterpret_cast<uintptr_t>(slots) & 3u))
    return MGB_ERR_MISALIGNED;
  MoveParams p{};
  if (!move_params(c, p)) return MGB_ERR_UNSUPPORTED;
  const int64_t parts = ((int64_t)p.page_size * p.nkv * p.ch + COPY_VECS - 1) / COPY_VECS;
  if (parts > INT32_MAX) return MGB_ERR_UNSUPPORTED;
  s = check_arch();
  if (s != MGB_OK) return s;
  if (n_copies == 0) return MGB_OK;
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  const int64_t all = 2 * (int64_t)n_copies * parts, most = (int64_t)device_sm_count() * COPY_BLOCKS;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(PROF_KV_MOVE, st);
  return launch_pdl(kv_copy_kernel, (int)(all < most ? all : most), dim3(CT), 0, st, p, (int)n_copies,
                    (int)parts, (int)(p.s_tok < p.s_head), src, dst, slots);
}

}  // extern "C"
