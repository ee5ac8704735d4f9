// Attention of one new token per sequence over a paged key/value cache.
//
// Per sequence s and query head h: o = softmax(q_h K_g^T / sqrt(d)) V_g over
// the first len[s] cached tokens, g = h / (nq / nkv). Bound: HBM (each cached
// key and value is used once per query head of its group).
//
// Work is cut into units: 64 (d = 64: 128) consecutive cached tokens of one
// (sequence, KV head, group of at most 16 query heads). An item is all units of one
// sequence and head group. Items stand one behind the other on a cost axis,
// sequence by sequence, head by head: an item with n units takes n UNIT + ITEM,
// its unit t beginning at t UNIT (ITEM is the fixed cost of an item: its
// queries, the join of the warps, the store). CTA c takes the units that begin
// in [c chunk, (c + 1) chunk): the same cost for every CTA whatever the lengths
// are. (All units of an item of at most WHOLE units count as beginning at its
// start: splitting it would cost more than it evens out.) An item that lies in
// one range is finished there. An item that spans CTAs is split: each CTA leaves
// its unnormalised sums, maximum and row sum in the workspace, and the last one
// to arrive (a counter per first CTA of a split item) joins the parts in CTA
// order, so results do not depend on who was last.
//
// The prepare kernel derives the ranges from the lengths (they are the same
// for every layer of a model's step) and zeroes the counters; each split item
// leaves its counter at zero again.
//
// Within a CTA (four warps) a unit is dealt out to the warps in stages of 4 KB of
// keys and as much of values, and each warp keeps its own running maximum, row
// sums and output sums; the warps' sums are joined at the end of an item. Each
// warp streams its tokens through a private ring in shared memory by 16-byte
// asynchronous copies, so the main loop has no CTA-wide barrier, any page size
// and any page layout works, and tokens past the length or of a bad page are never
// read (zero fill, weight 0). 2 (d = 64: 3) CTAs per SM keep 128 (96) KB in flight per SM.
//   bf16: products on mma.sync m16n8k16, transposed: S^T = K Q^T with 16 tokens
//   as the rows and the query heads as the columns, and O^T = V^T P^T with d as
//   the rows. There is one query token per sequence, so an item has at most 16
//   query rows and the 128 rows of a tcgen05 tile would stand empty; on the
//   narrow side the heads come in eights, and the products stay a small share of
//   the time.
//   float32: FFMA with a lane per (token, quarter of d) for the scores and a
//   lane per D / 32 columns for the output; the quarters' sums are dealt out so
//   that each lane keeps the softmax of a quarter of the heads.
//
// Measured: bf16, d = 128, 32 query and 8 KV heads: one sequence of 131001 cached
// tokens 88 us, 6.1 TB/s; 64 sequences of 33 to 16000 tokens 108 us, 6.3 TB/s (a
// copy reaches 6.79). d = 64, 16 query and KV heads, 200 sequences of 20 to 1200
// tokens: 44 us with the prepare kernel. float32, d = 128, 16 and 4 heads, 12
// sequences to 5000 tokens: 13.6 us for 49 MB; the start of the loads (2 us), the
// last CTAs' second item and the join (3 us) are as long as the copies.
#include "paged_rows.cuh"

namespace mgb {

namespace {

struct Layout {
  size_t header, start, counter, len, prefix, ml, part, total;
  int rows, groups;  // query heads per item at most; items per sequence
  int ctas;
};

Layout make_layout(int n, int nq, int nkv, int d) {
  Layout l;
  size_t o = 0;
  auto take = [&](size_t b) { const size_t at = o; o += (b + 255) & ~(size_t)255; return at; };
  const int G = nq / nkv, per = (G + MAXR - 1) / MAXR;
  l.rows = (G + per - 1) / per;
  l.groups = nkv * ((G + l.rows - 1) / l.rows);
  l.header = take(sizeof(Header));
  l.ctas = SMS * ctas_per_sm(d);
  l.start = take(sizeof(Start) * l.ctas);
  l.counter = take(4 * (size_t)l.ctas);
  l.len = take(4 * (size_t)n);
  l.prefix = take(8 * ((size_t)n + 1));
  l.ml = take(8 * (size_t)2 * l.ctas * l.rows);
  l.part = take(4 * (size_t)2 * l.ctas * l.rows * d);
  l.total = o;
  return l;
}

// ---------------------------------------------------------------- prepare
// One block: lengths copied (negative ones count as 0 and are an error), costs
// (per head group) summed up, the ranges' first units found, counters zeroed.
__global__ void __launch_bounds__(1024) decode_prepare_kernel(int n, int groups, int ctas, int tk, int item,
                                                              const int32_t* lens,
                                                              Header* hdr, Start* start,
                                                              uint32_t* counter, int32_t* len_out,
                                                              int64_t* prefix, int* err) {
  __shared__ int64_t warp_sum[32];
  __shared__ int64_t carry_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();  // the attention kernel may start up; it waits for this one's end
  int64_t carry = 0;
  for (int i = tid; i < ctas; i += 1024) counter[i] = 0;
  for (int base = 0; base < n; base += 1024) {
    const int i = base + tid;
    int64_t v = 0;
    if (i < n) {
      int len = lens[i];
      if (len < 0) {
        record_error(err, kErrIndex);
        len = 0;
      }
      len_out[i] = len;
      v = cost_of(tiles_of(len, tk), item);
    }
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int64_t w = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sum[lane] = w;
      if (lane == 31) carry_s = w;
    }
    __syncthreads();
    if (i < n) prefix[i] = carry + x - v + (warp > 0 ? warp_sum[warp - 1] : 0);
    carry += carry_s;
    __syncthreads();
  }
  if (tid == 0) prefix[n] = carry;
  __syncthreads();
  const int64_t cost = carry * groups;
  int64_t chunk = (cost + ctas - 1) / ctas;
  if (chunk < MIN_CHUNK) chunk = MIN_CHUNK;
  if (tid == 0) *hdr = Header{cost, chunk};
  for (int c = tid; c < ctas; c += 1024) {
    const int64_t u = c * chunk;
    Start st{cost, n, 0, 0, 0, 0, 0};
    if (u < cost) {
      int lo = 0, hi = n - 1;  // the largest s with prefix[s] * groups <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (prefix[mid] * groups <= u) lo = mid;
        else hi = mid - 1;
      }
      const int64_t per = prefix[lo + 1] - prefix[lo], r = u - prefix[lo] * groups;
      const int64_t h = r / per, into = r - h * per, t = (into + UNIT - 1) / UNIT;
      const int64_t nt = (per - item) / UNIT;
      st.at = prefix[lo] * groups + h * per;
      st.s = lo;
      st.h = (int)h;
      if (into == 0 || (nt > WHOLE && t < nt)) {
        st.t = (int)t;
      } else {  // the item's last unit begins before: the next item
        st.at += per;
        if (++st.h == groups) {
          st.h = 0;
          ++st.s;
        }
      }
      if (st.s < n) st.len = len_out[st.s];
      if (st.s + 1 < n) st.next_len = len_out[st.s + 1];
    }
    start[c] = st;
  }
}

template <typename T, int D, int NR>
mgb_status launch(const Params& p, cudaStream_t st) {
  using C = Cfg<T, D, NR>;
  auto k = paged_rows_kernel<T, D, NR, false>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  LaunchScope scope(PROF_ATTN_DECODE, st);
  return launch_pdl(k, SMS * ctas_per_sm(D), NT, C::SMEM, st, p);
}

// The smallest form that holds the item's query heads: the fewest products.
template <typename T, int D>
mgb_status launch_rows(const Params& p, cudaStream_t st) {
  if constexpr (sizeof(T) == 4)
    if (p.rows <= 4) return launch<T, D, 4>(p, st);
  return p.rows <= 8 ? launch<T, D, 8>(p, st) : launch<T, D, 16>(p, st);
}

mgb_status check_shape(int n, int nq, int nkv, int d) {
  if (n < 0 || nq < 1 || nkv < 1 || nq % nkv || nq > (1 << 20)) return MGB_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? MGB_OK : MGB_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace mgb

using namespace mgb;

extern "C" {

size_t mgb_attention_decode_ws_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                     int32_t head_dim) {
  if (check_shape(n_seqs, n_q_heads, n_kv_heads, head_dim) != MGB_OK) return 0;
  return make_layout(n_seqs, n_q_heads, n_kv_heads, head_dim).total;
}

mgb_status mgb_attention_decode_prepare(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                        int32_t head_dim, const int32_t* seq_lens, void* ws,
                                        size_t ws_bytes, mgb_attention_decode_plan* plan,
                                        void* stream) {
  if (fault_injected() || plan == nullptr) return MGB_ERR_INVALID_ARG;
  mgb_status s = check_shape(n_seqs, n_q_heads, n_kv_heads, head_dim);
  if (s != MGB_OK) return s;
  if (ws == nullptr || (n_seqs > 0 && seq_lens == nullptr)) return MGB_ERR_INVALID_ARG;
  if (!is_aligned16(ws) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u)) return MGB_ERR_MISALIGNED;
  const Layout l = make_layout(n_seqs, n_q_heads, n_kv_heads, head_dim);
  if (ws_bytes < l.total) return MGB_ERR_WORKSPACE_TOO_SMALL;
  s = check_arch();
  if (s != MGB_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return MGB_ERR_CUDA;
  char* b = static_cast<char*>(ws);
  if (n_seqs > 0) {
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LaunchScope scope(PROF_ATTN_DECODE, st);
    decode_prepare_kernel<<<1, 1024, 0, st>>>(
        n_seqs, l.groups, l.ctas, unit_tokens(head_dim), item_cost(head_dim), seq_lens,
        reinterpret_cast<Header*>(b + l.header),
        reinterpret_cast<Start*>(b + l.start), reinterpret_cast<uint32_t*>(b + l.counter),
        reinterpret_cast<int32_t*>(b + l.len), reinterpret_cast<int64_t*>(b + l.prefix), err);
    if (cudaGetLastError() != cudaSuccess) return MGB_ERR_CUDA;
  }
  *plan = mgb_attention_decode_plan{n_seqs, n_q_heads, n_kv_heads, head_dim, ws, ws_bytes};
  return MGB_OK;
}

mgb_status mgb_attention_decode(const mgb_attention_decode_plan* plan, const mgb_kv_cache* c,
                                const void* q, int64_t ld_q, void* o, int64_t ld_o, float* lse,
                                void* stream) {
  if (fault_injected() || plan == nullptr || plan->ws == nullptr) return MGB_ERR_INVALID_ARG;
  const int n = plan->n_seqs, nq = plan->n_q_heads, nkv = plan->n_kv_heads, d = plan->head_dim;
  mgb_status s = check_shape(n, nq, nkv, d);
  if (s != MGB_OK) return s;
  s = check_kv_cache(c, n);
  if (s != MGB_OK) return s;
  if (c->n_kv_heads != nkv || c->head_dim != d || (n > 0 && (!q || !o))) return MGB_ERR_INVALID_ARG;
  if (n > 1 && (ld_q < (int64_t)nq * d || ld_o < (int64_t)nq * d)) return MGB_ERR_INVALID_ARG;
  const int vn = c->dtype == MGB_BF16 ? 8 : 4;
  if (!is_aligned16(q) || !is_aligned16(o) || ld_q % vn || ld_o % vn || !is_aligned16(plan->ws) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MGB_ERR_MISALIGNED;
  const Layout l = make_layout(n, nq, nkv, d);
  if (plan->ws_bytes < l.total) return MGB_ERR_WORKSPACE_TOO_SMALL;
  if (o != nullptr && o == q) return MGB_ERR_INVALID_ARG;  // the CTAs of a split item read q late
  s = check_arch();
  if (s != MGB_OK) return s;
  if (n == 0) return MGB_OK;
  char* b = static_cast<char*>(plan->ws);
  Params p{};
  p.n = n; p.nkv = nkv; p.groups = l.groups; p.per_kv = l.groups / nkv; p.rows = l.rows;
  p.G = nq / nkv; p.nq = nq;
  p.hdr = reinterpret_cast<const Header*>(b + l.header);
  p.start = reinterpret_cast<const Start*>(b + l.start);
  p.counter = reinterpret_cast<uint32_t*>(b + l.counter);
  p.len = reinterpret_cast<const int32_t*>(b + l.len);
  p.ml = reinterpret_cast<float2*>(b + l.ml);
  p.part = reinterpret_cast<float*>(b + l.part);
  p.k = c->k; p.v = c->v; p.table = c->block_table;
  p.s_page = c->stride_page; p.s_tok = c->stride_token; p.s_head = c->stride_head;
  p.ld_table = c->ld_table;
  p.n_pages = c->n_pages; p.page_size = c->page_size;
  const int64_t cap = (int64_t)c->max_pages * c->page_size;
  p.cap = cap < INT32_MAX ? (int)cap : INT32_MAX;
  p.q = q; p.ld_q = ld_q; p.o = o; p.ld_o = ld_o; p.lse = lse;
  p.sl2 = LOG2E / sqrtf((float)d);
  p.err = device_error_word();
  if (p.err == nullptr) return MGB_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == MGB_BF16)
    return d == 64 ? launch_rows<bf16, 64>(p, st) : launch_rows<bf16, 128>(p, st);
  return d == 64 ? launch_rows<float, 64>(p, st) : launch_rows<float, 128>(p, st);
}

}  // extern "C"
