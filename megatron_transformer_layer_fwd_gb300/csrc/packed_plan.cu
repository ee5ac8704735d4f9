// Packed attention: the work lists from the row offsets, and the entry points.
//
// Block b of R query rows of a sequence costs the key tiles its rows see: for a
// causal sequence they grow with b, otherwise they are the sequence's. The
// attention kernels deal the entries out in snake order over the CTAs, which
// evens the sums out when the list is sorted by cost, so the list is counting-
// sorted here, longest first (1024 bins; costs beyond that share bins). Entries
// of one bin come out in no fixed order: that moves work between CTAs and
// changes no result, since every entry is computed by one CTA on its own.
#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mgb {

namespace {

constexpr int NTH = 1024;
constexpr int BINS = 1024;

struct Layout {
  size_t header, prefix, list256, list128, total;
  int64_t max256, max128;
};

Layout make_layout(int n, int tokens) {
  Layout l;
  size_t o = 0;
  auto take = [&](size_t b) { const size_t at = o; o += (b + 255) & ~(size_t)255; return at; };
  // a sequence has at most len / R + 1 blocks, and only if it has rows
  const int64_t live = n < tokens ? n : tokens;
  l.max256 = tokens / 256 + live;
  l.max128 = tokens / 128 + live;
  l.header = take(2 * sizeof(PackedHeader));
  l.prefix = take(2 * 4 * ((size_t)n + 1));
  l.list256 = take(sizeof(int4) * (size_t)l.max256);
  l.list128 = take(sizeof(int4) * (size_t)l.max128);
  l.total = o;
  return l;
}

// Row range of sequence s, (0, 0) and false if an offset is outside its range
// (decreasing, below 0, past the tokens).
__device__ __forceinline__ bool range_of(const int32_t* cu, int s, int tokens, int2& r) {
  const int a = cu[s], b = cu[s + 1];
  const bool ok = a >= 0 && b >= a && b <= tokens;
  r = ok ? make_int2(a, b - a) : make_int2(0, 0);
  return ok;
}

// Block x builds the list of R = 256 >> x query rows per entry.
__global__ void __launch_bounds__(NTH) packed_prepare_kernel(int n, int tokens, int causal,
                                                             const int32_t* cu, PackedHeader* hdr,
                                                             int32_t* prefix, int4* list256,
                                                             int4* list128, int* err) {
  __shared__ int warp_sum[32], warp_max[32];
  __shared__ int carry_s, top_s;
  __shared__ int bin[BINS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();  // the attention kernel may start up; it waits for this one's end
  const int R = blockIdx.x == 0 ? 256 : 128;
  int32_t* pre = prefix + (int64_t)blockIdx.x * (n + 1);
  int4* list = blockIdx.x == 0 ? list256 : list128;
  // inclusive sum over the block; returns the total in every thread
  auto scan = [&](int v, int& incl) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int w = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sum[lane] = w;
      if (lane == 31) carry_s = w;
    }
    __syncthreads();
    incl = x + (warp > 0 ? warp_sum[warp - 1] : 0);
    const int total = carry_s;
    __syncthreads();
    return total;
  };
  // the maximum of `before` and of v in the threads before this one
  auto max_before = [&](int v, int before) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = max(x, y);
    }
    if (lane == 31) warp_max[warp] = x;
    x = __shfl_up_sync(0xffffffffu, x, 1);
    int m = lane > 0 ? max(x, before) : before;
    __syncthreads();  // (warp_max is written again only behind scan()'s barriers)
    for (int w = 0; w < warp; ++w) m = max(m, warp_max[w]);
    return m;
  };
  bin[tid] = 0;
  if (tid == 0) top_s = 0;
  __syncthreads();
  int total = 0, longest = 0, reached = 0;
  bool bad = false;
  for (int base = 0; base < n; base += NTH) {
    const int s = base + tid;
    int v = 0, incl;
    int2 r = make_int2(0, 0);
    const bool ok = s >= n || range_of(cu, s, tokens, r);
    // Behind a bad sequence another may begin before the end of an earlier one and
    // share its rows: empty too, so that the lists and the work stay within those
    // of `tokens` rows.
    const bool bad_here = __syncthreads_or(!ok);
    bool take = true;
    if (bad || bad_here) {
      if (!bad && base > 0) reached = cu[base];  // (no offset before it was larger)
      bad = true;
      take = r.x >= max_before(r.x + r.y, reached);
      for (int w = 0; w < 32; ++w) reached = max(reached, warp_max[w]);
    }
    if (!ok || (!take && r.y > 0)) record_error(err, kErrIndex);
    if (take) {
      longest = max(longest, r.y);
      v = (r.y + R - 1) / R;
    }
    const int sum = scan(v, incl);
    if (s < n) pre[s] = total + incl - v;
    total += sum;
  }
  if (tid == 0) pre[n] = total;
  atomicMax(&top_s, longest);
  __syncthreads();
  // bins of equal cost (in 128-key tiles), or of 2^shift costs
  const int top = (top_s + 127) / 128;
  int shift = 0;
  while ((top >> shift) >= BINS) ++shift;
  auto entry = [&](int e, int4& w) {
    int lo = 0, hi = n - 1;  // the largest s with pre[s] <= e
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (pre[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    int2 r;
    range_of(cu, lo, tokens, r);
    const int q0 = (e - pre[lo]) * R;
    w = make_int4(r.x, r.y, q0, 0);
    const int seen = causal ? min(r.y, q0 + R) : r.y;
    return BINS - 1 - (((seen + 127) / 128) >> shift);  // bin 0 first
  };
  for (int e = tid; e < total; e += NTH) {
    int4 w;
    atomicAdd(&bin[entry(e, w)], 1);
  }
  __syncthreads();
  {
    int incl;
    const int v = bin[tid];
    scan(v, incl);
    bin[tid] = incl - v;
  }
  __syncthreads();
  for (int e = tid; e < total; e += NTH) {
    int4 w;
    const int b = entry(e, w);
    list[atomicAdd(&bin[b], 1)] = w;
  }
  if (tid == 0) hdr[blockIdx.x] = PackedHeader{total, {0, 0, 0}};
}

}  // namespace
}  // namespace mgb

using namespace mgb;

extern "C" {

size_t mgb_attention_packed_ws_bytes(int32_t n_seqs, int32_t tokens) {
  return n_seqs < 0 || tokens < 0 ? 0 : make_layout(n_seqs, tokens).total;
}

mgb_status mgb_attention_packed_prepare(int32_t n_seqs, int32_t tokens, int32_t causal,
                                        const int32_t* cu_seqlens, void* ws, size_t ws_bytes,
                                        mgb_attention_packed_plan* plan, void* stream) {
  if (fault_injected() || plan == nullptr) return MGB_ERR_INVALID_ARG;
  if (n_seqs < 0 || tokens < 0 || (causal & ~1) || ws == nullptr ||
      (n_seqs > 0 && cu_seqlens == nullptr))
    return MGB_ERR_INVALID_ARG;
  if (!is_aligned16(ws) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return MGB_ERR_MISALIGNED;
  const Layout l = make_layout(n_seqs, tokens);
  if (ws_bytes < l.total) return MGB_ERR_WORKSPACE_TOO_SMALL;
  const mgb_status s = check_arch();
  if (s != MGB_OK) return s;
  int* err = device_error_word();
  if (err == nullptr) return MGB_ERR_CUDA;
  if (n_seqs > 0 && tokens > 0) {
    char* b = static_cast<char*>(ws);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LaunchScope scope(PROF_ATTN_PACKED, st);
    packed_prepare_kernel<<<2, NTH, 0, st>>>(
        n_seqs, tokens, causal, cu_seqlens, reinterpret_cast<PackedHeader*>(b + l.header),
        reinterpret_cast<int32_t*>(b + l.prefix), reinterpret_cast<int4*>(b + l.list256),
        reinterpret_cast<int4*>(b + l.list128), err);
    if (cudaGetLastError() != cudaSuccess) return MGB_ERR_CUDA;
  }
  *plan = mgb_attention_packed_plan{n_seqs, tokens, causal, ws, ws_bytes};
  return MGB_OK;
}

mgb_status mgb_attention_packed_fwd(const mgb_attention_packed_plan* plan, int32_t n_q_heads,
                                    int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                    const void* q, const void* k, const void* v, int64_t ld_q,
                                    int64_t ld_kv, void* o, int64_t ld_o, float* lse, void* stream) {
  if (fault_injected() || plan == nullptr || plan->ws == nullptr) return MGB_ERR_INVALID_ARG;
  if (plan->n_seqs < 0 || plan->tokens < 0 || (plan->causal & ~1)) return MGB_ERR_INVALID_ARG;
  if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || n_q_heads > (1 << 20))
    return MGB_ERR_INVALID_ARG;
  if (dtype != MGB_BF16 && dtype != MGB_F32) return MGB_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MGB_ERR_UNSUPPORTED;
  const int64_t wq = (int64_t)n_q_heads * head_dim, wk = (int64_t)n_kv_heads * head_dim;
  if (ld_q < wq || ld_kv < wk || ld_o < wq) return MGB_ERR_INVALID_ARG;
  if (plan->tokens > 0 && (!q || !k || !v || !o)) return MGB_ERR_INVALID_ARG;
  const int vn = dtype == MGB_BF16 ? 8 : 4;
  if (!is_aligned16(q) || !is_aligned16(k) || !is_aligned16(v) || !is_aligned16(o) || ld_q % vn ||
      ld_kv % vn || ld_o % vn || !is_aligned16(plan->ws) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MGB_ERR_MISALIGNED;
  const Layout l = make_layout(plan->n_seqs, plan->tokens);
  if (plan->ws_bytes < l.total) return MGB_ERR_WORKSPACE_TOO_SMALL;
  // item numbers (entries x heads, up to four per entry) are 32-bit
  if (4 * l.max128 * n_q_heads >= (int64_t)1 << 30) return MGB_ERR_UNSUPPORTED;
  if (o != nullptr && (o == q || o == k || o == v)) return MGB_ERR_INVALID_ARG;
  const mgb_status s = check_arch();
  if (s != MGB_OK) return s;
  if (plan->n_seqs == 0 || plan->tokens == 0) return MGB_OK;
  const char* b = static_cast<const char*>(plan->ws);
  PackedArgs a{};
  a.tokens = plan->tokens; a.causal = plan->causal; a.nq = n_q_heads; a.nkv = n_kv_heads;
  a.d = head_dim;
  a.hdr256 = reinterpret_cast<const PackedHeader*>(b + l.header);
  a.hdr128 = a.hdr256 + 1;
  a.list256 = reinterpret_cast<const int4*>(b + l.list256);
  a.list128 = reinterpret_cast<const int4*>(b + l.list128);
  a.max256 = l.max256; a.max128 = l.max128;
  a.q = q; a.k = k; a.v = v; a.ld_q = ld_q; a.ld_kv = ld_kv; a.o = o; a.ld_o = ld_o; a.lse = lse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(PROF_ATTN_PACKED, st);
  return dtype == MGB_BF16 ? attention_packed_bf16(a, st) : attention_packed_f32(a, st);
}

}  // extern "C"
