// Attention of small drafts over a paged cache: items of up to 16 rows (drafted tokens times the
// query heads of a KV head) for the kernel of the decode step, in bf16 on mma.sync, in float32 on
// the CUDA cores. Its many small CTAs and warps with rings of their own stream through the
// caches of many short sequences without waiting for one another, where the 128 rows of a
// tcgen05 tile would stand empty. 96 sequences of 20 to 1200 tokens, 16 heads of 64, 1 to 8 rows
// 32 us, 4.1 TB/s; 64 of 2000 tokens, 8 KV heads of 128, 8 rows 86.6 us, 6.1 TB/s.
#include "paged_rows.cuh"

namespace mgb {

namespace {

template <typename T, int D, int NR>
mgb_status launch(const Params& p, cudaStream_t st) {
  using C = Cfg<T, D, NR>;
  auto k = paged_rows_kernel<T, D, NR, true>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return MGB_ERR_CUDA;
  return launch_pdl(k, SMS * ctas_per_sm(D), NT, C::SMEM, st, p);
}

// A part holds a multiple of TREE_ROW_STEP rows, up to MAXR: these are all forms that a plan asks for.
template <typename T, int D>
mgb_status launch_rows(const Params& p, cudaStream_t st) {
  static_assert(TREE_ROW_STEP == 8 && MAXR == 2 * TREE_ROW_STEP, "a form for each number of rows");
  return p.rows == TREE_ROW_STEP ? launch<T, D, TREE_ROW_STEP>(p, st) : launch<T, D, MAXR>(p, st);
}

}  // namespace

mgb_status attention_tree_rows(const TreeParams& t, int d, int dtype, cudaStream_t st) {
  Params p{};
  p.nkv = t.nkv; p.rows = t.rows; p.G = t.G; p.nq = t.nq;
  p.thdr = t.hdr; p.tstart = t.start; p.live = t.live; p.mask = t.mask;
  p.counter = t.counter; p.ml = t.ml; p.part = t.part;
  p.k = t.k; p.v = t.v; p.table = t.table;
  p.s_page = t.s_page; p.s_tok = t.s_tok; p.s_head = t.s_head; p.ld_table = t.ld_table;
  p.n_pages = t.n_pages; p.page_size = t.page_size; p.cap = t.cap;
  p.q = t.q; p.ld_q = t.ld_q; p.o = t.o; p.ld_o = t.ld_o; p.lse = t.lse;
  p.sl2 = t.sl2; p.err = t.err;
  if (dtype == MGB_BF16) return d == 64 ? launch_rows<bf16, 64>(p, st) : launch_rows<bf16, 128>(p, st);
  return d == 64 ? launch_rows<float, 64>(p, st) : launch_rows<float, 128>(p, st);
}

}  // namespace mgb
