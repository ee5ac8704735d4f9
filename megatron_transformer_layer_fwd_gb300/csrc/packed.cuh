// Shared by the packed-attention kernels: the work list in a plan's workspace
// and the arguments of one call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mgb {

// Work lists: one entry per 256 (128) query rows of a sequence, longest first:
// (sequence's first row, its length, first query row within it, 0).
struct PackedHeader {
  int32_t entries, pad[3];
};

struct PackedArgs {
  int tokens, causal, nq, nkv, d;
  const PackedHeader *hdr256, *hdr128;
  const int4 *list256, *list128;
  int64_t max256, max128;  // upper bounds of the entries (the counts are on the device)
  const void *q, *k, *v;
  int64_t ld_q, ld_kv;
  void* o;
  int64_t ld_o;
  float* lse;
};

mgb_status attention_packed_bf16(const PackedArgs& a, cudaStream_t st);
mgb_status attention_packed_f32(const PackedArgs& a, cudaStream_t st);

}  // namespace mgb
