// Draft trees: a request's nodes as the plan has them.  Not part of the ABI.
#pragma once

#include "msa_internal.cuh"

namespace msa {

constexpr int kTreeNodes = MSA_MAX_TREE_NODES;

struct Tree {
  int t0, n, base;             // first token, nodes (0 = no tree), cached tokens before them
  bool too_large;              // more nodes than a mask has bits
};

// The tree of request r < batch; none for idle and flagged requests.
__device__ __forceinline__ Tree tree_of(const WsView& ws, int r) {
  Tree t;
  const int L = ws.req_seq_len[r];
  t.t0 = ws.req_qstart[r];
  t.n = L > 0 ? ws.req_qstart[r + 1] - t.t0 : 0;
  t.too_large = t.n > kTreeNodes;
  if (t.too_large) t.n = 0;
  t.base = L - t.n;
  return t;
}

// NVFP4 pools: trees of up to that many query rows (nodes x group) a KV head go
// through the dense decode's kernel (dense_decode.cu).
constexpr int kTreeDenseRows = 64;
size_t tree_dense_scratch(const msa_config& c);
msa_status tree_dense_attention(const msa_config& c, const WsView& v, const void* q,
                                const void* k_pages, const void* v_pages, const int64_t* mask,
                                void* scratch, void* out, float* lse, cudaStream_t s);

}  // namespace msa
