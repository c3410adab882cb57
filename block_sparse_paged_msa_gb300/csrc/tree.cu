// msa_tree_plan and msa_tree_commit: the ends of a step that verifies a tree of
// drafted tokens -- what each node sees and where it stands, and the accepted
// nodes' cache rows moved together.
//
// The pages verify chains only (vLLM MiniMaxM3SparseMSAMetadataBuilder.build:
// decode_query_len); a tree is this library's extension of that step.
#include <algorithm>

#include "tree.cuh"

namespace msa {
namespace {

// ---------------------------------------------------------------- the plan
// One block per request, a thread per node.  A node's mask is its own bit and
// its parent's mask; with m_i the ancestors within 2^k steps and p_i the node
// 2^k steps up, m_i |= m_{p_i}, p_i = p_{p_i} doubles the reach: six rounds for
// 64 nodes.  The depth is the mask's population less one.
// Latency alone bounds it: 2 to 4 us for one request or 64.
__global__ void __launch_bounds__(kTreeNodes)
tree_plan_kernel(WsView ws, const int32_t* __restrict__ parents, int64_t* __restrict__ masks,
                 int64_t* __restrict__ positions) {
  __shared__ uint64_t m[2][kTreeNodes];
  __shared__ int up[2][kTreeNodes];
  const int i = threadIdx.x, r = blockIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  // tokens of no request that has a tree
  const int T = ws.hdr->num_tokens;
  for (int t = r * kTreeNodes + i; t < T; t += gridDim.x * kTreeNodes) {
    const int q = ws.tok_req[t];
    if (q >= 0 && tree_of(ws, q).n > 0) continue;
    masks[t] = 0;
    if (positions) positions[t] = -1;
  }
  if (r >= ws.hdr->batch) return;
  const Tree tr = tree_of(ws, r);
  if (tr.too_large && i == 0) set_error(ws.hdr, MSA_DEVERR_TREE);
  if (tr.n == 0) return;                       // (the whole block)
  int p = i < tr.n ? parents[tr.t0 + i] : -1;
  if (p < -1 || p >= i) {
    if (i < tr.n) set_error(ws.hdr, MSA_DEVERR_TREE);
    p = -1;
  }
  m[0][i] = (uint64_t)1 << i;
  up[0][i] = p;
#pragma unroll
  for (int k = 0; k < 6; ++k) {
    __syncthreads();
    const int a = k & 1, b = a ^ 1, q = up[a][i];
    m[b][i] = m[a][i] | (q >= 0 ? m[a][q] : 0);
    up[b][i] = q >= 0 ? up[a][q] : -1;
  }
  if (i >= tr.n) return;
  const uint64_t mask = m[0][i];
  masks[tr.t0 + i] = (int64_t)mask;
  if (positions) positions[tr.t0 + i] = (int64_t)tr.base + __popcll(mask) - 1;
}

// -------------------------------------------------------------- the commit
// A block per (request, some (layer, pool) pairs): it lists the request's moves
// (rows whose position changes) in shared memory, then every thread carries one
// column of bytes of one head through them, kDeep rows at a time.  accepted
// ascends, so the row j is read from is never below j: a thread that loads a
// batch of rows before it stores them, batch after batch, never reads a row that
// it has overwritten, and no other thread touches its column.
//
// What bounds it is the chain of dependent loads ahead of a block's rows (header,
// tree, path, block table: some 2 us) and, for many requests, the rows' traffic in
// sectors of 32 bytes.  So the grid is bounded (2432 blocks, of which 912 are resident: 78
// registers let six stand on an SM), and a block walks the chain once and then takes one
// pool after the other.
// 64 requests of 16 nodes, 32 layers of three bf16 pools: 21 us with cold caches, 51 MB
// read and as many written (a block per pool, 96 a request, each with its own walk of
// the chain: 26 us); one request, 4 NVFP4 layers: 4.4 us.
constexpr int kMoveThreads = 128, kDeep = 8, kMovePools = 192, kDistinctLayers = 1024;
constexpr int kMoveBlocks = 16 * 152;          // of a grid, about

struct Move {
  int32_t src_page, src_row, dst_page, dst_row;
};
struct MoveArgs {
  void* pool[kMovePools];
  uint8_t kind[kMovePools];                    // K, V, index K, index V
  int32_t pools, heads, max_blocks;            // pools: of the array
  int32_t bytes[4];                            // of a row of each kind
  int32_t slots[4], first[4];                  // slots of a page and head, the kind's own
};

template <typename V>
__device__ __forceinline__ void move_rows(uint8_t* pool, const Move* mv, int n, int heads,
                                          int slots, int first, int bytes) {
  const int cols = bytes / (int)sizeof(V);
  for (int x = threadIdx.x; x < heads * cols; x += kMoveThreads) {
    const int h = x / cols, c = x - h * cols;
    auto at = [&](int page, int row) {
      return reinterpret_cast<V*>(
                 pool + (((int64_t)page * heads + h) * slots + first) * kBlock * bytes +
                 (int64_t)row * bytes) + c;
    };
    for (int j0 = 0; j0 < n; j0 += kDeep) {
      V v[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (j0 + k < n) v[k] = *at(mv[j0 + k].src_page, mv[j0 + k].src_row);
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (j0 + k < n) *at(mv[j0 + k].dst_page, mv[j0 + k].dst_row) = v[k];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads)
tree_commit_kernel(WsView ws, const __grid_constant__ MoveArgs a,
                   const int32_t* __restrict__ accepted, const int32_t* __restrict__ num) {
  __shared__ Move mv[kTreeNodes];
  __shared__ int moves, bad;
  const int tid = threadIdx.x, lane = tid & 31, r = blockIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  if (r >= ws.hdr->batch) return;
  const Tree tr = tree_of(ws, r);
  if (tr.n == 0) return;
  const int k = num[r];
  if (tid == 0) bad = k < 0 || k > tr.n;
  __syncthreads();
  int node = 0;
  if (tid < kTreeNodes && !bad && tid < k) {
    node = accepted[(int64_t)r * kTreeNodes + tid];
    const int before = tid > 0 ? accepted[(int64_t)r * kTreeNodes + tid - 1] : -1;
    if (node <= before || node >= tr.n) atomicOr(&bad, 1);
  }
  __syncthreads();
  if (bad) {
    if (tid == 0 && blockIdx.y == 0) set_error(ws.hdr, MSA_DEVERR_TREE);
    return;
  }
  if (tid < 32) {                              // the first warp lists the moves, in order
    int n = 0;
    for (int j0 = 0; j0 < k; j0 += 32) {
      const int j = j0 + lane;
      Move w = {-1, 0, -1, 0};
      const int from = j < k ? accepted[(int64_t)r * kTreeNodes + j] : j;
      if (j < k && from != j) {
        const int s = tr.base + from, d = tr.base + j;
        w.src_page = ws.block_table[(int64_t)r * a.max_blocks + s / kBlock];
        w.dst_page = ws.block_table[(int64_t)r * a.max_blocks + d / kBlock];
        w.src_row = s % kBlock;
        w.dst_row = d % kBlock;
      }
      const bool on = w.src_page >= 0 && w.dst_page >= 0;
      const unsigned m = __ballot_sync(0xffffffffu, on);
      if (on) mv[n + __popc(m & ((1u << lane) - 1u))] = w;
      n += __popc(m);
    }
    if (lane == 0) moves = n;
  }
  __syncthreads();
  const int n = moves;
  for (int p = blockIdx.y; n > 0 && p < a.pools; p += gridDim.y) {
    uint8_t* pool = static_cast<uint8_t*>(a.pool[p]);
    const int kind = a.kind[p], bytes = a.bytes[kind];
    if (bytes % 16 == 0)
      move_rows<uint4>(pool, mv, n, a.heads, a.slots[kind], a.first[kind], bytes);
    else                                       // NVFP4: 72 bytes
      move_rows<uint2>(pool, mv, n, a.heads, a.slots[kind], a.first[kind], bytes);
  }
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_tree_plan(const msa_config* cfg, void* ws, const int32_t* parents,
                                    int64_t* tree_mask, int64_t* positions, msa_stream_t stream) {
  const msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (!ws || ((uintptr_t)ws & 255) != 0) return MSA_ERR_INVALID_ARG;
  if (max_tokens_of(*cfg) <= 0 || cfg->max_batch == 0) return MSA_OK;
  if (!parents || !tree_mask || ((uintptr_t)parents & 3) != 0 ||
      ((uintptr_t)tree_mask & 7) != 0 || ((uintptr_t)positions & 7) != 0)
    return MSA_ERR_INVALID_ARG;
  return launch_pdl(tree_plan_kernel, dim3(cfg->max_batch), dim3(kTreeNodes), 0,
                    (cudaStream_t)stream, view_of(*cfg, ws), parents, tree_mask, positions);
}

extern "C" msa_status msa_tree_commit(const msa_config* cfg, void* ws, const int32_t* accepted,
                                      const int32_t* num_accepted, int32_t num_layers,
                                      void* const* k_pages, void* const* v_pages,
                                      void* const* idx_k_pages, void* const* idx_v_pages,
                                      msa_stream_t stream) {
  const msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (!ws || ((uintptr_t)ws & 255) != 0 || num_layers < 0) return MSA_ERR_INVALID_ARG;
  if (max_tokens_of(*cfg) <= 0 || cfg->max_batch == 0 || num_layers == 0) return MSA_OK;
  if (!accepted || !num_accepted || !k_pages || !v_pages || ((uintptr_t)accepted & 3) != 0 ||
      ((uintptr_t)num_accepted & 3) != 0)
    return MSA_ERR_INVALID_ARG;
  void* const* kinds[4] = {k_pages, v_pages, idx_k_pages, idx_v_pages};
  for (int32_t l = 0; l < num_layers; ++l)
    for (int k = 0; k < 4; ++k)
      if (kinds[k] && (!kinds[k][l] || !aligned16(kinds[k][l]))) return MSA_ERR_INVALID_ARG;
  // a pool that stood twice in the lists would be moved by two blocks at once; an
  // NVFP4 pool is its layer's K and its V
  if (num_layers > kDistinctLayers) return MSA_ERR_UNSUPPORTED;
  const bool fp4 = cfg->kv_dtype == MSA_KV_NVFP4;
  uintptr_t sorted[4 * kDistinctLayers];
  int all = 0;
  for (int k = 0; k < 4; ++k)
    for (int32_t l = 0; kinds[k] && l < num_layers; ++l)
      sorted[all++] = (uintptr_t)kinds[k][l] | (fp4 && k == 1 ? 1 : 0);
  std::sort(sorted, sorted + all);
  if (std::adjacent_find(sorted, sorted + all) != sorted + all) return MSA_ERR_INVALID_ARG;
  MoveArgs a;
  const int32_t row = fp4 ? kFp4Row : (cfg->kv_dtype == MSA_KV_BF16 ? 2 * kHeadDim : kHeadDim);
  a.heads = cfg->num_kv_heads;
  a.max_blocks = cfg->max_blocks_per_req;
  for (int k = 0; k < 4; ++k) {
    a.bytes[k] = k < 2 ? row : 2 * cfg->index_dim;
    a.slots[k] = k < 2 && fp4 ? 2 : 1;
    a.first[k] = k == 1 && fp4 ? 1 : 0;
  }
  a.pools = 0;
  for (int32_t l = 0; l < num_layers; ++l) {
    for (int k = 0; k < 4; ++k) {
      if (!kinds[k]) continue;
      a.pool[a.pools] = kinds[k][l];
      a.kind[a.pools++] = (uint8_t)k;
    }
    if (a.pools <= kMovePools - 4 && l + 1 < num_layers) continue;
    const int share = (kMoveBlocks + cfg->max_batch - 1) / cfg->max_batch;
    const msa_status s2 = launch_pdl(
        tree_commit_kernel, dim3(cfg->max_batch, a.pools < share ? a.pools : share),
        dim3(kMoveThreads), 0, (cudaStream_t)stream, view_of(*cfg, ws), a, accepted, num_accepted);
    if (s2 != MSA_OK) return s2;
    a.pools = 0;
  }
  return MSA_OK;
}
