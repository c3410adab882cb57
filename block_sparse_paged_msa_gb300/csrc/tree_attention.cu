// msa_tree_attention: full-context attention of the nodes of a draft tree over a
// paged cache of bf16, e4m3 or NVFP4 rows (with a chain's masks: the dense decode
// and verify of any KV type).
//
// Mathematics.  For node i and query head q of KV head h's group, over the keys u
// that the node sees (the cached prefix, and the nodes of its mask):
//     s_u = scale q . k_u,   out = sum_u 2^(s'_u - m) v_u / sum_u 2^(s'_u - m),
// s' = s log2 e, in one pass with a running maximum m and sum.  Scores are bf16
// products (bf16 pools) or fp16 ones (codes and their block scales are exact fp16
// operands, and so are queries of 2^-14 .. 65504; larger ones are flagged, smaller
// ones keep the bits of fp16's subnormals), accumulated in fp32.  Values enter P V
// as fp16: exact for e4m3 and NVFP4, for bf16 within 2^-14 .. 65504 (as in the
// prefill tiles; larger ones are flagged).  The probabilities are rounded to fp16
// (2^-11 relative, below the bf16 rounding of the output), carried as 2^(s' - m +
// 7) so that fp16's normal range reaches 2^-21 below the maximum; their sum is
// taken before that rounding.  m is an unscaled score, and the scale is applied to
// the difference, which is exact near the maximum whatever the scores' size.  m
// moves only when a score is 2^8 above it in the exponent.
//
// Work split.  A request's query rows of a KV head (nodes x group, node by node)
// are M tiles of 128, taken two at a time; a unit of work is one 128-key page of
// one (request, head, pair of tiles).  The units of the step, in order, are cut
// into contiguous ranges of equal weight, one per CTA (one per SM), whatever the
// lengths and trees are; a group that lies in several ranges leaves one fp32
// partial per CTA in the scratch, which a second kernel merges in CTA order.
//
// A CTA: a loader warp (pages by TMA into a ring), four converter warps (Q rows,
// and the pages' rows as MMA operands), an MMA warp and eight softmax warps.  An
// item is one (page, tile): S = Q K^T (128 rows x 128 keys) into one of two TMEM
// buffers, the two softmax warpgroups take half a row a thread (TMEM lane = query
// row), write P over their half of S, and O += P V with P as the A operand from
// TMEM.  S of the next item is computed during the softmax of this one.  The two
// threads of a row agree on m through one barrier with a vote.
#include <atomic>
#include <cfloat>
#include <cstring>

#include "tcgen05.cuh"
#include "tree.cuh"

namespace msa {
namespace {

constexpr int kTile = 128;                     // query rows of an M tile
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kPairRows = 2 * kTile;
constexpr int kMaxCtas = 320;
constexpr float kBias = 7.f;                   // exponent offset of the probabilities
constexpr float kSlack = 8.f;                  // 2^(kBias + kSlack) is below fp16's largest

constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kConvWarp = kSoftWarps, kLoadWarp = kConvWarp + kConvWarps, kMmaWarp = kLoadWarp + 1,
              kIdleWarp = kMmaWarp + 1, kThreads = 512;
// threads x launch registers = 512 x 128 = 256 x 176 + 128 x 104 + 128 x 56
constexpr int kSoftRegs = 176, kConvRegs = 104, kMiscRegs = 56;

struct TreeArgs {
  int Hkv, Hq, G, max_blocks, rows;            // rows: of a partial
  uint32_t g_magic;                            // row / G = row * g_magic >> 20
  float scale_log2, v_scale, slack;            // slack: kSlack in unscaled scores
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  const int64_t* mask;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;                               // [2 * CTAs][rows][128]
  float2* ml_part;                             // [2 * CTAs][rows] (m, sum)
  int4* split;                                 // [CTAs] the split group that starts in the CTA's
                                               // range: (partials, first token, head, pair << 16
                                               // | rows); 0 partials = none

  __device__ __forceinline__ int node_of(int n) const { return (int)(n * g_magic >> 20); }
  // query row n of head h of a request whose tokens start at t0, as a row of q and out
  __device__ __forceinline__ int64_t q_row(int t0, int h, int n) const {
    const int i = node_of(n);
    return (int64_t)(t0 + i) * Hq + h * G + n - i * G;
  }
};

// KV types: tiles of the operand ring, raw stages in front of the converters.
template <int KV>
struct Form {
  static constexpr bool kRaw = KV != MSA_KV_BF16;
  static constexpr int kTiles = kRaw ? 3 : 5;
  static constexpr int kStages = KV == MSA_KV_FP8_E4M3 ? 4 : (KV == MSA_KV_NVFP4 ? 7 : 1);
  static constexpr int kStageBytes =
      KV == MSA_KV_FP8_E4M3 ? kBlock * kHeadDim : (KV == MSA_KV_NVFP4 ? kBlock * kFp4Row : 0);
  static constexpr int kSmem = (2 + kTiles) * kTileBytes + (kRaw ? kStages * kStageBytes : 0);
  // weight of a page for a pair of two tiles and of one
  static constexpr int kW2 = 1, kW1 = 1;
};

// What the roles share.
template <int KV>
struct Shared {
  using F = Form<KV>;
  uint64_t raw_full[F::kStages], raw_empty[F::kStages];
  uint64_t full[F::kTiles], ready[F::kTiles], empty[F::kTiles];
  uint64_t q_full[2], q_free[2];
  uint64_t s_ready[2], p_ready[2], o_done[2];
  uint64_t fin;
  unsigned long long bad[8];                   // by segment: nodes with values that are not finite
  float red[2][kTile];
  uint32_t tmem_base;
  // the CTA's range
  int r0;                                      // first request, and the weight before it
  uint32_t w0, from, to, total, ranges;
  uint32_t part[kThreads / 32];
};

// Weights.  A request: heads x pairs of tiles x pages.
struct Req {
  int n, t0, base, L, nb, rows, pairs;
  uint32_t pw, weight;                         // of a page over all pairs; of the request
};
template <int KV>
__device__ __forceinline__ Req request(const WsView& ws, const TreeArgs& a, int r) {
  using F = Form<KV>;
  const Tree t = tree_of(ws, r);
  Req q;
  q.n = t.n;
  q.t0 = t.t0;
  q.base = t.base;
  q.L = t.base + t.n;
  q.nb = t.n > 0 ? (q.L + kBlock - 1) / kBlock : 0;
  q.rows = t.n * a.G;
  const int tiles = (q.rows + kTile - 1) / kTile;
  q.pairs = (tiles + 1) / 2;
  q.pw = (uint32_t)(tiles / 2 * F::kW2 + (tiles & 1) * F::kW1);
  q.weight = q.pw * (uint32_t)q.nb * (uint32_t)a.Hkv;
  return q;
}

// The weight ranges: `ranges` of them, [total c / ranges, total (c + 1) / ranges).
__device__ __forceinline__ uint32_t range_start(uint32_t total, uint32_t ranges, uint32_t c) {
  return (uint32_t)((uint64_t)total * c / ranges);
}
__device__ __forceinline__ uint32_t range_of(uint32_t total, uint32_t ranges, uint32_t w) {
  return (uint32_t)((((uint64_t)w + 1) * ranges - 1) / total);
}

// A role's walk over its CTA's range: one segment per (request, head, pair).  A
// page belongs to the range in which its weight starts.
template <int KV>
struct Walk {
  using F = Form<KV>;
  int r;
  uint32_t wr, w, end;                         // weight before request r; of the next page; end
  Req q;
  // the segment
  int h, pair, j0, j1, tiles, rows;
  uint32_t last;                               // weight of its group's last page
  bool starts, whole;

  __device__ __forceinline__ void open(const WsView& ws, const TreeArgs& a, const Shared<KV>& sh) {
    r = sh.r0;
    wr = sh.w0;
    w = sh.from;
    end = sh.to;
    if (w < end) q = request<KV>(ws, a, r);
  }
  __device__ __forceinline__ bool next(const WsView& ws, const TreeArgs& a) {
    for (;;) {
      if (w >= end) return false;
      while (w >= wr + q.weight) {             // w < end <= the total: there is a next request
        wr += q.weight;
        q = request<KV>(ws, a, ++r);
      }
      const uint32_t hw = q.pw * (uint32_t)q.nb;                 // of a head
      const uint32_t x = w - wr;
      h = (int)(x / hw);
      const uint32_t y = x - h * hw, gw = (uint32_t)(F::kW2 * q.nb);
      pair = min((int)(y / gw), q.pairs - 1);
      rows = min(kPairRows, q.rows - pair * kPairRows);
      tiles = rows > kTile ? 2 : 1;
      const uint32_t step = tiles == 2 ? F::kW2 : F::kW1;
      const uint32_t g0 = wr + h * hw + pair * gw;               // weight before the group
      j0 = (int)((w - g0 + step - 1) / step);
      j1 = (int)min((uint32_t)q.nb, (end - g0 + step - 1) / step);
      last = g0 + (q.nb - 1) * step;
      w = g0 + q.nb * step;                    // the next group's start
      if (w > end) w = end;
      starts = j0 == 0;
      whole = starts && j1 == q.nb;
      if (j0 < j1) return true;
    }
  }
};

// ---------------------------------------------------------------- small helpers
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(p));
  return p != 0;
}
// Barrier over `count` threads that also tells whether any of them said so.
__device__ __forceinline__ bool named_bar_any(int id, int count, bool mine) {
  int any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n"
      " selp.b32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(id), "r"(count), "r"((int)mine)
      : "memory");
  return any != 0;
}

// ---------------------------------------------------------------- conversion
// Sixteen-bit pairs with an all-ones exponent -> 0; true if there was one.
__device__ __forceinline__ bool clear_non_finite(uint32_t (&h)[4]) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((h[i] & 0x7c00u) == 0x7c00u) { h[i] &= 0xffff0000u; any = true; }
    if ((h[i] & 0x7c000000u) == 0x7c000000u) { h[i] &= 0xffffu; any = true; }
  }
  return any;
}
__device__ __forceinline__ bool any_inf(const uint32_t (&h)[4]) {
  return f16x2_has_inf(h[0]) | f16x2_has_inf(h[1]) | f16x2_has_inf(h[2]) | f16x2_has_inf(h[3]);
}
__device__ __forceinline__ void to_f16(const uint4& x, uint32_t (&h)[4]) {
  h[0] = bf16x2_to_f16x2(x.x);
  h[1] = bf16x2_to_f16x2(x.y);
  h[2] = bf16x2_to_f16x2(x.z);
  h[3] = bf16x2_to_f16x2(x.w);
}

// One page's K or V slot -> the operand tile at `tile` (K-major rows, 128-byte
// swizzle), by 128 threads.  kValues: rows from `ntok` on become 0; of rows from
// `all` on (which not every query row sees: 0 * NaN is not 0) elements that are
// not finite become 0 and are noted in `bad` by node.  A bf16 tile is converted in
// place.  Returns whether a value left the fp16 range.
template <int KV, bool kValues>
__device__ __forceinline__ bool convert_page(const uint8_t* raw, uint8_t* tile, int tid, int ntok,
                                             int all, unsigned long long* bad) {
  bool ovf = false;
  auto special = [&](int key, uint32_t (&h)[4]) {
    if (key >= ntok) {
      h[0] = h[1] = h[2] = h[3] = 0u;
    } else {
      if (KV == MSA_KV_BF16) ovf |= any_inf(h);
      if (key >= all && clear_non_finite(h)) atomicOr(bad, 1ull << (key - all));
    }
  };
  if constexpr (KV == MSA_KV_BF16) {
    // a 16-byte chunk lies in one key row, 128 bytes per row and 64-dim half
    if (all >= kBlock) {
      uint32_t top = 0u;                       // largest magnitudes
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int off = (tid + 128 * i) * 16;
        uint32_t h[4];
        to_f16(*reinterpret_cast<const uint4*>(tile + off), h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t m = h[e] & 0x7fff7fffu;
          const __half2 x = __hmax2(*reinterpret_cast<const __half2*>(&top),
                                    *reinterpret_cast<const __half2*>(&m));
          top = *reinterpret_cast<const uint32_t*>(&x);
        }
        *reinterpret_cast<uint4*>(tile + off) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      ovf = f16x2_has_inf(top);
    } else {
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int off = (tid + 128 * i) * 16;
        uint32_t h[4];
        to_f16(*reinterpret_cast<const uint4*>(tile + off), h);
        special((off & (kTileBytes / 2 - 1)) >> 7, h);
        *reinterpret_cast<uint4*>(tile + off) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  } else if constexpr (KV == MSA_KV_FP8_E4M3) {
    // eight lanes take one 16-byte chunk of eight rows: the swizzles of the raw
    // tile and of the operand spread them over all banks
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int x = tid + 128 * i, key = (x & 7) | ((x >> 6) << 3), c = (x >> 3) & 7;
      const uint4 w = *reinterpret_cast<const uint4*>(raw + key * 128 + ((c ^ (key & 7)) << 4));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          h[2 * e] = e4m3x2_to_f16x2((uint16_t)u[2 * k + e]);
          h[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(u[2 * k + e] >> 16));
        }
        if (kValues && all < kBlock) special(key, h);
        *reinterpret_cast<uint4*>(tile + swz_tma(key, 2 * c + k)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  } else {
    // sixteen lanes take one block of sixteen rows: 72-byte rows spread over all
    // banks, and so does the operand's swizzle
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int x = tid + 128 * i, key = (x & 15) | ((x >> 7) << 4), b = (x >> 4) & 7;
      const uint8_t* row = raw + key * kFp4Row;
      const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * b);
      const uint32_t s = e4m3_scale_f16x2(row[kHeadDim / 2 + b]);
      uint32_t h[2][4];
      e2m1x8_to_f16x2(w.x, h[0]);
      e2m1x8_to_f16x2(w.y, h[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[k][e] = hmul2_u32(h[k][e], s);
        if (kValues && all < kBlock) special(key, h[k]);
        *reinterpret_cast<uint4*>(tile + swz_tma(key, 2 * b + k)) =
            make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
      }
    }
  }
  return ovf;
}

// Dim d of value row `row` of a page as the converters see it (fp16 range), for
// the few rows whose values are not finite.
template <int KV>
__device__ __forceinline__ float value_of(const uint8_t* v_pool, int64_t page, int Hkv, int h, int row,
                                       int d) {
  if (KV == MSA_KV_BF16) {
    const uint16_t x = reinterpret_cast<const uint16_t*>(
        v_pool)[((page * Hkv + h) * kBlock + row) * kHeadDim + d];
    return __half2float(__float2half_rn(__uint_as_float((uint32_t)x << 16)));
  }
  uint32_t u;
  if (KV == MSA_KV_FP8_E4M3) {
    u = e4m3x2_to_f16x2(v_pool[((page * Hkv + h) * kBlock + row) * kHeadDim + d]);
  } else {
    const uint8_t* at = v_pool + (((page * Hkv + h) * 2 + 1) * kBlock + row) * kFp4Row;
    uint32_t c[4];
    e2m1x8_to_f16x2((uint32_t)(at[d / 2] >> (4 * (d & 1))) & 15u, c);
    u = hmul2_u32(c[0], e4m3_scale_f16x2(at[kHeadDim / 2 + d / 16]));
  }
  return __half2float(__ushort_as_half((unsigned short)(u & 0xffffu)));
}

// ---------------------------------------------------------------- the kernel
template <int KV>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_kernel(WsView ws, TreeArgs a, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v) {
  using F = Form<KV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) Shared<KV> sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);         // uniform
  uint8_t* qbuf = smem;                        // two tiles
  uint8_t* tiles = smem + 2 * kTileBytes;
  uint8_t* raw = tiles + F::kTiles * kTileBytes;
  if (tid == 0) {
    for (int i = 0; i < F::kStages; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kConvWarps);
    }
    for (int i = 0; i < F::kTiles; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.ready[i], kConvWarps);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], kConvWarps);
      mbar_init(&sh.q_free[i], 1);
      mbar_init(&sh.s_ready[i], 1);
      mbar_init(&sh.p_ready[i], kSoftWarps);
      mbar_init(&sh.o_done[i], 1);
    }
    mbar_init(&sh.fin, 1);
    for (int i = 0; i < 8; ++i) sh.bad[i] = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    // before the wait: kernels of this library that use TMEM let their
    // dependents start only once they hold theirs
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's range: the weights of all requests, scanned by the block
  {
    const int batch = ws.hdr->batch;
    auto block_scan = [&](uint32_t x, uint32_t& sum) {           // exclusive
      uint32_t inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) sh.part[warp] = inc;
      __syncthreads();
      uint32_t before = 0, all = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += sh.part[i];
        all += sh.part[i];
      }
      sum = all;
      return before + inc - x;
    };
    uint32_t total = 0, mine = 0, before = 0, sum;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
      mine = b0 + tid < batch ? request<KV>(ws, a, b0 + tid).weight : 0;
      before = block_scan(mine, sum);
      total += sum;
    }
    const uint32_t most = F::kW2 > F::kW1 ? F::kW2 : F::kW1;
    const uint32_t ranges = min((uint32_t)gridDim.x, total / most);
    const bool any = blockIdx.x < ranges;
    const uint32_t from = any ? range_start(total, ranges, blockIdx.x) : 0;
    if (tid == 0) {
      sh.r0 = 0;
      sh.w0 = 0;
      sh.from = from;
      sh.to = any ? range_start(total, ranges, blockIdx.x + 1) : 0;
      sh.total = total;
      sh.ranges = ranges;
    }
    __syncthreads();
    if (any) {
      uint32_t base = 0;
      for (int b0 = 0; b0 < batch; b0 += kThreads) {
        if (batch > kThreads) {
          mine = b0 + tid < batch ? request<KV>(ws, a, b0 + tid).weight : 0;
          before = block_scan(mine, sum);
        }
        if (from >= base + before && from < base + before + mine) {
          sh.r0 = b0 + tid;
          sh.w0 = base + before;
        }
        if (batch > kThreads) base += sum;
      }
    }
    __syncthreads();
  }
  const uint32_t tmem = sh.tmem_base;

  if (warp >= kLoadWarp) {
    regs_down<kMiscRegs>();
  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loader
    // The pages of a segment 32 at a time (a lane each).
    Walk<KV> wk;
    wk.open(ws, a, sh);
    int arms = 0, at = 0;
    uint32_t phase = 0;
    constexpr int kSlots = F::kRaw ? F::kStages : F::kTiles;
    while (wk.next(ws, a)) {
      int mine = -1;
      for (int j = wk.j0; j < wk.j1; ++j) {
        const int k = (j - wk.j0) & 31;
        if (k == 0)
          mine = j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + j + lane] : -1;
        const int page = __shfl_sync(0xffffffffu, mine, k);
        for (int kind = 0; kind < 2; ++kind) {
          uint64_t* full = F::kRaw ? &sh.raw_full[at] : &sh.full[at];
          mbar_wait(F::kRaw ? &sh.raw_empty[at] : &sh.empty[at], phase ^ 1u, ws.hdr);
          __syncwarp();
          if (elect_one()) {
            if (page < 0) {
              mbar_arrive(full);
            } else if constexpr (KV == MSA_KV_NVFP4) {
              const int64_t slot = ((int64_t)page * a.Hkv + wk.h) * 2 + kind;
              const int rows = min(kBlock, wk.q.L - j * kBlock);
              const uint32_t bytes = (uint32_t)((rows + 1) & ~1) * kFp4Row;   // a multiple of 16
              mbar_arrive_expect_tx(full, bytes);
              bulk_load(raw + at * F::kStageBytes,
                        (kind ? a.v_pool : a.k_pool) + slot * (kBlock * kFp4Row), bytes, full);
            } else {
              const int y = (page * a.Hkv + wk.h) * kBlock;
              const void* map = kind ? (const void*)&tmap_v : (const void*)&tmap_k;
              if constexpr (KV == MSA_KV_FP8_E4M3) {
                mbar_arrive_expect_tx(full, F::kStageBytes);
                tma_load_2d(raw + at * F::kStageBytes, map, 0, y, full);
              } else {
                mbar_arrive_expect_tx(full, kTileBytes);
                tma_load_2d(tiles + at * kTileBytes, map, 0, y, full);
                tma_load_2d(tiles + at * kTileBytes + kTileBytes / 2, map, 64, y, full);
              }
            }
          }
          __syncwarp();
          ++arms;
          if (++at == kSlots) { at = 0; phase ^= 1u; }
        }
      }
    }
    // Normally the converters and the MMAs wait for every copy issued here.
    // After a wait gave up they may not have: let the copies in flight land.
    if (lane == 0 && (*reinterpret_cast<volatile int*>(&ws.hdr->err) & MSA_DEVERR_TIMEOUT))
      for (int i = 0; i < kSlots && i < arms; ++i)
        mbar_drain(F::kRaw ? &sh.raw_full[i] : &sh.full[i],
                   (uint32_t)(((arms - 1 - i) / kSlots) & 1));
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs
    // Item by item, S one ahead: S_{k+1} once P_{k-1} V has read the buffer it
    // overwrites, then O += P_k V.
    struct Cursor {                            // over (page, tile) items
      Walk<KV> wk;
      int j, t, k, kv;                         // k: item number; kv: pages before this one
      int qsel, qb;                            // buffer of the segment's first Q tile
      bool more, first;                        // first: page of the segment
    };
    uint32_t q_phase = 0;                      // bit b: uses of Q buffer b so far, odd or even
    const uint32_t idesc_s = idesc_f16(F::kRaw ? 0 : 1, kTile, kBlock),
                   idesc_o = idesc_f16_bmn(0, kTile, kHeadDim);
    Cursor cs, cp;
    auto enter = [&](Cursor& c) {              // a segment's first item
      c.j = c.wk.j0;
      c.t = 0;
      c.first = true;
      c.qb = c.wk.tiles == 2 ? 0 : c.qsel;
      if (c.wk.tiles == 1) c.qsel ^= 1;
    };
    auto advance = [&](Cursor& c) {
      ++c.k;
      if (++c.t < c.wk.tiles) return;
      c.t = 0;
      ++c.kv;
      c.first = false;
      if (++c.j < c.wk.j1) return;
      c.more = c.wk.next(ws, a);
      if (c.more) enter(c);
    };
    cs.wk.open(ws, a, sh);
    cs.k = cs.kv = cs.qsel = 0;
    cs.more = cs.wk.next(ws, a);
    if (cs.more) enter(cs);
    cp = cs;
    const uint64_t dq = kstep_desc(smem_u32(qbuf), 0, kTile), dk = kstep_desc(smem_u32(tiles), 0, 128),
                   dv = sdesc_sw128_mn(smem_u32(tiles), kTileBytes / 2);
    const uint32_t hi = (uint32_t)(dk >> 32), vhi = (uint32_t)(dv >> 32);
    auto issue_s = [&]() {
      Cursor& c = cs;
      const int tile = 2 * c.kv, b = tile % F::kTiles, buf = c.k & 1, qb = (c.qb + c.t) & 1;
      if (c.t == 0)
        mbar_wait(F::kRaw ? &sh.ready[b] : &sh.full[b], (uint32_t)(tile / F::kTiles) & 1u, ws.hdr);
      if (c.first) {
        mbar_wait(&sh.q_full[qb], q_phase >> qb & 1u, ws.hdr);
        q_phase ^= 1u << qb;
      }
      if (c.k >= 2) mbar_wait(&sh.o_done[buf], (uint32_t)((c.k - 2) >> 1) & 1u, ws.hdr);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        const uint32_t qlo = (uint32_t)dq + qb * (kTileBytes >> 4),
                       klo = (uint32_t)dk + b * (kTileBytes >> 4), d = tmem + buf * 128;
        umma_ss<false>(d, qlo, hi, klo, hi, idesc_s);
#pragma unroll
        for (int ks = 1; ks < 8; ++ks) {
          const uint32_t o = (ks >> 2) * (kTileBytes >> 5) + (ks & 3) * 2;
          umma_ss<true>(d, qlo + o, hi, klo + o, hi, idesc_s);
        }
        umma_commit(&sh.s_ready[buf]);
        if (c.t + 1 == c.wk.tiles) umma_commit(&sh.empty[b]);
        if (c.j + 1 == c.wk.j1) umma_commit(&sh.q_free[qb]);
      }
      __syncwarp();
      advance(c);
    };
    if (cs.more) issue_s();
    while (cp.more) {
      if (cs.more) issue_s();
      const int tile = 2 * cp.kv + 1, b = tile % F::kTiles, buf = cp.k & 1;
      if (cp.t == 0) {
        // bf16: of an odd ring's uses every second one holds values
        const int use = F::kRaw ? tile / F::kTiles : tile / (2 * F::kTiles);
        mbar_wait(&sh.ready[b], (uint32_t)use & 1u, ws.hdr);
      }
      mbar_wait(&sh.p_ready[buf], (uint32_t)(cp.k >> 1) & 1u, ws.hdr);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        // P: keys 0..63 in columns 0..31 of the buffer, 64..127 in 64..95
        const uint32_t p = tmem + buf * 128, d = tmem + 256 + cp.t * 128,
                       vlo = (uint32_t)dv + b * (kTileBytes >> 4);
        if (cp.first) umma_ts<false>(d, p, vlo, vhi, idesc_o);
        else umma_ts<true>(d, p, vlo, vhi, idesc_o);
#pragma unroll
        for (int ks = 1; ks < 8; ++ks)
          umma_ts<true>(d, p + (ks >> 2) * 64 + (ks & 3) * 8, vlo + 128 * ks, vhi, idesc_o);
        umma_commit(&sh.o_done[buf]);
        if (cp.t + 1 == cp.wk.tiles) umma_commit(&sh.empty[b]);
      }
      __syncwarp();
      advance(cp);
    }
    // every MMA issued here has completed before TMEM goes and the smem is left
    if (elect_one()) umma_commit(&sh.fin);
    __syncwarp();
    mbar_drain(&sh.fin, 0);
  } else if (warp == kIdleWarp) {
    // tokens of no request that has a tree
    const int T = ws.hdr->num_tokens;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
      const int r = ws.tok_req[t];
      if (r >= 0) {
        const Tree tr = tree_of(ws, r);
        if (tr.n > 0) continue;
        if (tr.too_large && lane == 0) set_error(ws.hdr, MSA_DEVERR_TREE);
      }
      for (int x = lane; x < a.Hq * (kHeadDim / 8); x += 32)
        reinterpret_cast<uint4*>(a.out + (int64_t)t * a.Hq * kHeadDim)[x] = make_uint4(0, 0, 0, 0);
      for (int x = lane; x < a.Hq; x += 32) a.lse[(int64_t)t * a.Hq + x] = -INFINITY;
    }
  }
  } else if (warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    regs_down<kConvRegs>();
    const int ct = tid - kConvWarp * 32;
    Walk<KV> wk;
    wk.open(ws, a, sh);
    int n = 0, seg = 0, qsel = 0;
    uint32_t q_used = 0, q_phase = 0;          // bit b: Q buffer b was used; its uses, odd or even
    auto done = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    while (wk.next(ws, a)) {
      // ---- Q rows of the segment's tiles, zero past the last
      for (int t = 0; t < wk.tiles; ++t) {
        const int b = wk.tiles == 2 ? t : qsel;
        if (q_used >> b & 1u) mbar_wait(&sh.q_free[b], (q_phase >> b & 1u) ^ 1u, ws.hdr);
        q_used |= 1u << b;
        q_phase ^= 1u << b;
        bool ovf = false;
        const int first = wk.pair * kPairRows + t * kTile, rows = wk.rows - t * kTile;
#pragma unroll 8
        for (int i = 0; i < 16; ++i) {
          const int x = ct + 128 * i, row = x >> 4, ch = x & 15;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows)
            v = *reinterpret_cast<const uint4*>(
                a.q + a.q_row(wk.q.t0, wk.h, first + row) * kHeadDim + 8 * ch);
          if (F::kRaw) {
            uint32_t h[4];
            to_f16(v, h);
            ovf |= any_inf(h);
            v = make_uint4(h[0], h[1], h[2], h[3]);
          }
          *reinterpret_cast<uint4*>(qbuf + b * kTileBytes + kmaj_off(row, ch, kTile)) = v;
        }
        if (F::kRaw && __any_sync(0xffffffffu, ovf) && lane == 0)
          set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
        done(&sh.q_full[b]);
      }
      if (wk.tiles == 1) qsel ^= 1;
      // ---- pages
      int mine = -1;
      bool ovf = false;
      for (int j = wk.j0; j < wk.j1; ++j, n += 2) {
        const int k = (j - wk.j0) & 31;
        if (k == 0)
          mine = j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + j + lane] : -1;
        const bool usable = __shfl_sync(0xffffffffu, mine, k) >= 0;
        const int ntok = usable ? wk.q.L - j * kBlock : 0;       // keys that exist
        const int all = usable ? wk.q.base - j * kBlock : 0;     // and that every row sees
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int i = n + kind, b = i % F::kTiles;
          uint8_t* tile = tiles + b * kTileBytes;
          if (F::kRaw) {
            const int st = i % F::kStages;
            mbar_wait(&sh.raw_full[st], (uint32_t)(i / F::kStages) & 1u, ws.hdr);
            mbar_wait(&sh.empty[b], ((uint32_t)(i / F::kTiles) & 1u) ^ 1u, ws.hdr);
            if (kind == 0)
              convert_page<KV, false>(raw + st * F::kStageBytes, tile, ct, ntok, all, nullptr);
            else
              convert_page<KV, true>(raw + st * F::kStageBytes, tile, ct, ntok, all,
                                     &sh.bad[seg & 7]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.raw_empty[st]);
            done(&sh.ready[b]);
          } else if (kind == 1) {
            mbar_wait(&sh.full[b], (uint32_t)(i / F::kTiles) & 1u, ws.hdr);
            ovf |= convert_page<KV, true>(nullptr, tile, ct, ntok, all, &sh.bad[seg & 7]);
            done(&sh.ready[b]);
          }
        }
      }
      if (__any_sync(0xffffffffu, ovf) && lane == 0) set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
      ++seg;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    regs_up<kSoftRegs>();
    // Control flow depends on the plan's data and on votes of all eight warps
    // alone (never on what a wait saw): the named barriers match even after a
    // wait gave up.
    constexpr int kBar = 1, kCount = kSoftWarps * 32;
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    Walk<KV> wk;
    wk.open(ws, a, sh);
    int k = 0, seg = 0;
    int4 split = make_int4(0, 0, 0, 0);
    while (wk.next(ws, a)) {
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      uint64_t mk[2];                          // the two rows' masks
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int n = wk.pair * kPairRows + t * kTile + row;
        mk[t] = 0;
        if (n < wk.q.rows) {
          const int i = a.node_of(n);
          mk[t] = a.mask ? (uint64_t)a.mask[wk.q.t0 + i] : ~0ull >> (63 - i);
          if (wk.q.n < 64) mk[t] &= (1ull << wk.q.n) - 1;
        }
      }
      int mine = -1;
      for (int j = wk.j0; j < wk.j1; ++j) {
        const int at = (j - wk.j0) & 31;
        if (at == 0)
          mine = j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + j + lane] : -1;
        const bool usable = __shfl_sync(0xffffffffu, mine, at) >= 0;
        // keys before the nodes, from this thread's first column on
        const int d = wk.q.base - j * kBlock - 64 * wg;
        const bool plain = usable && wk.q.base >= (j + 1) * kBlock;
#pragma unroll 1
        for (int t = 0; t < wk.tiles; ++t, ++k) {
          const int buf = k & 1;
          const uint32_t ts = lanes + buf * 128 + 64 * wg;
          mbar_wait(&sh.s_ready[buf], (uint32_t)(k >> 1) & 1u, ws.hdr);
          tc_fence_after();
          uint32_t x[64];
          tmem_ld64(ts, x);
          tmem_ld_wait();
          if (!plain) {
            const uint64_t mask = t ? mk[1] : mk[0];
            uint64_t vis;
            if (!usable) vis = 0;
            else if (d >= 64) vis = ~0ull;
            else if (d > 0) vis = ((1ull << d) - 1) | (mask << d);
            else vis = d > -64 ? mask >> -d : 0;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!(vis >> i & 1)) x[i] = 0xff800000u;
          }
          float m = t ? m1 : m0, l = t ? l1 : l0;
          float mx = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
          float my = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
          for (int i = 4; i < 64; i += 4) {
            mx = fmax3(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            my = fmax3(my, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
          mx = fmaxf(mx, my);
          // the difference, exact near m; -inf - -inf is NaN: no move
          if (named_bar_any(kBar, kCount, mx - m > a.slack)) {
            sh.red[wg][row] = mx;
            named_bar_sync(kBar, kCount);
            const float mn = fmax3(m, sh.red[0][row], sh.red[1][row]);
            const float alpha = mn == -INFINITY ? 1.f : ex2_approx((m - mn) * a.scale_log2);
            m = mn;
            l *= alpha;
            if (j > wk.j0) {
              // O of this tile: its last P V has to be done
              const int kp = k - wk.tiles;
              mbar_wait(&sh.o_done[kp & 1], (uint32_t)(kp >> 1) & 1u, ws.hdr);
              tc_fence_after();
              if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(lanes + 256 + t * 128 + 64 * wg + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                  tmem_st32(lanes + 256 + t * 128 + 64 * wg + c, o);
                }
                tmem_st_wait();
              }
            }
          }
          // P = 2^((s - m) scale + bias), over this half of S
          const float ref = m == -INFINITY ? 0.f : -m;
          const uint64_t sl = f2(a.scale_log2, a.scale_log2), bias = f2(kBias, kBias),
                         rf = f2(ref, ref);
          uint64_t sum0 = 0, sum1 = 0;
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float p0, p1, p2, p3;
            f2_split(fma_f2(add_f2(f2u(x[2 * i], x[2 * i + 1]), rf), sl, bias), p0, p1);
            f2_split(fma_f2(add_f2(f2u(x[2 * i + 2], x[2 * i + 3]), rf), sl, bias), p2, p3);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            p2 = ex2_approx(p2);
            p3 = ex2_approx(p3);
            sum0 = add_f2(sum0, f2(p0, p1));
            sum1 = add_f2(sum1, f2(p2, p3));
            pk[i] = pack_f16(p0, p1);
            pk[i + 1] = pack_f16(p2, p3);
          }
          tmem_st32(ts, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_ready[buf]);
          float s0, s1;
          f2_split(add_f2(sum0, sum1), s0, s1);
          l += s0 + s1;
          if (t) {
            m1 = m;
            l1 = l;
          } else {
            m0 = m;
            l0 = l;
          }
        }
      }

      // ---- the segment's result: whole rows, or a partial
      const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.starts ? 1 : 0);
#pragma unroll 1
      for (int t = 0; t < wk.tiles; ++t) {
        const int kp = k - wk.tiles + t;
        mbar_wait(&sh.o_done[kp & 1], (uint32_t)(kp >> 1) & 1u, ws.hdr);
        tc_fence_after();
        const float m = t ? m1 : m0;
        named_bar_sync(kBar, kCount);
        sh.red[wg][row] = t ? l1 : l0;
        named_bar_sync(kBar, kCount);
        const float sum = sh.red[0][row] + sh.red[1][row];
        const unsigned long long bad = sh.bad[seg & 7] & (t ? mk[1] : mk[0]);
        const int n = t * kTile + row;         // row of the pair
        const bool on = n < wk.rows;
        const int64_t out_row = on ? a.q_row(wk.q.t0, wk.h, wk.pair * kPairRows + n) : 0;
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          const int dim = 64 * wg + c;
          uint32_t o[32];
          tmem_ld32(lanes + 256 + t * 128 + dim, o);
          tmem_ld_wait();
          if (!on) continue;
          float* part = a.o_part + (slot * a.rows + n) * kHeadDim + dim;
          if (wk.whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * kHeadDim + dim);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                 __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
              dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(part)[i] =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        // rare: values that are not finite, of nodes that the row sees
        for (unsigned long long b = on ? bad : 0; b; b &= b - 1) {
          const int u = wk.q.base + __ffsll((long long)b) - 1;
          const int page = ws.block_table[(int64_t)wk.r * a.max_blocks + u / kBlock];
          for (int dim = 64 * wg; dim < 64 * wg + 64; ++dim) {
            const float v = value_of<KV>(a.v_pool, page, a.Hkv, wk.h, u % kBlock, dim);
            if (fabsf(v) < INFINITY) continue;
            if (wk.whole) {
              __nv_bfloat16* y = a.out + out_row * kHeadDim + dim;
              *y = __float2bfloat16_rn(__bfloat162float(*y) + v);
            } else {
              a.o_part[(slot * a.rows + n) * kHeadDim + dim] += v;
            }
          }
        }
        if (on && wg == 0) {
          if (wk.whole)
            a.lse[out_row] =
                sum == 0.f ? -INFINITY : (m * a.scale_log2 + log2f(sum) - kBias) * kLn2;
          else
            a.ml_part[slot * a.rows + n] = make_float2(m, sum);
        }
      }
      tc_fence_before();
      named_bar_sync(kBar, kCount);            // bad is read, red is free
      if (tid == 0) {
        sh.bad[seg & 7] = 0;
        if (wk.starts && !wk.whole) {          // the range ends inside this group
          const int c1 = (int)range_of(sh.total, sh.ranges, wk.last);
          split = make_int4(c1 - (int)blockIdx.x + 1, wk.q.t0, wk.h, wk.pair << 16 | wk.rows);
        }
      }
      ++seg;
    }
    if (tid == 0) a.split[blockIdx.x] = split;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the merge
// The groups that lie in several CTAs' ranges: every block lists them in order,
// then takes its share of (group, row), a warp a row (a lane four dims).
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeChunks = (kMaxCtas + kMergeThreads - 1) / kMergeThreads;
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(TreeArgs a, int ctas) {
  __shared__ int4 list[kMaxCtas];
  __shared__ int owner[kMaxCtas];
  __shared__ int counts[kMergeChunks * kMergeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  int4 rec[kMergeChunks];
  unsigned starts[kMergeChunks];
#pragma unroll
  for (int k = 0; k < kMergeChunks; ++k) {
    const int c = k * kMergeThreads + tid;
    rec[k] = c < ctas ? a.split[c] : make_int4(0, 0, 0, 0);
    starts[k] = __ballot_sync(0xffffffffu, rec[k].x > 0);
    if (lane == 0) counts[k * kMergeWarps + warp] = __popc(starts[k]);
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int k = 0; k < kMergeChunks; ++k) {
    int at = n + __popc(starts[k] & ((1u << lane) - 1u));
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) {
      const int cnt = counts[k * kMergeWarps + i];
      if (i < warp) at += cnt;
      n += cnt;
    }
    if (rec[k].x > 0) {
      list[at] = rec[k];
      owner[at] = k * kMergeThreads + tid;
    }
  }
  __syncthreads();
  const int64_t items = (int64_t)n * a.rows;
  for (int64_t item = (int64_t)blockIdx.x * kMergeWarps + warp; item < items;
       item += (int64_t)gridDim.x * kMergeWarps) {
    const int gi = (int)(item / a.rows), row = (int)(item - (int64_t)gi * a.rows);
    const int4 g = list[gi];
    if (row >= (g.w & 0xffff)) continue;
    const int64_t c0 = owner[gi];
    // partial i: the second slot of c0, the first of c0 + i
    auto at = [&](int i) { return (2 * (c0 + i) + (i == 0 ? 1 : 0)) * a.rows + row; };
    float M = -INFINITY;
    for (int i = lane; i < g.x; i += 32) M = fmaxf(M, a.ml_part[at(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int i = 0; i < g.x; ++i) {
      const float2 ml = a.ml_part[at(i)];
      const float4 v = *reinterpret_cast<const float4*>(a.o_part + at(i) * kHeadDim + 4 * lane);
      const float f = M == -INFINITY ? 1.f : ex2_approx((ml.x - M) * a.scale_log2);
      l = fmaf(f, ml.y, l);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    const int64_t hq = a.q_row(g.y, g.z, (g.w >> 16) * kPairRows + row);
    const float inv = l == 0.f ? 0.f : a.v_scale / l;
    reinterpret_cast<uint2*>(a.out + hq * kHeadDim)[lane] =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (lane == 0)
      a.lse[hq] = l == 0.f ? -INFINITY : (M * a.scale_log2 + log2f(l) - kBias) * kLn2;
  }
}

template <int KV>
msa_status launch_tree(const WsView& v, const TreeArgs& a, int64_t pool_rows, int64_t units,
                       cudaStream_t s) {
  using F = Form<KV>;
  static std::atomic<bool> ready[64];          // shared-memory limit raised, per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MSA_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(tree_attention_kernel<KV>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem) != cudaSuccess)
      return MSA_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  if (KV != MSA_KV_NVFP4 &&
      (!make_pool_map(&tk, a.k_pool, pool_rows, KV == MSA_KV_FP8_E4M3) ||
       !make_pool_map(&tv, a.v_pool, pool_rows, KV == MSA_KV_FP8_E4M3)))
    return MSA_ERR_CUDA;
  int64_t grid = sm_count();                   // one CTA an SM
  if (grid <= 0) return MSA_ERR_CUDA;
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (grid > units) grid = units;
  msa_status st = launch_pdl(tree_attention_kernel<KV>, dim3((unsigned)grid), dim3(kThreads),
                             F::kSmem, s, v, a, tk, tv);
  if (st != MSA_OK) return st;
  int64_t blocks = grid * ((a.rows + kMergeWarps - 1) / kMergeWarps);
  if (blocks > 8 * sm_count()) blocks = 8 * sm_count();
  return launch_pdl(tree_merge_kernel, dim3((unsigned)blocks), dim3(kMergeThreads), 0, s, a,
                    (int)grid);
}

bool tree_supported(const msa_config& c) {
  return (int64_t)c.max_batch * c.max_blocks_per_req * c.num_kv_heads < (1 << 27) &&
         (int64_t)c.num_pages * c.num_kv_heads < (1 << 24);
}

// Query rows of a partial: of the largest request's pair of tiles.
int part_rows(const msa_config& c) {
  const int64_t nodes = max_tokens_of(c) < kTreeNodes ? max_tokens_of(c) : kTreeNodes;
  const int64_t rows = nodes * (c.num_q_heads / c.num_kv_heads);
  return rows < 1 ? 1 : (rows < kPairRows ? (int)rows : kPairRows);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" size_t msa_tree_attention_scratch_bytes(const msa_config* cfg) {
  if (check_config(cfg) != MSA_OK || !tree_supported(*cfg)) return 0;
  const size_t rows = (size_t)part_rows(*cfg);
  return align_up(2 * (size_t)kMaxCtas * rows * kHeadDim * 4) +
         align_up(2 * (size_t)kMaxCtas * rows * 8) + align_up(kMaxCtas * sizeof(int4));
}

extern "C" msa_status msa_tree_attention(const msa_config* cfg, void* ws, const void* q,
                                         const void* k_pages, const void* v_pages,
                                         const int64_t* tree_mask, void* scratch, void* out,
                                         float* lse, msa_stream_t stream) {
  const msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (!tree_supported(*cfg)) return MSA_ERR_UNSUPPORTED;
  if (!ws || !q || !k_pages || !v_pages || !scratch || !out || !lse) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
      ((uintptr_t)ws & 255) != 0 || ((uintptr_t)scratch & 255) != 0 || ((uintptr_t)lse & 3) != 0 ||
      ((uintptr_t)tree_mask & 7) != 0)
    return MSA_ERR_INVALID_ARG;
  const bool bf16 = cfg->kv_dtype == MSA_KV_BF16;
  TreeArgs a;
  a.scale_log2 = cfg->softmax_scale * (bf16 ? 1.f : cfg->k_scale) * kLog2e;
  if (!(a.scale_log2 > 0.f && a.scale_log2 < INFINITY)) return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0 || cfg->max_batch == 0) return MSA_OK;
  a.slack = fminf(kSlack / a.scale_log2, FLT_MAX);
  a.v_scale = bf16 ? 1.f : cfg->v_scale;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.G = a.Hq / a.Hkv;
  a.g_magic = ((1u << 20) + a.G - 1) / a.G;    // exact for rows up to 1024 and G <= 16
  a.max_blocks = cfg->max_blocks_per_req;
  a.rows = part_rows(*cfg);
  a.q = (const __nv_bfloat16*)q;
  a.k_pool = (const uint8_t*)k_pages;
  a.v_pool = (const uint8_t*)v_pages;
  a.mask = tree_mask;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.o_part = (float*)scratch;
  a.ml_part = (float2*)((char*)scratch + align_up(2 * (size_t)kMaxCtas * a.rows * kHeadDim * 4));
  a.split = (int4*)((char*)a.ml_part + align_up(2 * (size_t)kMaxCtas * a.rows * 8));
  const WsView v = view_of(*cfg, ws);
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t pool_rows = (int64_t)cfg->num_pages * a.Hkv * kBlock;
  const int64_t units = (int64_t)cfg->max_batch * cfg->max_blocks_per_req * a.Hkv * 4;
  switch (cfg->kv_dtype) {
    case MSA_KV_BF16: return launch_tree<MSA_KV_BF16>(v, a, pool_rows, units, s);
    case MSA_KV_FP8_E4M3: return launch_tree<MSA_KV_FP8_E4M3>(v, a, pool_rows, units, s);
    default: return launch_tree<MSA_KV_NVFP4>(v, a, pool_rows, units, s);
  }
}
