// msa_dense_decode: attention over the whole context of every request, held in
// an NVFP4 cache -- the full-attention layers of a hybrid model, whose sparse
// layers go through msa_sparse_decode on the same plan and pools.
//
// sglang minimax_sparse_backend.py (MiniMaxHybridAttnBackend) routes each layer
// by its id to the sparse backend or to a dense one; vLLM
// sparse_attention_msa.py (MiniMaxM3SparseMSANvfp4Backend) gives the NVFP4
// pages: per KV head a key slot 2h and a value slot 2h + 1, rows of 64 bytes
// of E2M1 codes and 8 E4M3 block scales.
//
// Mathematics.  For token t and query head q of KV head h's group, over the
// keys u at positions <= position(t):
//     s_u = scale * k_scale * sum_d q_d * e2m1(K_ud) * e4m3(K_u,d/16)
//     out = v_scale * sum_u 2^(s'_u - m) v_u / sum_u 2^(s'_u - m),   s' = s log2 e,
// in one pass with a running maximum m and sum.  e2m1 x e4m3 has at most 6
// significant bits and magnitudes 0 or 2^-10 .. 2688, so keys and values are
// exact fp16 operands, and so are bf16 queries of fp16 magnitude (others are
// flagged, MSA_DEVERR_FP16_RANGE); products accumulate in fp32.  The
// probabilities are rounded to fp16 for P V (2^-11 relative, below the bf16
// rounding of the output); they are carried as 2^(s' - m + 7) so that fp16's
// normal range reaches 2^-21 below the running maximum.  Their sum is taken
// before that rounding.
//
// Work split.  One unit of work is a 128-key page of one (request, KV head).
// The step's units, request by request and head by head, are cut into equal
// contiguous ranges, one per CTA, whatever the lengths are; a (request, head)
// whose units lie in several CTAs leaves one partial per CTA in the scratch,
// merged in CTA order by the second kernel.  All G * q_len query rows of a
// head share each read of a key.
#include "msa_device.cuh"

namespace msa {
namespace {

constexpr int kTileWarps = 4;                  // warps that share a page, 32 keys each
constexpr int kMaxRows = 64;                   // query rows (tokens x group) of a KV head
constexpr int kCtasMax = 640;                  // partial slots: two per CTA
constexpr int kPageBytes = kBlock * kFp4Row;   // one K or V slot, 9216 bytes
constexpr float kBias = 7.f;                   // exponent offset of the probabilities

struct DenseArgs {
  int Hkv, Hq, G, q_len, max_blocks, rows;     // rows = G * q_len
  float scale_log2, v_scale;
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;                               // [2 * CTAs][rows][128]
  float2* ml_part;                             // [2 * CTAs][rows] (m, sum)
};

// The range of units of CTA c of n: [U c / n, U (c + 1) / n).
__device__ __forceinline__ int64_t range_of(int64_t U, int c, int n) { return U * c / n; }
// The CTA whose range holds unit u.
__device__ __forceinline__ int cta_of(int64_t U, int64_t u, int n) {
  return (int)(((u + 1) * n - 1) / U);
}

// The request that holds unit u: the last r with cu[r] * Hkv <= u (requests
// without blocks hold none).  One warp, 32 probes at a time.
__device__ __forceinline__ int request_of(const int32_t* cu, int batch, int Hkv, int64_t u,
                                          int lane) {
  int lo = 0, n = batch;                       // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool below = i < lo + n && (int64_t)cu[i] * Hkv <= u;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));   // lane 0 is always below
    const int end = lo + n;
    lo += k * step;
    n = min(step, end - lo);
  }
  return lo;
}

// Key n of k-step group nt (n-tile nt, column col) of a warp's 32 keys.  Keys
// 4 apart sit 72 words = 8 banks apart, so the eight rows a warp reads together
// (K: columns 0..7; V: columns of one parity) fall on distinct banks.
__device__ __forceinline__ int key_of(int nt, int col) { return 4 * (col ^ (col >> 2)) + nt; }

// Two keys' code words (8 elements each) -> f16x2 pairs (key a, key b) of
// elements 0..7, times the pair of block scales.
__device__ __forceinline__ void pair_values(uint32_t wa, uint32_t wb, uint32_t sc,
                                            uint32_t (&h)[8]) {
  constexpr uint32_t m = 0x0f0f0f0fu;
  const uint32_t even = (wa & m) | ((wb << 4) & ~m);
  const uint32_t odd = ((wa >> 4) & m) | (wb & ~m);
  uint32_t e[4], o[4];
  e2m1x8_to_f16x2(even, e);
  e2m1x8_to_f16x2(odd, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = hmul2_u32(e[i], sc);
    h[2 * i + 1] = hmul2_u32(o[i], sc);
  }
}

// Running state of MT 16-row tiles over this warp's keys.
template <int MT>
struct State {
  float acc[MT][16][4];        // tile e: dims 32 c + e (0, 2) and 32 c + 16 + e (1, 3)
  float m[MT][2], l[MT][2];    // rows g and g + 8; l is this lane's part of the sum

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[i][e][0] = acc[i][e][1] = acc[i][e][2] = acc[i][e][3] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
  }
};

// One page: this warp's 32 keys against MT row tiles.  kt, vt: the warp's rows
// of the K and V slot.  lim[mt][i]: keys of the warp's 32 that row i may see
// (only read if EDGE; any value, <= 0 is none); ntok: keys that exist.
template <int MT, bool EDGE>
__device__ __forceinline__ void page_step(State<MT>& st, const uint4* qf, const uint8_t* kt,
                                          const uint8_t* vt, float scale_log2, int lane,
                                          const int (&lim)[MT][2], int ntok, int all) {
  const int g = lane >> 2, c = lane & 3;
  // ---- S = Q K^T: lane (g, c) holds blocks c and 4 + c of key column g
  float sc[MT][4][4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    const uint8_t* kr = kt + key_of(nt, g) * kFp4Row;
    const uint2 wa = *reinterpret_cast<const uint2*>(kr + 8 * c);
    const uint2 wb = *reinterpret_cast<const uint2*>(kr + 32 + 8 * c);
    const uint2 sb = *reinterpret_cast<const uint2*>(kr + kHeadDim / 2);
    const uint32_t s2 =
        e4m3x2_to_f16x2((uint16_t)__byte_perm(sb.x, sb.y, (uint32_t)(c | (4 + c) << 4)));
    const uint32_t words[4] = {wa.x, wa.y, wb.x, wb.y};
#pragma unroll
    for (int i = 0; i < MT; ++i) sc[i][nt][0] = sc[i][nt][1] = sc[i][nt][2] = sc[i][nt][3] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t sp = __byte_perm(s2, 0u, w < 2 ? 0x1010u : 0x3232u);
      uint32_t h[4];
      e2m1x8_to_f16x2(words[w], h);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t b0 = hmul2_u32(h[2 * s], sp), b1 = hmul2_u32(h[2 * s + 1], sp);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint4 q4 = qf[(i * 8 + 2 * w + s) * 32 + lane];
          const uint32_t a[4] = {q4.x, q4.y, q4.z, q4.w};
          mma_f16(sc[i][nt], a, b0, b1);
        }
      }
    }
  }
  // ---- online softmax (log2 domain)
  uint32_t pa[MT][2][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = sc[i][nt][e] * scale_log2;
        if (EDGE && key_of(nt, 2 * c + (e & 1)) >= lim[i][e >> 1]) x = -INFINITY;
        sc[i][nt][e] = x;
        mx[e >> 1] = fmaxf(mx[e >> 1], x);
      }
    }
    float mref[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
      mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
      const float mn = fmaxf(st.m[i][k], mx[k]);
      mref[k] = mn == -INFINITY ? 0.f : mn;
      const float alpha = ex2_approx(st.m[i][k] - mref[k]);
      st.m[i][k] = mn;
      st.l[i][k] *= alpha;
      mref[k] -= kBias;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        st.acc[i][e][2 * k] *= alpha;
        st.acc[i][e][2 * k + 1] *= alpha;
      }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const float p0 = ex2_approx(sc[i][nt][0] - mref[0]), p1 = ex2_approx(sc[i][nt][1] - mref[0]);
      const float p2 = ex2_approx(sc[i][nt][2] - mref[1]), p3 = ex2_approx(sc[i][nt][3] - mref[1]);
      st.l[i][0] += p0 + p1;
      st.l[i][1] += p2 + p3;
      pa[i][nt >> 1][(nt & 1) * 2] = pack_f16(p0, p1);
      pa[i][nt >> 1][(nt & 1) * 2 + 1] = pack_f16(p2, p3);
    }
  }
  // ---- O += P V: lane (g, c) holds block g of key columns 2c, 2c + 1
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint32_t b[2][16];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ka = key_of(2 * kk + j, 2 * c), kb = key_of(2 * kk + j, 2 * c + 1);
      const uint8_t *ra = vt + ka * kFp4Row, *rb = vt + kb * kFp4Row;
      const uint2 xa = *reinterpret_cast<const uint2*>(ra + 8 * g);
      const uint2 xb = *reinterpret_cast<const uint2*>(rb + 8 * g);
      uint32_t sa = ra[kHeadDim / 2 + g], sb = rb[kHeadDim / 2 + g];
      if (EDGE) {
        // rows past the end may hold anything, and a row some query may not
        // see may hold a NaN scale: 0 * NaN is not 0 (page_nan adds them back)
        if (ka >= ntok || (ka >= all && (sa & 0x7f) == 0x7f)) sa = 0;
        if (kb >= ntok || (kb >= all && (sb & 0x7f) == 0x7f)) sb = 0;
      }
      const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(sa | sb << 8));
      uint32_t h[8];
      pair_values(xa.x, xb.x, s2, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) b[j][e] = h[e];
      pair_values(xa.y, xb.y, s2, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) b[j][8 + e] = h[e];
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
#pragma unroll
      for (int i = 0; i < MT; ++i) mma_f16(st.acc[i][e], pa[i][kk], b[0][e], b[1][e]);
  }
  // NaN scales among the keys that only later tokens see
  if (EDGE) {
    for (int u = max(all, 0); u < min(ntok, 32); ++u) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if ((vt[u * kFp4Row + kHeadDim / 2 + 2 * c + half] & 0x7f) != 0x7f) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (u < lim[i][k])
#pragma unroll
              for (int e = 0; e < 16; ++e) st.acc[i][e][2 * k + half] = NAN;
      }
    }
  }
}

// MT row tiles of 16 per warp, RG groups of such warps: 16 MT RG rows.
template <int MT, int RG>
__global__ void __launch_bounds__(kTileWarps* RG * 32)
dense_decode_kernel(WsView ws, DenseArgs a) {
  constexpr int kThreadsN = kTileWarps * RG * 32, kRows = 16 * MT * RG;
  __shared__ __align__(16) uint4 qfrag[MT * RG * 8 * 32];
  __shared__ float red_m[kTileWarps][kRows], red_l[kTileWarps][kRows];
  extern __shared__ __align__(16) float obuf[];           // [4][kRows][64]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rg = warp / kTileWarps, kw = warp % kTileWarps;
  const int g = lane >> 2, c = lane & 3;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t U = (int64_t)ws.hdr->total_blocks * a.Hkv;
  const int n = (int)min((int64_t)gridDim.x, U);
  if ((int)blockIdx.x >= n) return;
  const int64_t end = range_of(U, blockIdx.x + 1, n);
  int64_t u = range_of(U, blockIdx.x, n);
  const int batch = ws.hdr->batch;
  int r = request_of(ws.req_cu_nb, batch, a.Hkv, u, lane);
  while (u < end) {
    while (r + 1 < batch && (int64_t)ws.req_cu_nb[r + 1] * a.Hkv <= u) ++r;
    const int nb = ws.req_nb[r], L = ws.req_seq_len[r], qs = ws.req_qstart[r];
    const int nq = ws.req_qstart[r + 1] - qs;
    const int64_t first = (int64_t)ws.req_cu_nb[r] * a.Hkv;
    const int h = (int)((u - first) / nb);
    const int64_t ga = first + (int64_t)h * nb, gb = ga + nb;      // the group's units
    const int j0 = (int)(u - ga), j1 = (int)(min(gb, end) - ga);
    const int64_t seg = u;
    u = ga + j1;
    if (nq > a.q_len) {                                            // more tokens than the config's
      if (tid == 0) set_error(ws.hdr, MSA_DEVERR_SEQ_LEN);
      continue;
    }
    const int rows = nq * a.G;
    // ---- the rows' A fragments: k-step 2 w + s of lane (g, c) takes dims
    // 16 c + 64 (w / 2) + 8 (w % 2) + 4 s + 0..3
    bool ovf = false;
    __syncthreads();
    for (int x = warp; x < MT * RG * 8; x += kTileWarps * RG) {
      const int ks = x & 7, w = ks >> 1;
      const int dim = 16 * c + 64 * (w >> 1) + 8 * (w & 1) + 4 * (ks & 1);
      uint32_t f[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (x >> 3) * 16 + g + 8 * k;
        uint2 v = make_uint2(0u, 0u);
        if (row < rows)
          v = *reinterpret_cast<const uint2*>(
              a.q + ((int64_t)(qs + row / a.G) * a.Hq + h * a.G + row % a.G) * kHeadDim + dim);
        f[k] = bf16x2_to_f16x2(v.x);
        f[k + 2] = bf16x2_to_f16x2(v.y);
        ovf |= f16x2_has_inf(f[k]) | f16x2_has_inf(f[k + 2]);
      }
      qfrag[x * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
    }
    if (__any_sync(0xffffffffu, ovf) && lane == 0) set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
    __syncthreads();

    State<MT> st;
    st.clear();
    int seen[MT][2];                           // keys of the request each row sees
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (rg * MT + i) * 16 + g + 8 * k;
        seen[i][k] = L - nq + min(row / a.G, max(nq - 1, 0)) + 1;
      }
    const uint4* qf = qfrag + rg * MT * 8 * 32;
    for (int j = j0; j < j1; ++j) {
      const int page = ws.block_table[(int64_t)r * a.max_blocks + j];
      if (page < 0) continue;                  // flagged by the plan
      const int base = j * kBlock + kw * 32;   // this warp's first key
      const int64_t slot = ((int64_t)page * a.Hkv + h) * 2;
      const uint8_t* kt = a.k_pool + slot * kPageBytes + kw * 32 * kFp4Row;
      const uint8_t* vt = a.v_pool + (slot + 1) * kPageBytes + kw * 32 * kFp4Row;
      int lim[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) lim[i][k] = seen[i][k] - base;
      const int all = L - nq + 1 - base;       // keys that every row sees
      if (all >= 32)
        page_step<MT, false>(st, qf, kt, vt, a.scale_log2, lane, lim, 32, 32);
      else if (L - base > 0)
        page_step<MT, true>(st, qf, kt, vt, a.scale_log2, lane, lim, L - base, all);
    }

    // ---- merge the four warps of each row group
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = st.l[i][k];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c == 0) {
          const int row = (rg * MT + i) * 16 + g + 8 * k;
          red_m[kw][row] = st.m[i][k];
          red_l[kw][row] = x;
        }
      }
    __syncthreads();
    float f[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (rg * MT + i) * 16 + g + 8 * k;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) M = fmaxf(M, red_m[w][row]);
        f[i][k] = M == -INFINITY ? 1.f : ex2_approx(st.m[i][k] - M);
      }
    const bool whole = seg == ga && u == gb;
    const int slot = 2 * (int)blockIdx.x + (seg == ga ? 1 : 0);
#pragma unroll
    for (int p = 0; p < 2; ++p) {              // dims 32 c + 16 half + 8 p + 0..7
      if (p) __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = (rg * MT + i) * 16 + g + 8 * k;
            float4* dst = reinterpret_cast<float4*>(obuf + (kw * kRows + row) * 64 + 16 * c +
                                                    8 * half);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = st.acc[i][8 * p + e][2 * k + half] * f[i][k];
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
      __syncthreads();
      for (int x = tid; x < kRows * 8; x += kThreadsN) {
        const int row = x >> 3, part = x & 7;
        if (row >= rows) continue;
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) M = fmaxf(M, red_m[w][row]);
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w)
          sum += red_l[w][row] * (M == -INFINITY ? 1.f : ex2_approx(red_m[w][row] - M));
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) {
          const float4* s4 =
              reinterpret_cast<const float4*>(obuf + (w * kRows + row) * 64 + 8 * part);
          const float4 x0 = s4[0], x1 = s4[1];
          v[0] += x0.x; v[1] += x0.y; v[2] += x0.z; v[3] += x0.w;
          v[4] += x1.x; v[5] += x1.y; v[6] += x1.z; v[7] += x1.w;
        }
        const int dim = 16 * part + 8 * p;
        if (whole) {
          const int64_t hq = (int64_t)(qs + row / a.G) * a.Hq + h * a.G + row % a.G;
          const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pk[e] = pack_bf16(v[2 * e] * inv, v[2 * e + 1] * inv);
          *reinterpret_cast<uint4*>(a.out + hq * kHeadDim + dim) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
          if (p == 0 && part == 0)
            a.lse[hq] = sum == 0.f ? -INFINITY : (M + log2f(sum) - kBias) * kLn2;
        } else {
          float4* dst = reinterpret_cast<float4*>(
              a.o_part + ((int64_t)slot * a.rows + row) * kHeadDim + dim);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (p == 0 && part == 0)
            a.ml_part[(int64_t)slot * a.rows + row] = make_float2(M, sum);
        }
      }
    }
    __syncthreads();
  }
}

// Merges the partials of the (request, head) groups that lie in several CTAs'
// ranges, in CTA order: block (x, y) takes the group that starts in CTA x's
// range and ends behind it, and rows y * kMergeRows .. of it, four warps a
// row.  Tokens without a valid request get out = 0, lse = -inf.
constexpr int kMergeRows = 2;
__global__ void __launch_bounds__(kMergeRows * 128)
dense_merge_kernel(WsView ws, DenseArgs a, int ctas) {
  __shared__ float4 part[kMergeRows][4][32];
  __shared__ float part_l[kMergeRows][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mr = warp >> 2, w4 = warp & 3;
  griddep_launch_dependents();
  griddep_wait();
  const int T = ws.hdr->num_tokens, batch = ws.hdr->batch;
  const int64_t U = (int64_t)ws.hdr->total_blocks * a.Hkv;
  // idle tokens, and those of requests with more tokens than the config's
  for (int64_t x = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kMergeRows * 4 + warp;
       x < (int64_t)T * a.Hq; x += (int64_t)gridDim.x * gridDim.y * kMergeRows * 4) {
    const int t = (int)(x / a.Hq);
    const int r = ws.tok_req[t];
    if (r >= 0 && ws.req_qstart[r + 1] - ws.req_qstart[r] <= a.q_len) continue;
    reinterpret_cast<uint2*>(a.out + x * kHeadDim)[lane] = make_uint2(0u, 0u);
    if (lane == 0) a.lse[x] = -INFINITY;
  }
  const int n = (int)min((int64_t)ctas, U);
  const int c0 = blockIdx.x;
  if (c0 >= n) return;
  const int64_t lo = range_of(U, c0, n), hi = range_of(U, c0 + 1, n);
  const int r = request_of(ws.req_cu_nb, batch, a.Hkv, hi - 1, lane);
  const int nb = ws.req_nb[r], qs = ws.req_qstart[r], nq = ws.req_qstart[r + 1] - qs;
  const int64_t first = (int64_t)ws.req_cu_nb[r] * a.Hkv;
  const int h = (int)((hi - 1 - first) / nb);
  const int64_t ga = first + (int64_t)h * nb, gb = ga + nb;
  if (ga < lo || gb <= hi || nq > a.q_len) return;           // block-uniform
  const int c1 = cta_of(U, gb - 1, n), np = c1 - c0 + 1;
  const int row = blockIdx.y * kMergeRows + mr;
  const bool on = row < nq * a.G;
  // partial i: the second slot of c0, the first of c0 + i
  auto slot_of = [&](int i) { return 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0); };
  float M = -INFINITY;
  if (on)
    for (int i = lane; i < np; i += 32)
      M = fmaxf(M, a.ml_part[slot_of(i) * a.rows + row].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (on) {
#pragma unroll 4
    for (int i = w4; i < np; i += 4) {
      const float2 ml = a.ml_part[slot_of(i) * a.rows + row];
      const float4 v = *reinterpret_cast<const float4*>(
          a.o_part + (slot_of(i) * a.rows + row) * kHeadDim + 4 * lane);
      const float f = M == -INFINITY ? 1.f : ex2_approx(ml.x - M);
      l = fmaf(f, ml.y, l);
      o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
  }
  part[mr][w4][lane] = o;
  if (lane == 0) part_l[mr][w4] = l;
  __syncthreads();
  if (!on || w4 != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 v = part[mr][w][lane];
    o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
    l += part_l[mr][w];
  }
  const int64_t hq = (int64_t)(qs + row / a.G) * a.Hq + h * a.G + row % a.G;
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
  reinterpret_cast<uint2*>(a.out + hq * kHeadDim)[lane] =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (lane == 0) a.lse[hq] = l == 0.f ? -INFINITY : (M + log2f(l) - kBias) * kLn2;
}

template <int MT, int RG>
msa_status launch_dense(const WsView& v, const DenseArgs& a, int64_t units, cudaStream_t s) {
  constexpr int kThreadsN = kTileWarps * RG * 32;
  const size_t smem = (size_t)kTileWarps * 16 * MT * RG * 64 * 4;
  // set on every call: cheap, and right on whatever device is current
  if (cudaFuncSetAttribute(dense_decode_kernel<MT, RG>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return MSA_ERR_CUDA;
  int64_t grid = (int64_t)sm_count() * 3;
  if (grid > kCtasMax) grid = kCtasMax;
  if (grid > units) grid = units;
  if (grid <= 0) return MSA_ERR_CUDA;
  msa_status st = launch_pdl(dense_decode_kernel<MT, RG>, dim3((unsigned)grid), dim3(kThreadsN),
                             smem, s, v, a);
  if (st != MSA_OK) return st;
  return launch_pdl(dense_merge_kernel,
                    dim3((unsigned)grid, (unsigned)((a.rows + kMergeRows - 1) / kMergeRows)),
                    dim3(kMergeRows * 128), 0, s, v, a, (int)grid);
}

bool dense_supported(const msa_config& c) {
  return !is_prefill(c) && c.kv_dtype == MSA_KV_NVFP4 &&
         (int64_t)c.num_q_heads / c.num_kv_heads * c.q_len <= kMaxRows;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" size_t msa_dense_decode_scratch_bytes(const msa_config* cfg) {
  if (check_config(cfg) != MSA_OK || !dense_supported(*cfg)) return 0;
  const size_t rows = (size_t)(cfg->num_q_heads / cfg->num_kv_heads) * cfg->q_len;
  return align_up(2 * (size_t)kCtasMax * rows * kHeadDim * 4) +
         align_up(2 * (size_t)kCtasMax * rows * 8);
}

extern "C" msa_status msa_dense_decode(const msa_config* cfg, void* ws, const void* q,
                                       const void* k_pages, const void* v_pages, void* scratch,
                                       void* out, float* lse, msa_stream_t stream) {
  msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (is_prefill(*cfg)) return MSA_ERR_INVALID_ARG;
  if (!dense_supported(*cfg)) return MSA_ERR_UNSUPPORTED;
  if (!ws || !q || !k_pages || !v_pages || !scratch || !out || !lse) return MSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
      ((uintptr_t)scratch & 255) != 0 || ((uintptr_t)lse & 3) != 0)
    return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0) return MSA_OK;
  DenseArgs a;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.G = a.Hq / a.Hkv;
  a.q_len = cfg->q_len;
  a.max_blocks = cfg->max_blocks_per_req;
  a.rows = a.G * a.q_len;
  a.scale_log2 = cfg->softmax_scale * cfg->k_scale * kLog2e;
  a.v_scale = cfg->v_scale;
  a.q = (const __nv_bfloat16*)q;
  a.k_pool = (const uint8_t*)k_pages;
  a.v_pool = (const uint8_t*)v_pages;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.o_part = (float*)scratch;
  a.ml_part = (float2*)((char*)scratch + align_up(2 * (size_t)kCtasMax * a.rows * kHeadDim * 4));
  const WsView v = view_of(*cfg, ws);
  const int64_t units = (int64_t)cfg->max_batch * cfg->max_blocks_per_req * a.Hkv;
  cudaStream_t s = (cudaStream_t)stream;
  if (a.rows <= 16) return launch_dense<1, 1>(v, a, units, s);
  if (a.rows <= 32) return launch_dense<2, 1>(v, a, units, s);
  return launch_dense<2, 2>(v, a, units, s);
}
