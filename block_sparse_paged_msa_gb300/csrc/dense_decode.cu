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
// contiguous ranges, one per team of warps, whatever the lengths are; a (request,
// head) whose units lie in several ranges leaves one partial per team in the
// scratch, merged in team order by the second kernel.  All G * q_len query rows of a
// head share each read of a key.
#include <atomic>

#include "msa_device.cuh"

namespace msa {
namespace {

constexpr int kTileWarps = 4;                  // warps that share a page, 32 keys each
constexpr int kTileTokens = kBlock / kTileWarps;
constexpr int kMaxRows = 64;                   // query rows (tokens x group) of a KV head
constexpr int kTeamsMax = 640;                  // partial slots: two per team
constexpr int kPageBytes = kBlock * kFp4Row;   // one K or V slot, 9216 bytes
constexpr float kBias = 7.f;                   // exponent offset of the probabilities
constexpr float kSlack = 8.f;                  // 2^(kBias + kSlack) is below fp16's largest

struct DenseArgs {
  int Hkv, Hq, G, q_len, max_blocks, max_batch, rows;   // rows = G * q_len
  float scale_log2, v_scale;
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;                               // [2 * teams][rows][128]
  float2* ml_part;                             // [2 * teams][rows] (m, sum)
};

// The range of units of team c of n: [U c / n, U (c + 1) / n).
__device__ __forceinline__ int64_t range_of(int64_t U, int c, int n) { return U * c / n; }
// The team whose range holds unit u.
__device__ __forceinline__ int team_of(int64_t U, int64_t u, int n) {
  return (int)(((u + 1) * n - 1) / U);
}

// The request that holds unit u: the last r with cu[r] * Hkv <= u (requests
// without blocks hold none).  One warp, 32 probes at a time; `first` is this
// lane's cu[min(lane, max_batch)], so that a batch of up to 32 needs no load.
__device__ __forceinline__ int request_of(const int32_t* cu, int first, int batch, int Hkv,
                                          int64_t u, int lane) {
  int lo = 0, n = batch;                       // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool in = i < lo + n;
    const int at = batch <= 32 ? first : (in ? cu[i] : 0);
    const bool below = in && (int64_t)at * Hkv <= u;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));   // lane 0 is always below
    const int end = lo + n;
    lo += k * step;
    n = min(step, end - lo);
  }
  return lo;
}

// A team's walk over its range: one segment per (request, KV head) it meets.
struct Walk {
  int64_t u, end;              // next unit, end of the range
  int r;                       // request of unit u
  // the current segment
  int h, j0, j1, nq, qs, L, nb;
  bool starts, whole;          // it starts its group; it is all of its group

  // The range of team vid; false if it has none.  One warp, all lanes alike.
  __device__ __forceinline__ bool open(const WsView& ws, int max_batch, int Hkv, int vid,
                                       int teams, int lane) {
    const int first = ws.req_cu_nb[min(lane, max_batch)];
    const int batch = ws.hdr->batch;
    const int64_t U = (int64_t)ws.hdr->total_blocks * Hkv;
    const int n = (int)min((int64_t)teams, U);
    if (vid >= n) return false;
    u = range_of(U, vid, n);
    end = range_of(U, vid + 1, n);
    r = request_of(ws.req_cu_nb, first, batch, Hkv, u, lane);
    return true;
  }
  // The next segment; false at the end of the range.
  __device__ __forceinline__ bool next(const WsView& ws, int Hkv) {
    if (u >= end) return false;
    int cu0 = ws.req_cu_nb[r], cu1 = ws.req_cu_nb[r + 1];   // u is below the last request's end
    while ((int64_t)cu1 * Hkv <= u) {
      ++r;
      cu0 = cu1;
      cu1 = ws.req_cu_nb[r + 1];
    }
    qs = ws.req_qstart[r];
    nq = ws.req_qstart[r + 1] - qs;
    L = ws.req_seq_len[r];
    nb = cu1 - cu0;
    const int64_t first = (int64_t)cu0 * Hkv;
    h = (int)((u - first) / nb);
    const int64_t ga = first + (int64_t)h * nb;             // the group's units: [ga, ga + nb)
    j0 = (int)(u - ga);
    j1 = (int)(min(ga + nb, end) - ga);
    starts = j0 == 0;
    whole = starts && j1 == nb;
    u = ga + j1;
    return true;
  }
};

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
  float m[MT][2];              // reference exponents of rows g and g + 8
  uint64_t l[MT][2];           // this thread's part of the sums, as f32 pairs
};

// S = Q K^T of the warp's 32 keys (kt: their rows): lane (g, c) holds blocks c
// and 4 + c of key column g, k-step 2 w + s takes elements 4 s .. 4 s + 3 of
// its code word w.
template <int MT>
__device__ __forceinline__ void scores(float (&sc)[MT][4][4], const uint4* qf, const uint8_t* kt,
                                       int lane) {
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* kr = kt + key_of(0, g) * kFp4Row;
  uint32_t s2[4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    const uint2 sb = *reinterpret_cast<const uint2*>(kr + nt * kFp4Row + kHeadDim / 2);
    s2[nt] = e4m3x2_to_f16x2((uint16_t)__byte_perm(sb.x, sb.y, (uint32_t)(c | (4 + c) << 4)));
#pragma unroll
    for (int i = 0; i < MT; ++i) sc[i][nt][0] = sc[i][nt][1] = sc[i][nt][2] = sc[i][nt][3] = 0.f;
  }
#pragma unroll
  for (int wb = 0; wb < 2; ++wb) {
    uint2 x[4];
    uint32_t sp[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      x[nt] = *reinterpret_cast<const uint2*>(kr + nt * kFp4Row + 32 * wb + 8 * c);
      sp[nt] = __byte_perm(s2[nt], 0u, wb ? 0x3232u : 0x1010u);
    }
#pragma unroll
    for (int wi = 0; wi < 2; ++wi) {
      uint32_t q[MT][2][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 v = qf[(i * 8 + 4 * wb + 2 * wi + s) * 32 + lane];
          q[i][s][0] = v.x; q[i][s][1] = v.y; q[i][s][2] = v.z; q[i][s][3] = v.w;
        }
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        uint32_t h[4];
        e2m1x8_to_f16x2(wi ? x[nt].y : x[nt].x, h);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t b0 = hmul2_u32(h[2 * s], sp[nt]), b1 = hmul2_u32(h[2 * s + 1], sp[nt]);
#pragma unroll
          for (int i = 0; i < MT; ++i) mma_f16(sc[i][nt], q[i][s], b0, b1);
        }
      }
    }
  }
}

// Scores -> probabilities 2^(s' - m + kBias) as A fragments, with the sums.
// The reference m of a row moves (and the row's output is rescaled) only when
// it is still unset or a score passes it by more than kSlack: any m within
// fp16's range of the maximum gives the same quotient.
template <int MT, bool EDGE>
__device__ __forceinline__ void softmax_step(State<MT>& st, float (&sc)[MT][4][4],
                                             uint32_t (&pa)[MT][2][4], float scale_log2, int lane,
                                             const int (&lim)[MT][2]) {
  const int c = lane & 3;
  bool move = false;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float mx[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (EDGE && key_of(nt, 2 * c + e) >= lim[i][k]) sc[i][nt][2 * k + e] = -INFINITY;
      mx[k] = fmax3(fmax3(sc[i][0][2 * k], sc[i][0][2 * k + 1], sc[i][1][2 * k]),
                    fmax3(sc[i][1][2 * k + 1], sc[i][2][2 * k], sc[i][2][2 * k + 1]),
                    fmaxf(sc[i][3][2 * k], sc[i][3][2 * k + 1]));
      move |= mx[k] * scale_log2 > st.m[i][k] + kSlack;
    }
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = sc[i][0][2 * k];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) x = fmax3(x, sc[i][nt][2 * k], sc[i][nt][2 * k + 1]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float mn = fmaxf(st.m[i][k], x * scale_log2);
        const float alpha = mn == -INFINITY ? 1.f : ex2_approx(st.m[i][k] - mn);
        st.m[i][k] = mn;
        st.l[i][k] = mul_f2(st.l[i][k], f2(alpha, alpha));
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          st.acc[i][e][2 * k] *= alpha;
          st.acc[i][e][2 * k + 1] *= alpha;
        }
      }
  }
  const uint64_t sl = f2(scale_log2, scale_log2);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float off = kBias - (st.m[i][k] == -INFINITY ? 0.f : st.m[i][k]);
      const uint64_t o2 = f2(off, off);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float x0, x1;
        f2_split(fma_f2(f2(sc[i][nt][2 * k], sc[i][nt][2 * k + 1]), sl, o2), x0, x1);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        st.l[i][k] = add_f2(st.l[i][k], f2(p0, p1));
        pa[i][nt >> 1][(nt & 1) * 2 + k] = pack_f16(p0, p1);
      }
    }
}

// O += P V of the warp's 32 keys (vt: their rows): lane (g, c) holds block g of
// key columns 2c and 2c + 1.  EDGE: ntok keys exist, and every row sees `all`
// of them.
template <int MT, bool EDGE>
__device__ __forceinline__ void values(State<MT>& st, const uint32_t (&pa)[MT][2][4],
                                       const uint8_t* vt, int lane, const int (&lim)[MT][2],
                                       int ntok, int all) {
  const int g = lane >> 2, c = lane & 3;
  const int ka = key_of(0, 2 * c), kb = key_of(0, 2 * c + 1);
  const uint8_t *va = vt + ka * kFp4Row, *vb = vt + kb * kFp4Row;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint2 xa[2], xb[2];
    uint32_t s2[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nt = 2 * kk + j;
      xa[j] = *reinterpret_cast<const uint2*>(va + nt * kFp4Row + 8 * g);
      xb[j] = *reinterpret_cast<const uint2*>(vb + nt * kFp4Row + 8 * g);
      uint32_t sa = va[nt * kFp4Row + kHeadDim / 2 + g], sb = vb[nt * kFp4Row + kHeadDim / 2 + g];
      if (EDGE) {
        // rows past the end may hold anything, and a row that some query may
        // not see may hold a NaN scale: 0 * NaN is not 0 (added back below)
        if (ka + nt >= ntok || (ka + nt >= all && (sa & 0x7f) == 0x7f)) sa = 0;
        if (kb + nt >= ntok || (kb + nt >= all && (sb & 0x7f) == 0x7f)) sb = 0;
      }
      s2[j] = e4m3x2_to_f16x2((uint16_t)(sa | sb << 8));
    }
#pragma unroll
    for (int wi = 0; wi < 2; ++wi) {
      uint32_t b[2][8];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        pair_values(wi ? xa[j].y : xa[j].x, wi ? xb[j].y : xb[j].x, s2[j], b[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 0; i < MT; ++i) mma_f16(st.acc[i][8 * wi + e], pa[i][kk], b[0][e], b[1][e]);
    }
  }
  if (EDGE) {
    // NaN scales among the keys that only later tokens see
    for (int u = max(all, 0); u < min(ntok, kTileTokens); ++u) {
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

// A CTA is TEAMS independent teams, each with its own range of units, ring and
// loader warp: RG groups of four consumer warps with MT row tiles of 16 each.
// Registers move from the loaders' warpgroup to the consumers (setmaxnreg; the
// shares add up to what the launch gets).
template <int MT, int RG>
struct Shape {
  static constexpr int kRows = 16 * MT * RG;
  static constexpr int kTeams = kRows == 16 ? 3 : (kRows == 32 ? 2 : 1);
  static constexpr int kTeamWarps = kTileWarps * RG;
  static constexpr int kConsumerThreads = kTeamWarps * 32;        // of a team
  static constexpr int kThreads = kTeams * kConsumerThreads + 128;
  // 512 threads x 128 = 384 x 160 + 128 x 32; 384 x 168 = 256 x 224 + 128 x 56
  static constexpr int kConsumerRegs = kRows == 16 ? 160 : 224;
  static constexpr int kLoaderRegs = kRows == 16 ? 32 : 56;
  static constexpr int kQBytes = MT * RG * 4096;
  static constexpr int kOBytes = kTileWarps * kRows * 64 * 4;
  static constexpr int kStages = kRows == 16 ? 5 : (kRows == 32 ? 6 : 12);
  static constexpr int kTeamSmem = kStages * kPageBytes + kQBytes + kOBytes;
  static constexpr int kSmem = kTeams * kTeamSmem;
};

template <int MT, int RG>
struct TeamShared {
  using S = Shape<MT, RG>;
  float red_m[kTileWarps][S::kRows], red_l[kTileWarps][S::kRows];
  uint64_t full_bar[S::kStages], empty_bar[S::kStages];
  int usable[S::kStages];                      // K slots: 0 = the plan flagged the page
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int MT, int RG>
__global__ void __launch_bounds__(Shape<MT, RG>::kThreads, 1)
dense_decode_kernel(WsView ws, DenseArgs a) {
  using S = Shape<MT, RG>;
  constexpr int kRows = S::kRows, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) TeamShared<MT, RG> shared[S::kTeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kConsumerWarps = S::kTeams * S::kTeamWarps;
  const bool loader = warp >= kConsumerWarps;
  const int team = loader ? warp - kConsumerWarps : warp / S::kTeamWarps;
  if (tid < S::kTeams) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&shared[tid].full_bar[i], 1);
      mbar_init(&shared[tid].empty_bar[i], S::kTeamWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const int vid = team * (int)gridDim.x + (int)blockIdx.x;        // neighbours on other SMs
  const int teams = S::kTeams * (int)gridDim.x;
  uint8_t* ring = smem + (loader && team >= S::kTeams ? 0 : team) * S::kTeamSmem;
  uint4* qfrag = reinterpret_cast<uint4*>(ring + kStages * kPageBytes);
  float* obuf = reinterpret_cast<float*>(ring + kStages * kPageBytes + S::kQBytes);
  Walk wk;
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++stage == kStages) { stage = 0; phase ^= 1u; }
  };

  if (loader) {
    // ---------------------------------------------------------------- loader
    // The pages of a segment 32 at a time (a lane each), one bulk copy per
    // K and V slot; of the last page only the rows that exist.
    regs_down<S::kLoaderRegs>();
    if (team >= S::kTeams || !wk.open(ws, a.max_batch, a.Hkv, vid, teams, lane)) return;
    TeamShared<MT, RG>& sh = shared[team];
    int arms = 0;
    while (wk.next(ws, a.Hkv)) {
      if (wk.nq > a.q_len) continue;
      const int32_t* bt = ws.block_table + (int64_t)wk.r * a.max_blocks;
      int ahead = wk.j0 + lane < wk.j1 ? bt[wk.j0 + lane] : -1;
      for (int jb = wk.j0; jb < wk.j1; jb += 32) {
        const int mine = ahead;
        ahead = jb + 32 + lane < wk.j1 ? bt[jb + 32 + lane] : -1;
        for (int j = jb; j < min(jb + 32, wk.j1); ++j) {
          const int page = __shfl_sync(0xffffffffu, mine, j - jb);
          if (lane == 0) {
            const int rows = min(kBlock, wk.L - j * kBlock);
            const uint32_t bytes = (uint32_t)((rows + 1) & ~1) * kFp4Row;   // a multiple of 16
            const int64_t slot = ((int64_t)page * a.Hkv + wk.h) * 2;
            mbar_wait(&sh.empty_bar[stage], phase ^ 1u, ws.hdr);
            sh.usable[stage] = page >= 0;
            if (page < 0) {
              mbar_arrive(&sh.full_bar[stage]);
              ++arms;
              advance();
            } else {
              mbar_arrive_expect_tx(&sh.full_bar[stage], bytes);
              bulk_load(ring + stage * kPageBytes, a.k_pool + slot * kPageBytes, bytes,
                        &sh.full_bar[stage]);
              advance();
              mbar_wait(&sh.empty_bar[stage], phase ^ 1u, ws.hdr);
              mbar_arrive_expect_tx(&sh.full_bar[stage], bytes);
              bulk_load(ring + stage * kPageBytes, a.v_pool + (slot + 1) * kPageBytes, bytes,
                        &sh.full_bar[stage]);
              arms += 2;
              advance();
            }
          }
        }
      }
    }
    // Normally the consumers wait for every copy issued here.  After a wait
    // gave up they may not have: let the copies in flight land.
    if (lane == 0 && (*reinterpret_cast<volatile int*>(&ws.hdr->err) & MSA_DEVERR_TIMEOUT))
      for (int i = 0; i < kStages && i < arms; ++i)
        mbar_drain(&sh.full_bar[i], (uint32_t)(((arms - 1 - i) / kStages) & 1));
    return;
  }

  // -------------------------------------------------------------- consumers
  regs_up<S::kConsumerRegs>();
  if (!wk.open(ws, a.max_batch, a.Hkv, vid, teams, lane)) return;
  TeamShared<MT, RG>& sh = shared[team];
  const int tw = warp - team * S::kTeamWarps, ttid = tw * 32 + lane;   // within the team
  const int rg = tw / kTileWarps, kw = tw % kTileWarps;
  const int g = lane >> 2, c = lane & 3;
  const uint4* qf = qfrag + rg * MT * 8 * 32;
  auto sync = [&]() { named_bar_sync(1 + team, S::kConsumerThreads); };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty_bar[stage]);
    advance();
  };
  while (wk.next(ws, a.Hkv)) {
    if (wk.nq > a.q_len) {                     // more tokens than the config's
      if (ttid == 0) set_error(ws.hdr, MSA_DEVERR_SEQ_LEN);
      continue;
    }
    const int rows = wk.nq * a.G;
    // ---- the rows' A fragments: k-step 2 w + s of lane (g, c) takes dims
    // 16 c + 64 (w / 2) + 8 (w % 2) + 4 s + 0..3
    bool ovf = false;
    for (int x = tw; x < MT * RG * 8; x += S::kTeamWarps) {
      const int ks = x & 7, w = ks >> 1;
      const int dim = 16 * c + 64 * (w >> 1) + 8 * (w & 1) + 4 * (ks & 1);
      uint32_t f[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (x >> 3) * 16 + g + 8 * k;
        uint2 v = make_uint2(0u, 0u);
        if (row < rows)
          v = *reinterpret_cast<const uint2*>(
              a.q +
              ((int64_t)(wk.qs + row / a.G) * a.Hq + wk.h * a.G + row % a.G) * kHeadDim + dim);
        f[k] = bf16x2_to_f16x2(v.x);
        f[k + 2] = bf16x2_to_f16x2(v.y);
        ovf |= f16x2_has_inf(f[k]) | f16x2_has_inf(f[k + 2]);
      }
      qfrag[x * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
    }
    if (__any_sync(0xffffffffu, ovf) && lane == 0) set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
    sync();

    State<MT> st;
    int seen[MT][2];                           // keys of the request each row sees
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        st.acc[i][e][0] = st.acc[i][e][1] = st.acc[i][e][2] = st.acc[i][e][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        st.m[i][k] = -INFINITY;
        st.l[i][k] = 0ull;
        const int row = (rg * MT + i) * 16 + g + 8 * k;
        seen[i][k] = wk.L - wk.nq + min(row / a.G, max(wk.nq - 1, 0)) + 1;
      }
    }
    for (int j = wk.j0; j < wk.j1; ++j) {
      mbar_wait(&sh.full_bar[stage], phase, ws.hdr);
      if (!sh.usable[stage]) {
        release();
        continue;
      }
      const int base = j * kBlock + kw * kTileTokens;   // this warp's first key
      const int ntok = wk.L - base;                     // its keys that exist
      const int all = ntok - wk.nq + 1;                 // and that every row sees
      int lim[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) lim[i][k] = seen[i][k] - base;
      float sc[MT][4][4];
      uint32_t pa[MT][2][4];
      const uint8_t* tile = ring + kw * kTileTokens * kFp4Row;
      if (ntok > 0) scores<MT>(sc, qf, tile + stage * kPageBytes, lane);
      release();
      if (all >= kTileTokens)
        softmax_step<MT, false>(st, sc, pa, a.scale_log2, lane, lim);
      else if (ntok > 0)
        softmax_step<MT, true>(st, sc, pa, a.scale_log2, lane, lim);
      mbar_wait(&sh.full_bar[stage], phase, ws.hdr);
      if (all >= kTileTokens)
        values<MT, false>(st, pa, tile + stage * kPageBytes, lane, lim, ntok, all);
      else if (ntok > 0)
        values<MT, true>(st, pa, tile + stage * kPageBytes, lane, lim, ntok, all);
      release();
    }

    // ---- merge the four warps of each row group
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        f2_split(st.l[i][k], x, y);
        x += y;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c == 0) {
          const int row = (rg * MT + i) * 16 + g + 8 * k;
          sh.red_m[kw][row] = st.m[i][k];
          sh.red_l[kw][row] = x;
        }
      }
    sync();
    float f[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = (rg * MT + i) * 16 + g + 8 * k;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) M = fmaxf(M, sh.red_m[w][row]);
        f[i][k] = M == -INFINITY ? 1.f : ex2_approx(st.m[i][k] - M);
      }
    const int slot = 2 * vid + (wk.starts ? 1 : 0);
#pragma unroll
    for (int p = 0; p < 2; ++p) {              // dims 32 c + 16 half + 8 p + 0..7
      if (p) sync();
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
      sync();
      for (int x = ttid; x < kRows * 8; x += S::kConsumerThreads) {
        const int row = x >> 3, part = x & 7;
        if (row >= rows) continue;
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) M = fmaxf(M, sh.red_m[w][row]);
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w)
          sum += sh.red_l[w][row] * (M == -INFINITY ? 1.f : ex2_approx(sh.red_m[w][row] - M));
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
        if (wk.whole) {
          const int64_t hq =
              (int64_t)(wk.qs + row / a.G) * a.Hq + wk.h * a.G + row % a.G;
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
    sync();
  }
}

// Merges the partials of the (request, head) groups that lie in several teams'
// ranges, in team order: block (x, y) takes the group that starts in team x's
// range and ends behind it, and rows y * kMergeRows .. of it, four warps a
// row.  Tokens without a valid request get out = 0, lse = -inf.
constexpr int kMergeRows = 2;
__global__ void __launch_bounds__(kMergeRows * 128)
dense_merge_kernel(WsView ws, DenseArgs a, int teams) {
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
  const int n = (int)min((int64_t)teams, U);
  const int c0 = blockIdx.x;
  if (c0 >= n) return;
  const int64_t lo = range_of(U, c0, n), hi = range_of(U, c0 + 1, n);
  const int r = request_of(ws.req_cu_nb, ws.req_cu_nb[min(lane, a.max_batch)], batch, a.Hkv,
                           hi - 1, lane);
  const int nb = ws.req_nb[r], qs = ws.req_qstart[r], nq = ws.req_qstart[r + 1] - qs;
  const int64_t first = (int64_t)ws.req_cu_nb[r] * a.Hkv;
  const int h = (int)((hi - 1 - first) / nb);
  const int64_t ga = first + (int64_t)h * nb, gb = ga + nb;
  if (ga < lo || gb <= hi || nq > a.q_len) return;           // block-uniform
  const int c1 = team_of(U, gb - 1, n), np = c1 - c0 + 1;
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
  using S = Shape<MT, RG>;
  static std::atomic<bool> ready[64];          // shared-memory limit raised, per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MSA_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dense_decode_kernel<MT, RG>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem) != cudaSuccess)
      return MSA_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  int64_t grid = sm_count();                   // one CTA an SM
  if (grid > kTeamsMax / S::kTeams) grid = kTeamsMax / S::kTeams;
  if (grid > units) grid = units;
  if (grid <= 0) return MSA_ERR_CUDA;
  const int teams = (int)grid * S::kTeams;
  msa_status st = launch_pdl(dense_decode_kernel<MT, RG>, dim3((unsigned)grid),
                             dim3(S::kThreads), S::kSmem, s, v, a);
  if (st != MSA_OK) return st;
  return launch_pdl(dense_merge_kernel,
                    dim3((unsigned)teams, (unsigned)((a.rows + kMergeRows - 1) / kMergeRows)),
                    dim3(kMergeRows * 128), 0, s, v, a, teams);
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
  return align_up(2 * (size_t)kTeamsMax * rows * kHeadDim * 4) +
         align_up(2 * (size_t)kTeamsMax * rows * 8);
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
  a.max_batch = cfg->max_batch;
  a.rows = a.G * a.q_len;
  a.scale_log2 = cfg->softmax_scale * cfg->k_scale * kLog2e;
  a.v_scale = cfg->v_scale;
  a.q = (const __nv_bfloat16*)q;
  a.k_pool = (const uint8_t*)k_pages;
  a.v_pool = (const uint8_t*)v_pages;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.o_part = (float*)scratch;
  a.ml_part = (float2*)((char*)scratch + align_up(2 * (size_t)kTeamsMax * a.rows * kHeadDim * 4));
  const WsView v = view_of(*cfg, ws);
  const int64_t units = (int64_t)cfg->max_batch * cfg->max_blocks_per_req * a.Hkv;
  cudaStream_t s = (cudaStream_t)stream;
  if (a.rows <= 16) return launch_dense<1, 1>(v, a, units, s);
  if (a.rows <= 32) return launch_dense<2, 1>(v, a, units, s);
  return launch_dense<2, 2>(v, a, units, s);
}
