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
// exact fp16 operands.  So are bf16 queries of 2^-14 .. 65504; larger ones are
// flagged (MSA_DEVERR_FP16_RANGE), smaller ones keep the bits that fp16's
// subnormals have, an error of up to 2^-25 absolute.  Products accumulate in
// fp32.  The probabilities are rounded to fp16 for P V (2^-11 relative, below
// the bf16 rounding of the output); they are carried as 2^(s' - m + 7) so that
// fp16's normal range reaches 2^-21 below the running maximum (smaller ones are
// off by up to 2^-25, 2^-32 of the sum).  Their sum is taken before that
// rounding.  m is kept as an unscaled score and the scale applied to the
// difference, which is exact near the maximum: scores past 2^24, where a step of
// fp32 is more than 7, keep their weights too.  m follows the row's maximum only
// when a score is 2^8 above it in the exponent, which the difference decides as
// well: 2^15 is the largest probability.
//
// Work split.  One unit of work is a 128-key page of one (request, KV head).
// The step's units, request by request and head by head, are cut into equal
// contiguous ranges, one per team of warps, whatever the lengths are; a
// (request, head) whose units lie in several ranges leaves one partial per team
// in the scratch, merged in team order by the second kernel.  All G * q_len
// query rows of a head share each read of a key.
//
// Layout.  A thread dequantises one key row (its TMEM lane) and four value dims
// of 32 keys (V transposed: 16 lanes x 256 bits is the fragment in which a
// thread's pairs of neighbouring keys go out); both are the A operands of
//     S^T = K Q^T (128 keys x rows)   and   O^T += V^T P (128 dims x rows),
// so that N is the number of query rows and no MMA row is padding.  S^T comes
// back in the same fragment, a thread holding 8 keys of 2 rows in 8; stmatrix
// transposes the probabilities into the B operand.  K passes through TMEM in
// two halves, in turns with V's: 128 columns a team, four teams an SM.
//
// What bounds it.  32 requests of 8k-32k tokens, 64 + 8 heads (754 MB): 139 us,
// 5.4 TB/s, 0.80 of the measured copy bandwidth; a page takes an SM about 1000
// cycles, of them 655 issue slots a scheduler (2620 warp instructions, 1024 of
// them the conversions and scalings of its 32768 codes), the rest waits of a
// tile's chain that four teams do not cover.  The same dequantisation in front
// of mma.sync took 192 us: an mma.sync holds its scheduler for about 8 cycles,
// 64 of them a page and warp.  16 requests of 32772 tokens with 4 new ones each
// (32 rows): 149 us, 4.1 TB/s, against 295 us by mma.sync.  Two requests of
// 1.5k tokens, one head: 8 us, the chain of one tile and two launches.
#include <atomic>
#include <cfloat>

#include "tcgen05.cuh"

namespace msa {
namespace {

constexpr int kMaxRows = 64;                   // query rows (tokens x group) of a KV head
constexpr int kTeamsMax = 640;                 // partial slots: two per team
constexpr int kPageBytes = kBlock * kFp4Row;   // one K or V slot, 9216 bytes
constexpr float kBias = 7.f;                   // exponent offset of the probabilities
constexpr float kSlack = 8.f;                  // 2^(kBias + kSlack) is below fp16's largest

struct DenseArgs {
  int Hkv, Hq, G, q_len, max_blocks, max_batch, rows;   // rows = G * q_len
  int teams;                                   // of the grid
  uint32_t g_magic;                            // row / G = row * g_magic >> 16
  float scale_log2, v_scale, slack;            // slack: kSlack in unscaled scores
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;                               // [2 * teams][rows][128]
  float2* ml_part;                             // [2 * teams][rows] (m, sum)
  int4* split;                                 // [teams] the split group that starts in the
                                               // team's range: (partials, first token, head,
                                               // tokens); 0 partials = none

  __device__ __forceinline__ int token_of(int row) const { return (int)(row * g_magic >> 16); }
  // row n of head h of a request whose tokens start at qs, as a row of q and out
  __device__ __forceinline__ int64_t q_row(int qs, int h, int n) const {
    const int t = token_of(n);
    return (int64_t)(qs + t) * Hq + h * G + n - t * G;
  }
};

// U units in n contiguous ranges, the first U % n of them one unit longer.
struct Partition {
  uint32_t q, rem;
  __device__ __forceinline__ Partition(uint32_t U, uint32_t n) : q(U / n), rem(U - U / n * n) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const {
    const uint32_t longer = rem * (q + 1);
    return u < longer ? u / (q + 1) : rem + (u - longer) / q;
  }
};

// The request that holds unit u: the last r with cu[r] * Hkv <= u (requests
// without blocks hold none).  One warp: up to 128 requests from `first`, this
// lane's cu[4 lane .. 4 lane + 3]; more by 32 probes at a time.
__device__ __forceinline__ int request_of(const int32_t* cu, const int4& first, int batch,
                                          uint32_t Hkv, uint32_t u, int lane) {
  if (batch <= 128) {
    const int at[4] = {first.x, first.y, first.z, first.w};
    int below = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) below += 4 * lane + i < batch && (uint32_t)at[i] * Hkv <= u;
    return __reduce_add_sync(0xffffffffu, below) - 1;
  }
  int lo = 0, n = batch;                       // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool below = i < lo + n && (uint32_t)cu[i] * Hkv <= u;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));   // lane 0 is always below
    const int end = lo + n;
    lo += k * step;
    n = min(step, end - lo);
  }
  return lo;
}

// A team's walk over its range: one segment per (request, KV head) it meets.
struct Walk {
  uint32_t u, end;             // next unit, end of the range
  int r;                       // request of unit u
  // the current segment
  int h, j0, j1, nq, qs, L;
  uint32_t last;               // its group's last unit
  int page;                    // kPages: this lane's page, of block j0 + lane
  bool starts, whole;          // it starts its group; it is all of its group

  // The range of team vid; false if it has none.  One warp, all lanes alike.
  __device__ __forceinline__ bool open(const WsView& ws, const DenseArgs& a, int vid, int teams,
                                       int lane) {
    // the region is padded to 256 bytes: the last int4 of the list is whole
    const int4 first = reinterpret_cast<const int4*>(ws.req_cu_nb)[min(lane, a.max_batch / 4)];
    const int batch = ws.hdr->batch;
    const uint32_t U = (uint32_t)ws.hdr->total_blocks * a.Hkv;
    const uint32_t n = min((uint32_t)teams, U);
    if ((uint32_t)vid >= n) return false;
    const Partition p(U, n);
    u = p.start(vid);
    end = p.start(vid + 1);
    r = request_of(ws.req_cu_nb, first, batch, a.Hkv, u, lane);
    return true;
  }
  // The next segment; false at the end of the range.  kPages: with its first 32
  // pages (loaded beside the rest, the request alone being known).
  template <bool kPages = false>
  __device__ __forceinline__ bool next(const WsView& ws, const DenseArgs& a, int lane = 0) {
    if (u >= end) return false;
    const uint32_t Hkv = a.Hkv;
    uint32_t cu0 = ws.req_cu_nb[r], cu1 = ws.req_cu_nb[r + 1];   // u is before the last one's end
    while (cu1 * Hkv <= u) {
      ++r;
      cu0 = cu1;
      cu1 = ws.req_cu_nb[r + 1];
    }
    qs = ws.req_qstart[r];
    nq = ws.req_qstart[r + 1] - qs;
    L = ws.req_seq_len[r];
    const uint32_t nb = cu1 - cu0;
    h = (int)((u - cu0 * Hkv) / nb);
    const uint32_t ga = cu0 * Hkv + h * nb;                 // the group's units: [ga, ga + nb)
    last = ga + nb - 1;
    j0 = (int)(u - ga);
    j1 = (int)(min(ga + nb, end) - ga);
    starts = j0 == 0;
    whole = starts && j1 == (int)nb;
    u = ga + j1;
    if (kPages)
      page = j0 + lane < j1 ? ws.block_table[(int64_t)r * a.max_blocks + j0 + lane] : -1;
    return true;
  }
};

// ---------------------------------------------------------------- TMEM moves
// 16 lanes x 256 bits a repetition: thread (g, c) = (lane / 4, lane % 4) holds,
// per 8 columns, columns 2c, 2c + 1 of lane g (registers 0, 1) and of lane
// g + 8 (registers 2, 3).
template <int NG>
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[4 * NG]) {
  static_assert(NG == 1 || NG == 2 || NG == 4 || NG == 8, "repetitions");
  if constexpr (NG == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (NG == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    if constexpr (NG == 8)
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
          "%13,%14,%15}, [%16];"
          : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
            "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
            "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
          : "r"(taddr + 32)
          : "memory");
  }
}
__device__ __forceinline__ void tmem_st_16x256_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Lane i of the warp's quarter, 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Four 8 x 8 matrices of 16-bit values, transposed on the way: thread (g, c)
// holds row g, columns 2c and 2c + 1 of each; lane 8 i + k gives the address
// where column k of matrix i goes (8 values, 16 bytes).
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                          uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void named_bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
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

// ---------------------------------------------------------------- dequantisation
// K: 64 dims (half 0 or 1) of this thread's key row (72 bytes) -> its TMEM
// lane, 32 columns of two dims.
__device__ __forceinline__ void key_half(const uint8_t* row, uint32_t taddr, int half) {
  const uint32_t s4 = *reinterpret_cast<const uint32_t*>(row + kHeadDim / 2 + 4 * half);
  const uint32_t sp[2] = {e4m3x2_to_f16x2((uint16_t)(s4 & 0xffffu)),
                          e4m3x2_to_f16x2((uint16_t)(s4 >> 16))};
  uint32_t h[32];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint2 x = *reinterpret_cast<const uint2*>(row + 32 * half + 8 * b);
    const __half2 sh2 = *reinterpret_cast<const __half2*>(&sp[b >> 1]);
    const __half2 sc2 = b & 1 ? __high2half2(sh2) : __low2half2(sh2);
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(&sc2);
    uint32_t lo[4], hi[4];
    e2m1x8_to_f16x2(x.x, lo);
    e2m1x8_to_f16x2(x.y, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[8 * b + e] = hmul2_u32(lo[e], sc);
      h[8 * b + 4 + e] = hmul2_u32(hi[e], sc);
    }
  }
  tmem_st32(taddr, h);
}

// V, transposed: this warp's dims 32 w .. 32 w + 31 of 64 keys (half 0 or 1 of
// the tile) -> TMEM lanes 32 w + 8 i + g = dim 32 w + 4 g + i, 32 columns of
// two keys.  The warp's two scale blocks go through `pairs` (64 words): a lane
// converts those of two keys, all read them as (key, key + 1).
// Keys from ntok on do not exist (their rows may hold anything), and a NaN
// scale of a key that not every row sees becomes 0 here: 0 * NaN is not 0 (the
// rows that see it get it back at the end).
__device__ __forceinline__ void value_half(const uint8_t* vt, uint32_t taddr, int half,
                                           uint32_t* pairs, int w, int lane, int ntok, int all) {
  constexpr uint32_t m = 0x0f0f0f0fu;
  const int g = lane >> 2, c = lane & 3;
  const uint8_t* codes = vt + (64 * half + 4 * c) * kFp4Row + 16 * w + 2 * g;
  {
    const int key = 64 * half + 2 * lane;
    const uint8_t* at = vt + key * kFp4Row + kHeadDim / 2 + 2 * w;
    uint32_t s[2] = {*reinterpret_cast<const uint16_t*>(at),
                     *reinterpret_cast<const uint16_t*>(at + kFp4Row)};
    if (all < kBlock) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (key + i >= ntok) s[i] = 0;
        if (key + i >= all) {
          if ((s[i] & 0x7fu) == 0x7fu) s[i] &= 0xff00u;
          if ((s[i] & 0x7f00u) == 0x7f00u) s[i] &= 0xffu;
        }
      }
    }
    const uint32_t h0 = e4m3x2_to_f16x2((uint16_t)s[0]), h1 = e4m3x2_to_f16x2((uint16_t)s[1]);
    pairs[lane] = __byte_perm(h0, h1, 0x5410);
    pairs[32 + lane] = __byte_perm(h0, h1, 0x7632);
    __syncwarp();
  }
  const uint32_t* sp = pairs + (g >> 2) * 32 + 2 * c;
  uint32_t lo[16], hi[16];
#pragma unroll
  for (int qq = 0; qq < 4; ++qq) {             // keys 64 half + 16 qq + 4 c + 0..3
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = *reinterpret_cast<const uint16_t*>(codes + (16 * qq + i) * kFp4Row);
    const uint2 s = *reinterpret_cast<const uint2*>(sp + 8 * qq);
    const uint32_t a = __byte_perm(u[0], u[2], 0x5410), b = __byte_perm(u[1], u[3], 0x5410);
    const uint32_t even = (a & m) | ((b << 4) & ~m), odd = ((a >> 4) & m) | (b & ~m);
    uint32_t e[4], o[4];                       // dims 0, 2 | 1, 3 of keys 0 1, then of 2 3
    e2m1x8_to_f16x2(even, e);
    e2m1x8_to_f16x2(odd, o);
    lo[4 * qq] = hmul2_u32(e[0], s.x);
    lo[4 * qq + 1] = hmul2_u32(e[2], s.y);
    lo[4 * qq + 2] = hmul2_u32(o[0], s.x);
    lo[4 * qq + 3] = hmul2_u32(o[2], s.y);
    hi[4 * qq] = hmul2_u32(e[1], s.x);
    hi[4 * qq + 1] = hmul2_u32(e[3], s.y);
    hi[4 * qq + 2] = hmul2_u32(o[1], s.x);
    hi[4 * qq + 3] = hmul2_u32(o[3], s.y);
  }
  tmem_st_16x256_x4(taddr, lo);
  tmem_st_16x256_x4(taddr + (16u << 16), hi);
}

// The tiles (pages) of a range, one after the other, for a role that walks
// them by itself.
struct Tiles {
  Walk wk;
  int j, seg;                  // block of the current tile, its segment's number
  bool first, last;            // of the segment

  __device__ __forceinline__ bool open(const WsView& ws, const DenseArgs& a, int vid, int teams,
                                       int lane) {
    j = 0;
    seg = -1;
    last = true;
    return wk.open(ws, a, vid, teams, lane);
  }
  // Skips the segments of requests without new tokens, or with more than the
  // config's (the consumers flag those).
  template <bool kPages = false>
  __device__ __forceinline__ bool next(const WsView& ws, const DenseArgs& a, int lane = 0) {
    first = last;
    if (last) {
      do {
        if (!wk.next<kPages>(ws, a, lane)) return false;
      } while (wk.nq > a.q_len || wk.nq == 0);
      ++seg;
      j = wk.j0;
    } else {
      ++j;
    }
    last = j + 1 == wk.j1;
    return true;
  }
};

// A CTA is kTeams independent teams of four consumer warps, each with its own
// range of units, ring, TMEM columns, loader warp and MMA warp.  NG: groups of
// 8 query rows.
template <int NG, int TEAMS>
struct Shape {
  static constexpr int kN = NG < 2 ? 16 : 8 * NG;                 // MMA N
  static constexpr int kTeams = TEAMS;
  static constexpr int kThreads = kTeams * 128 + 256;
  // threads x launch registers = consumers x theirs + 256 x the others':
  // 768 x 80 = 512 x 96 + 256 x 48; 640 x 96 = 384 x 128 + 256 x 48;
  // 512 x 128 = 256 x 200 + 256 x 56
  static constexpr int kConsumerRegs = TEAMS == 4 ? 96 : (TEAMS == 3 ? 128 : 200);
  static constexpr int kMiscRegs = TEAMS >= 3 ? 48 : 56;
  // TMEM columns of a team: K (64 dims) | V | S | O
  static constexpr int kCols = 96 + 2 * kN;
  static constexpr int kFit = (218 * 1024 / kTeams - 3 * kN * kHeadDim * 2) / kPageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kOperand = kN * kHeadDim * 2;              // a Q buffer, and P
  static constexpr int kTeamSmem = 3 * kOperand + kStages * kPageBytes;
  static constexpr int kSmem = kTeams * kTeamSmem;
  static_assert(kTeams * kCols <= 512, "TMEM");
};

// Phase parity of the use number t of buffer t & 1.
__device__ __forceinline__ uint32_t par(int t) { return (uint32_t)(t >> 1) & 1u; }

template <int NG, int TEAMS>
struct TeamShared {
  using S = Shape<NG, TEAMS>;
  float red[4][S::kN];         // per warp: row maxima, row sums
  float alpha[S::kN], ref[S::kN];              // rescaling, final references
  uint32_t pairs[4][64];       // per warp: scales of V (value_half)
  uint64_t full_bar[S::kStages], empty_bar[S::kStages];
  uint64_t q_free[2];          // Q buffer free again
  uint64_t k_ready, k_free;    // a half of K written (two a tile); the first half read
  uint64_t s_ready;            // S written, K read
  uint64_t p_ready, o_ready;   // P and V written; O updated and P and V read
  int usable[S::kStages];      // K slots: 0 = the plan flagged the page
  int tok[S::kN];              // token of each row within the request
  unsigned nan[S::kN];         // value blocks that are NaN for the row
};

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

template <int NG, int TEAMS>
__global__ void __launch_bounds__(Shape<NG, TEAMS>::kThreads, 1)
dense_decode_kernel(WsView ws, DenseArgs a) {
  using S = Shape<NG, TEAMS>;
  constexpr int kN = S::kN, kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) TeamShared<NG, TEAMS> shared[S::kTeams];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);         // uniform
  const int extra = warp - 4 * S::kTeams;      // loaders, then MMA warps
  const int team = extra < 0 ? warp / 4 : (extra < S::kTeams ? extra : extra - S::kTeams);
  const bool keeper = extra == S::kTeams;      // MMA warp 0 keeps the TMEM allocation
  if (tid < S::kTeams) {
    TeamShared<NG, TEAMS>& st = shared[tid];
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&st.full_bar[i], 1);
      mbar_init(&st.empty_bar[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&st.q_free[i], 4);
    }
    mbar_init(&st.k_ready, 4);
    mbar_init(&st.k_free, 1);
    mbar_init(&st.s_ready, 1);
    mbar_init(&st.p_ready, 4);
    mbar_init(&st.o_ready, 1);
    fence_barrier_init();
  }
  if (keeper) {
    // before the wait: kernels of this library that use TMEM let their
    // dependents start only once they hold theirs
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();                 // (as this one does)
  griddep_wait();
  constexpr int kDone = 15;                    // named barrier: every consumer and MMA warp
  constexpr int kDoneCount = S::kTeams * 160;
  if (extra >= 0) regs_down<S::kMiscRegs>();
  if (extra >= 2 * S::kTeams) return;
  TeamShared<NG, TEAMS>& sh = shared[team];
  const int vid = team * (int)gridDim.x + (int)blockIdx.x;        // neighbours on other SMs
  // As an argument it stays in a register, which up to three teams have to spare
  // (32 requests of 16384 tokens, 16 rows: 131.6 us, computed here 135.2; verify
  // of 16 x 32772 149.0 and 151.8); four do not (32 of 8k-32k 142.6 and 139.0).
  const int teams = TEAMS < 4 ? a.teams : TEAMS * (int)gridDim.x;
  uint8_t* qbuf = smem + team * S::kTeamSmem;  // Q x 2 and P: K-major, 128-byte swizzle
  uint8_t* pbuf = qbuf + 2 * S::kOperand;
  uint8_t* ring = pbuf + S::kOperand;

  if (extra >= S::kTeams) {
    // ------------------------------------------------------------------ MMAs
    // The whole warp runs, an elected lane issues: under elect.sync an MMA of
    // 16 columns issues every 9 cycles, under `lane == 0` (its operands then
    // move to uniform registers one by one) every 46.
    constexpr uint32_t idesc = idesc_f16(0, 128, kN);
    const uint64_t dq = kstep_desc(smem_u32(qbuf), 0, kN), dp = kstep_desc(smem_u32(pbuf), 0, kN);
    const uint32_t plo = (uint32_t)dp, hi = (uint32_t)(dq >> 32);
    Tiles tl;
    bool more = tl.open(ws, a, vid, teams, lane) && tl.next(ws, a);
    const uint32_t tk = __shfl_sync(0xffffffffu, tmem_base, 0) + team * S::kCols, tv = tk + 32,
                   ts = tk + 96, to = ts + kN;
    const bool issued = more;
    uint32_t ph = 0;
    for (; more; ph ^= 1u) {
      const uint32_t qlo = (uint32_t)dq + (tl.seg & 1) * (S::kOperand >> 4);
      if (tl.first) {
        // the segment's Q, bf16 -> fp16 rows of the B operand, zero past the last
        const Walk& wk = tl.wk;
        const int nrows = wk.nq * a.G, b = tl.seg & 1;
        if (tl.seg >= 2) mbar_wait(&sh.q_free[b], par(tl.seg - 2), ws.hdr);
        bool ovf = false;
        for (int x = nrows * 16 + lane; x < kN * 16; x += 32)
          *reinterpret_cast<uint4*>(qbuf + b * S::kOperand + kmaj_off(x >> 4, x & 15, kN)) =
              make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
        for (int x = lane; x < nrows * 16; x += 32) {
          const int n = x >> 4, ch = x & 15;
          uint4 v =
              *reinterpret_cast<const uint4*>(a.q + a.q_row(wk.qs, wk.h, n) * kHeadDim + 8 * ch);
          v.x = bf16x2_to_f16x2(v.x);
          v.y = bf16x2_to_f16x2(v.y);
          v.z = bf16x2_to_f16x2(v.z);
          v.w = bf16x2_to_f16x2(v.w);
          ovf |= f16x2_has_inf(v.x) | f16x2_has_inf(v.y) | f16x2_has_inf(v.z) |
                 f16x2_has_inf(v.w);
          *reinterpret_cast<uint4*>(qbuf + b * S::kOperand + kmaj_off(n, ch, kN)) = v;
        }
        if (__any_sync(0xffffffffu, ovf) && lane == 0)
          set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
        fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {   // S^T = K Q^T (128 keys x rows), 64 dims at a time
        mbar_wait(&sh.k_ready, half, ws.hdr);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t b = qlo + half * (kN * 8) + ks * 2;
            if (half == 0 && ks == 0) umma_ts<false>(ts, tk, b, hi, idesc);
            else umma_ts<true>(ts, tk + 8 * ks, b, hi, idesc);
          }
          umma_commit(half ? &sh.s_ready : &sh.k_free);
        }
        __syncwarp();
      }
      mbar_wait(&sh.p_ready, ph, ws.hdr);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {                       // O^T += V^T P (128 dims x rows)
        if (tl.first) umma_ts<false>(to, tv, plo, hi, idesc);
        else umma_ts<true>(to, tv, plo, hi, idesc);
#pragma unroll
        for (int ks = 1; ks < 8; ++ks)
          umma_ts<true>(to, tv + 8 * ks, plo + (ks >> 2) * (kN * 8) + (ks & 3) * 2, hi, idesc);
        umma_commit(&sh.o_ready);
      }
      __syncwarp();
      more = tl.next(ws, a);
    }
    // Normally the consumers have waited for the last MMAs.  After a wait gave
    // up they may not have: let them finish before TMEM goes.
    if (issued && (*reinterpret_cast<volatile int*>(&ws.hdr->err) & MSA_DEVERR_TIMEOUT))
      mbar_drain(&sh.o_ready, ph ^ 1u);
    __syncwarp();
    if (keeper) {
      named_bar_sync(kDone, kDoneCount);
      tc_fence_after();
      tmem_dealloc(tmem_base, 512);
    } else {
      named_bar_arrive(kDone, kDoneCount);
    }
    return;
  }

  if (extra >= 0) {
    // ---------------------------------------------------------------- loader
    // The pages of a segment 32 at a time (a lane each), one bulk copy per
    // K and V slot; of the last page only the rows that exist.
    Tiles tl;
    const bool any = tl.open(ws, a, vid, teams, lane);
    int arms = 0, stage = 0, mine = 0;
    uint32_t phase = 0;
    while (any && tl.next<true>(ws, a, lane)) {
      const Walk& wk = tl.wk;
      const int at = (tl.j - wk.j0) & 31;
      if (tl.first)
        mine = wk.page;
      else if (at == 0)
        mine = tl.j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + tl.j + lane]
                                   : -1;
      const int page = __shfl_sync(0xffffffffu, mine, at);
      const int rows = min(kBlock, wk.L - tl.j * kBlock);
      const uint32_t bytes = (uint32_t)((rows + 1) & ~1) * kFp4Row;       // a multiple of 16
      const int64_t slot = ((int64_t)page * a.Hkv + wk.h) * 2;
      for (int kind = 0; kind < 2; ++kind) {
        mbar_wait(&sh.empty_bar[stage], phase ^ 1u, ws.hdr);
        __syncwarp();
        if (elect_one()) {
          sh.usable[stage] = page >= 0;
          if (page >= 0) {
            mbar_arrive_expect_tx(&sh.full_bar[stage], bytes);
            bulk_load(ring + stage * kPageBytes,
                      (kind ? a.v_pool : a.k_pool) + (slot + kind) * kPageBytes, bytes,
                      &sh.full_bar[stage]);
          } else {
            mbar_arrive(&sh.full_bar[stage]);
          }
        }
        __syncwarp();
        ++arms;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    // tokens of no request, and of requests with more tokens than the config's
    const int T = ws.hdr->num_tokens;
    for (int t = vid; t < T; t += teams) {
      const int r = ws.tok_req[t];
      if (r >= 0 && ws.req_qstart[r + 1] - ws.req_qstart[r] <= a.q_len) continue;
      for (int x = lane; x < a.Hq * (kHeadDim / 8); x += 32)
        reinterpret_cast<uint4*>(a.out + (int64_t)t * a.Hq * kHeadDim)[x] = make_uint4(0, 0, 0, 0);
      for (int x = lane; x < a.Hq; x += 32) a.lse[(int64_t)t * a.Hq + x] = -INFINITY;
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
  // Control flow depends on the plan's data alone (never on what a wait saw),
  // so that the team's named barriers match even after a wait gave up.
  const int w = warp & 3, ttid = tid & 127;    // within the team; ttid = key of a tile
  const int g = lane >> 2, c = lane & 3;
  const int bar = 1 + team;                    // the team's named barrier
  const uint32_t lanes = (uint32_t)(32 * w) << 16;
  int stage = 0;
  uint32_t phase = 0, ph = 0, o_phase = 0;     // ph: of the tile's S
  // this lane's address for the transposed store of P: matrix i = keys 32 w + 8 i ..,
  // column k = row 8 grp + k
  const int pchunk = 4 * w + (lane >> 3);
  const uint32_t paddr = smem_u32(pbuf) + (pchunk >> 3) * kN * 128 + (lane & 7) * 128 +
                         (((pchunk & 7) ^ (lane & 7)) << 4);
  if (8 * NG < kN)                             // P rows that no group fills
    for (int x = ttid; x < S::kOperand / 16; x += 128)
      reinterpret_cast<uint4*>(pbuf)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  auto written = [&](uint64_t* bar_) {         // this warp's TMEM stores are done
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_);
  };
  auto step = [&]() {
    if (++stage == kStages) { stage = 0; phase ^= 1u; }
  };
  Walk wk;
  const bool any = wk.open(ws, a, vid, teams, lane);
  const uint32_t tm = tmem_base + team * S::kCols + lanes;
  const uint32_t tk = tm, tv = tm + 32, ts = tm + 96, to = ts + kN;
  int4 split = make_int4(0, 0, 0, 0);
  for (int seg = 0; any && wk.next(ws, a);) {
    if (wk.nq > a.q_len || wk.nq == 0) {       // more tokens than the config's, or none
      if (ttid == 0 && wk.nq > 0) set_error(ws.hdr, MSA_DEVERR_SEQ_LEN);
      continue;
    }
    const int rows = wk.nq * a.G;
    if (ttid < kN) {
      sh.tok[ttid] = min(a.token_of(ttid), wk.nq - 1);
      sh.nan[ttid] = 0u;
    }
    named_bar_sync(bar, 128);

    float m[NG][2], l[NG][2];                  // rows 8 i + 2 c + {0, 1}
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
    for (int j = wk.j0; j < wk.j1; ++j) {
      // ---- K and V -> TMEM by halves, in turns: the first half of K is read
      // by its MMAs (S^T = K Q^T) while the first half of V is written
      mbar_wait(&sh.full_bar[stage], phase, ws.hdr);
      const int ntok = sh.usable[stage] ? wk.L - j * kBlock : 0;   // keys that exist
      const int all = ntok - wk.nq + 1;                            // and that every row sees
      const int kst = stage;
      const uint8_t* kt = ring + kst * kPageBytes + ttid * kFp4Row;
      step();
      key_half(kt, tk, 0);
      written(&sh.k_ready);
      if (j > wk.j0) {                         // the last P V has read V
        mbar_wait(&sh.o_ready, o_phase, ws.hdr);
        o_phase ^= 1u;
        tc_fence_after();
      }
      mbar_wait(&sh.full_bar[stage], phase, ws.hdr);
      const uint8_t* vt = ring + stage * kPageBytes;
      value_half(vt, tv, 0, sh.pairs[w], w, lane, ntok, all);
      mbar_wait(&sh.k_free, ph, ws.hdr);
      tc_fence_after();
      key_half(kt, tk, 1);
      written(&sh.k_ready);
      if (lane == 0) mbar_arrive(&sh.empty_bar[kst]);
      value_half(vt, tv + 32, 1, sh.pairs[w], w, lane, ntok, all);
      if (all < kBlock) {
        if (ttid >= all && ttid < ntok) {      // NaN scales that only later tokens see
          unsigned bad = 0;
          for (int b = 0; b < 8; ++b)
            bad |= (vt[ttid * kFp4Row + kHeadDim / 2 + b] & 0x7f) == 0x7f ? 1u << b : 0u;
          if (bad)
            for (int n = 0; n < rows; ++n)
              if (ttid < all + sh.tok[n]) atomicOr(&sh.nan[n], bad);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty_bar[stage]);
      step();
      // ---- softmax of S^T: 8 keys (16 hf + g, + 8) of rows 8 i + 2 c + {0, 1}
      mbar_wait(&sh.s_ready, ph, ws.hdr);
      ph ^= 1u;
      tc_fence_after();
      uint32_t x[2][4 * NG];
      tmem_ld_16x256<NG>(ts, x[0]);
      tmem_ld_16x256<NG>(ts + (16u << 16), x[1]);
      tmem_ld_wait();
      if (all < kBlock) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 4 * NG; ++e) {
            const int key = 32 * w + 16 * hf + g + 8 * ((e >> 1) & 1);
            const int lim = min(ntok, all + sh.tok[8 * (e >> 2) + 2 * c + (e & 1)]);
            if (key >= lim) x[hf][e] = 0xff800000u;
          }
      }
      auto xf = [&](int hf, int i, int e) { return __uint_as_float(x[hf][4 * i + e]); };
      bool move = false;
      float mx[NG][2];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[i][k] = fmaxf(fmax3(xf(0, i, k), xf(0, i, k + 2), xf(1, i, k)), xf(1, i, k + 2));
          // the difference, exact near m (m + slack is rounded by up to half a step
          // of fp32: for |m| from 2^28 on, at a scale of 0.75 * 128^-0.5, that lets
          // P pass fp16's largest value); -inf - -inf is NaN: no move
          move |= mx[i][k] - m[i][k] > a.slack;
        }
      if (named_bar_any(bar, 128, move)) {
        // new references: the row maxima over the team's keys
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1)
              mx[i][k] = fmaxf(mx[i][k], __shfl_xor_sync(0xffffffffu, mx[i][k], o));
            if (g == 0) sh.red[w][8 * i + 2 * c + k] = mx[i][k];
          }
        named_bar_sync(bar, 128);
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = 8 * i + 2 * c + k;
            const float mn = fmaxf(fmax3(m[i][k], sh.red[0][n], sh.red[1][n]),
                                   fmaxf(sh.red[2][n], sh.red[3][n]));
            const float alpha =
                mn == -INFINITY ? 1.f : ex2_approx((m[i][k] - mn) * a.scale_log2);
            m[i][k] = mn;
            l[i][k] *= alpha;
            if (w == 0 && g == 0) sh.alpha[n] = alpha;
          }
        named_bar_sync(bar, 128);
        if (j > wk.j0) {
#pragma unroll
          for (int n0 = 0; n0 < 8 * NG; n0 += 16) {
            uint32_t o[16];
            tmem_ld16(to + n0, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (n0 + e < 8 * NG)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * sh.alpha[n0 + e]);
            tmem_st16(to + n0, o);
          }
          tmem_st_wait();
        }
      }
      // ---- P = 2^((s - m) scale + bias) as the B operand [row][key]
      const uint64_t sl = f2(a.scale_log2, a.scale_log2), bias = f2(kBias, kBias);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint64_t ref = f2(m[i][0] == -INFINITY ? 0.f : -m[i][0],
                                m[i][1] == -INFINITY ? 0.f : -m[i][1]);
        uint64_t sum = f2(l[i][0], l[i][1]);
        uint32_t p[4];
#pragma unroll
        for (int o = 0; o < 4; ++o) {          // keys 8 o + g
          float p0, p1;
          const uint64_t s2 =
              f2u(x[o >> 1][4 * i + 2 * (o & 1)], x[o >> 1][4 * i + 2 * (o & 1) + 1]);
          f2_split(fma_f2(add_f2(s2, ref), sl, bias), p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          sum = add_f2(sum, f2(p0, p1));
          p[o] = pack_f16(p0, p1);
        }
        f2_split(sum, l[i][0], l[i][1]);
        stsm_x4_t(paddr + i * 1024, p[0], p[1], p[2], p[3]);
      }
      fence_proxy_async_smem();
      written(&sh.p_ready);
    }

    // ---- the segment's result: whole rows, or a partial
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1)
          l[i][k] += __shfl_xor_sync(0xffffffffu, l[i][k], o);
        const int n = 8 * i + 2 * c + k;
        if (g == 0) sh.red[w][n] = l[i][k];
        if (w == 0 && g == 0) sh.ref[n] = m[i][k];
      }
    mbar_wait(&sh.o_ready, o_phase, ws.hdr);
    o_phase ^= 1u;
    tc_fence_after();
    named_bar_sync(bar, 128);
    // O^T -> [row][dim] in the segment's Q buffer and in P (S and P V are done)
    const int dim = 32 * w + 4 * (lane & 7) + (lane >> 3);        // of this thread's TMEM lane
    uint8_t* qcur = qbuf + (seg & 1) * S::kOperand;
    auto o_row = [&](int n) {
      return reinterpret_cast<float*>((n < kN / 2 ? qcur : pbuf) + (n & (kN / 2 - 1)) * 512);
    };
#pragma unroll
    for (int n0 = 0; n0 < 8 * NG; n0 += 16) {
      uint32_t o[16];
      tmem_ld16(to + n0, o);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (n0 + e < 8 * NG) o_row(n0 + e)[dim] = __uint_as_float(o[e]);
    }
    tc_fence_before();
    named_bar_sync(bar, 128);
    const int64_t slot = 2 * vid + (wk.starts ? 1 : 0);
#pragma unroll 1
    for (int x = ttid; x < rows * 16; x += 128) {
      const int n = x >> 4, part = x & 15;     // 8 dims, half a value block
      const float sum = sh.red[0][n] + sh.red[1][n] + sh.red[2][n] + sh.red[3][n];
      const float4* src = reinterpret_cast<const float4*>(o_row(n) + 8 * part);
      float4 y0 = src[0], y1 = src[1];
      if ((sh.nan[n] >> (part >> 1)) & 1u) y0 = y1 = make_float4(NAN, NAN, NAN, NAN);
      if (wk.whole) {
        const int64_t row = a.q_row(wk.qs, wk.h, n);
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
        *reinterpret_cast<uint4*>(a.out + row * kHeadDim + 8 * part) =
            make_uint4(pack_bf16(y0.x * inv, y0.y * inv), pack_bf16(y0.z * inv, y0.w * inv),
                       pack_bf16(y1.x * inv, y1.y * inv), pack_bf16(y1.z * inv, y1.w * inv));
        if (part == 0)
          a.lse[row] =
              sum == 0.f ? -INFINITY : (sh.ref[n] * a.scale_log2 + log2f(sum) - kBias) * kLn2;
      } else {
        float4* dst =
            reinterpret_cast<float4*>(a.o_part + (slot * a.rows + n) * kHeadDim + 8 * part);
        dst[0] = y0;
        dst[1] = y1;
        if (part == 0) a.ml_part[slot * a.rows + n] = make_float2(sh.ref[n], sum);
      }
    }
    if (wk.starts && !wk.whole) {              // the range ends inside this group
      const uint32_t U = (uint32_t)ws.hdr->total_blocks * a.Hkv;
      const int c1 = (int)Partition(U, min((uint32_t)teams, U)).owner(wk.last);
      split = make_int4(c1 - vid + 1, wk.qs, wk.h, wk.nq);
    }
    if (8 * NG == kN)                          // P rows are refilled; Q goes to the MMA warp
      fence_proxy_async_smem();
    named_bar_sync(bar, 128);                  // red, ref, tok, nan and P are free again
    if (lane == 0) mbar_arrive(&sh.q_free[seg & 1]);
    ++seg;
  }
  if (ttid == 0) a.split[vid] = split;
  tc_fence_before();
  named_bar_arrive(kDone, kDoneCount);
}

// Merges the partials of the (request, head) groups that lie in several teams'
// ranges, in team order.  Every block lists the split groups in order, then
// takes its share of (group, two rows), four warps a row.  Rows of more than
// kMany partials then get a whole block each: one request of 131071 tokens, 76
// partials a row, 39.5 us in all against 41.6 without; from 9 partials on it
// costs time instead, 61 requests of up to 6001 tokens 20.8 us against 18.0.
constexpr int kMergeWarps = 8, kMergeThreads = kMergeWarps * 32;
constexpr int kMergeRows = 2, kRowWarps = kMergeWarps / kMergeRows;
constexpr int kMergeChunks = (kTeamsMax + kMergeThreads - 1) / kMergeThreads;
constexpr int kMany = 32;
__global__ void __launch_bounds__(kMergeThreads) dense_merge_kernel(DenseArgs a, int teams) {
  __shared__ int4 list[kTeamsMax];
  __shared__ int owner[kTeamsMax];
  __shared__ int counts[kMergeChunks * kMergeWarps], many;
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float part_l[kMergeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  int4 rec[kMergeChunks];
  unsigned starts[kMergeChunks];
#pragma unroll
  for (int k = 0; k < kMergeChunks; ++k) {          // all loads in flight together
    const int c = k * kMergeThreads + tid;
    rec[k] = c < teams ? a.split[c] : make_int4(0, 0, 0, 0);
  }
  if (tid == 0) many = 0;
#pragma unroll
  for (int k = 0; k < kMergeChunks; ++k) {
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
      if (rec[k].x > kMany) many = 1;
    }
  }
  __syncthreads();
  // one row by `warps` warps of the block, this one the w-th, from warp w0 on
  auto merge_row = [&](const int4& rec, int64_t c0, int row, int w, int warps, int w0) {
    const int np = rec.x;
    const bool on = row < rec.w * a.G;
    // partial i: the second slot of c0, the first of c0 + i
    auto at = [&](int i) { return (2 * (c0 + i) + (i == 0 ? 1 : 0)) * a.rows + row; };
    float M = -INFINITY;
    if (on)
      for (int i = lane; i < np; i += 32) M = fmaxf(M, a.ml_part[at(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (on) {
#pragma unroll 8
      for (int i = w; i < np; i += warps) {
        const float2 ml = a.ml_part[at(i)];
        const float4 v = *reinterpret_cast<const float4*>(a.o_part + at(i) * kHeadDim + 4 * lane);
        const float f = M == -INFINITY ? 1.f : ex2_approx((ml.x - M) * a.scale_log2);
        l = fmaf(f, ml.y, l);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
      }
    }
    part[warp][lane] = o;
    if (lane == 0) part_l[warp] = l;
    __syncthreads();
    if (on && w == 0) {
      for (int i = 1; i < warps; ++i) {
        const float4 v = part[w0 + i][lane];
        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        l += part_l[w0 + i];
      }
      const int64_t hq = a.q_row(rec.y, rec.z, row);
      const float inv = l == 0.f ? 0.f : a.v_scale / l;
      reinterpret_cast<uint2*>(a.out + hq * kHeadDim)[lane] =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (lane == 0)
        a.lse[hq] = l == 0.f ? -INFINITY : (M * a.scale_log2 + log2f(l) - kBias) * kLn2;
    }
    __syncthreads();
  };
  const int chunks = (a.rows + kMergeRows - 1) / kMergeRows;
  for (int item = blockIdx.x; item < n * chunks; item += gridDim.x) {
    const int gi = item / chunks;
    if (list[gi].x <= kMany)
      merge_row(list[gi], owner[gi], (item - gi * chunks) * kMergeRows + warp / kRowWarps,
                warp % kRowWarps, kRowWarps, warp / kRowWarps * kRowWarps);
  }
  if (!many) return;
  for (int item = blockIdx.x; item < n * a.rows; item += gridDim.x) {
    const int gi = item / a.rows;
    if (list[gi].x > kMany)
      merge_row(list[gi], owner[gi], item - gi * a.rows, warp, kMergeWarps, 0);
  }
}

template <int NG, int TEAMS>
msa_status launch_dense(const WsView& v, DenseArgs& a, int64_t units, cudaStream_t s) {
  using S = Shape<NG, TEAMS>;
  static std::atomic<bool> ready[64];          // shared-memory limit raised, per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MSA_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dense_decode_kernel<NG, TEAMS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem) != cudaSuccess)
      return MSA_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  const int sms = sm_count();
  int64_t grid = sms;                          // one CTA an SM
  if (grid > kTeamsMax / S::kTeams) grid = kTeamsMax / S::kTeams;
  if (grid <= 0) return MSA_ERR_CUDA;
  if (grid > units) grid = units;
  const int teams = a.teams = (int)grid * S::kTeams;
  msa_status st = launch_pdl(dense_decode_kernel<NG, TEAMS>, dim3((unsigned)grid),
                             dim3(S::kThreads), S::kSmem, s, v, a);
  if (st != MSA_OK) return st;
  int64_t blocks = (int64_t)teams * ((a.rows + kMergeRows - 1) / kMergeRows);
  if (blocks > 4 * sms) blocks = 4 * sms;
  return launch_pdl(dense_merge_kernel, dim3((unsigned)blocks), dim3(kMergeThreads), 0, s, a,
                    teams);
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
         align_up(2 * (size_t)kTeamsMax * rows * 8) + align_up(kTeamsMax * sizeof(int4));
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
      ((uintptr_t)ws & 255) != 0 || ((uintptr_t)scratch & 255) != 0 || ((uintptr_t)lse & 3) != 0)
    return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0 || cfg->max_batch == 0) return MSA_OK;
  DenseArgs a;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.G = a.Hq / a.Hkv;
  a.q_len = cfg->q_len;
  a.max_blocks = cfg->max_blocks_per_req;
  a.max_batch = cfg->max_batch;
  a.rows = a.G * a.q_len;
  a.scale_log2 = cfg->softmax_scale * cfg->k_scale * kLog2e;
  if (!(a.scale_log2 > 0.f && a.scale_log2 < INFINITY)) return MSA_ERR_INVALID_ARG;
  a.slack = fminf(kSlack / a.scale_log2, FLT_MAX);
  a.v_scale = cfg->v_scale;
  a.q = (const __nv_bfloat16*)q;
  a.k_pool = (const uint8_t*)k_pages;
  a.v_pool = (const uint8_t*)v_pages;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.o_part = (float*)scratch;
  a.g_magic = (65536u + a.G - 1) / a.G;        // exact for rows below 128 and G <= 16
  a.ml_part = (float2*)((char*)scratch + align_up(2 * (size_t)kTeamsMax * a.rows * kHeadDim * 4));
  a.split = (int4*)((char*)a.ml_part + align_up(2 * (size_t)kTeamsMax * a.rows * 8));
  const WsView v = view_of(*cfg, ws);
  const int64_t units = (int64_t)cfg->max_batch * cfg->max_blocks_per_req * a.Hkv;
  if (units > 0x7fffffff) return MSA_ERR_UNSUPPORTED;   // units are counted in 32 bits
  cudaStream_t s = (cudaStream_t)stream;
  // Teams an SM: four up to 8 rows, three up to 32, two up to 64, as many as TMEM
  // holds -- except for 9 to 16 rows, where a fourth would fit.  It gains on long
  // steps only (12 requests of 32768 tokens, 8 heads, 162 pages an SM: 99.4 us,
  // with three 100.2; 32 of 16384, 216 pages: 128.7 and 131.7; 108 pages: 70.7
  // and 70.1) and costs up to a fifth on short ones (54 pages: 45.4 and 41.8 us;
  // 61 requests of up to 6001 tokens, one head: 21.6 and 17.9).  The host knows
  // the config's largest step, not this one's size, and a fourth team that gets
  // no range on short steps costs as much as one that does (21.9 us).  Up to 8
  // rows four teams cost next to nothing on short steps (216 pages an SM: 114 and
  // 122 us; 54: 37.9 and 38.3; 2 requests of 1.5k tokens, one head: 8.1 and 8.0).
  if (a.rows <= 8) return launch_dense<1, 4>(v, a, units, s);
  if (a.rows <= 16) return launch_dense<2, 3>(v, a, units, s);
  if (a.rows <= 32) return launch_dense<4, 3>(v, a, units, s);
  return launch_dense<8, 2>(v, a, units, s);
}
