// msa_tree_attention: full-context attention of the nodes of a draft tree over a
// paged cache of bf16, e4m3 or NVFP4 rows (with a chain's masks: the dense decode
// and verify of any KV type).
//
// Mathematics.  For node i and query head q of KV head h's group, over the keys u
// that the node sees (the cached prefix, and the nodes of its mask):
//     s_u = scale q . k_u,   out = sum_u 2^(s'_u - m) v_u / sum_u 2^(s'_u - m),
// s' = s log2 e, in one pass with a running maximum m and sum.  Scores are sums in fp32
// of products of
//   bf16 pools   bf16 operands, as they are;
//   e4m3 pools   e4m3 operands: the keys' codes as stored, a query row as two e4m3 rows
//                times a power of two (split_e4m3: an element is off by at most 2^-17 of
//                its row's largest; any finite bf16 query, none is flagged);
//   NVFP4 pools  fp16 operands: codes times block scales are exact, and so are queries
//                of 2^-14 .. 65504 (larger ones are flagged, smaller ones keep the bits
//                of fp16's subnormals).
// Values enter P V as fp16: exact for e4m3 and NVFP4, for bf16 within 2^-14 .. 65504 (as
// in the prefill tiles; larger ones are flagged).  The probabilities are rounded to fp16
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
// A CTA: a loader warp (pages by TMA into a ring), four converter warps (Q rows, and the
// pages' values as MMA operands; four more for the keys of NVFP4 pages), two MMA warps and
// two softmax warpgroups, and a warp that clears the rows of tokens that have no tree.  An
// item is one (page, tile): S = Q K^T (128 rows x 128 keys), softmax by a thread a
// row (its TMEM lane), P over S, O += P V with P as the A operand from TMEM.  Items
// alternate between the warpgroups, each of which has TMEM of its own for S and O:
// of a pair of tiles each takes one, of a single tile every second page, whose two
// results (m, sum, O) are joined at the end of the segment.  While one warpgroup
// has its softmax, the tensor cores work for the other.
//
// What bounds it.  16 requests of 8k-32k tokens, 32 nodes, 64 + 8 heads, bf16 (1.31 GB,
// 333 GFLOP): 282 us, 4.7 TB/s (0.69 of the measured copy bandwidth) and 1.2 PFLOP/s
// together; the tensor pipe is active for 54 % of the time.  One request of 131071
// tokens, 64 nodes, e4m3: 212 us, 1.3 PFLOP/s (0.67): an item takes an SM 0.93 us, some
// 1770 cycles, of them 1024 of MMAs and, beside them, 1024 of exponentials at 16 a
// cycle.  32 requests of 8k-32k tokens, 6 nodes (48 rows of a single tile): bf16 390 us,
// the copy bandwidth; e4m3 258 us, 0.77 of it; NVFP4 of 9 and 16 nodes 386 and 392 us,
// the conversions.  61 requests of 40-6001 tokens, 1-40 nodes, 16 + 1 heads, e4m3: 67 us,
// some 30 of them items, the rest the beginnings and ends of 260 segments and the merge.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "kv_quant.cuh"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace msa {
namespace {

constexpr int kTile = 128;                     // query rows of an M tile
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kPairRows = 2 * kTile;
constexpr int kMaxCtas = 192;
constexpr float kBias = 7.f;                   // exponent offset of the probabilities
constexpr float kMaxSum = 60000.f;             // a row's sum over a page that fp16 holds
constexpr float kNear = 64.f;                  // |m| of the fast path, in exponents
constexpr float kSlack = 8.f;                  // m lags by up to that

constexpr int kSoftWarps = 8, kConvWarp = kSoftWarps, kConvThreads = 128;   // of a group
constexpr int kBads = 16;

struct TreeArgs {
  int Hkv, Hq, G, max_blocks, rows;            // rows: of a partial
  bool out32;                                  // out is 32-byte aligned
  uint32_t g_magic;                            // row / G = row * g_magic >> 20
  float scale_log2, v_scale;
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  const int64_t* mask;
  __nv_bfloat16* out;
  float* lse;
  float* o_part;                               // [2 * CTAs][32][rows][4]: 4 dims of all rows side
                                               // by side, as the threads of a tile have them
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

// KV types.  Keys and values have rings of operand tiles of their own, a page's
// tile after the other's:
//   bf16   both arrive in their rings; values are converted to fp16 in place;
//   e4m3   keys arrive in their ring (the scores are e4m3 products); values arrive
//          in raw stages and are converted into theirs;
//   NVFP4  both go through raw stages.
template <int KV>
struct Form {
  static constexpr bool kBf16 = KV == MSA_KV_BF16, kE4m3 = KV == MSA_KV_FP8_E4M3,
                        kFp4 = KV == MSA_KV_NVFP4;
  static constexpr int kKeys = kE4m3 ? 3 : 2, kVals = kBf16 ? 3 : 2;           // tiles
  static constexpr int kKeyBytes = kE4m3 ? kTileBytes / 2 : kTileBytes;
  static constexpr int kRawKeys = kFp4 ? 1 : 0, kRawVals = kBf16 ? 0 : (kE4m3 ? 3 : 2);
  static constexpr int kRawBytes = kE4m3 ? kBlock * kHeadDim : kBlock * kFp4Row;
  // shared memory: two Q tiles, keys, values, raw stages
  static constexpr int kKeyAt = 2 * kTileBytes, kValAt = kKeyAt + kKeys * kKeyBytes,
                       kRawAt = kValAt + kVals * kTileBytes,
                       kSmem = kRawAt + (kRawKeys + kRawVals) * kRawBytes;
  // Warps: softmax, converters (four for the values; four for the keys where those
  // are converted too), loader, two for the MMAs, one for idle tokens.
  static constexpr int kConvWarps = kFp4 ? 8 : 4, kLoadWarp = kConvWarp + kConvWarps,
                       kMmaWarp = kLoadWarp + 1, kIdleWarp = kMmaWarp + 2,
                       kThreads = 32 * (kIdleWarp + 1);
  // threads x launch registers: 512 x 128 = 256 x 176 + 128 x 96 + 128 x 64;
  // 640 x 96 >= 256 x 152 + 256 x 56 + 128 x 56
  static constexpr int kSoftRegs = kFp4 ? 152 : 176, kConvRegs = kFp4 ? 56 : 96,
                       kMiscRegs = kFp4 ? 56 : 64;
  // weight of a page for a pair of two tiles and of one, and of a group's beginning and
  // end (Q, the first S, the last P V, the result)
  static constexpr int kW2 = 4, kW1 = 3, kHead = 9;
};

constexpr int at_least(int n) { return n < 1 ? 1 : n; }

// What the roles share.
template <int KV>
struct Shared {
  using F = Form<KV>;
  // full: arrived; ready: converted; empty: read by the MMAs
  uint64_t k_full[F::kKeys], k_ready[F::kKeys], k_empty[F::kKeys];
  uint64_t v_full[F::kVals], v_ready[F::kVals], v_empty[F::kVals];
  uint64_t kr_full[at_least(F::kRawKeys)], kr_empty[at_least(F::kRawKeys)];
  uint64_t vr_full[at_least(F::kRawVals)], vr_empty[at_least(F::kRawVals)];
  uint64_t q_full[2], q_free[2];
  uint64_t s_ready[2], p_ready[2], o_done[2], turn[2], mid[2], fin[2];
  unsigned long long bad[kBads];               // by segment: nodes with values that are not finite
  float2 ml[2][kTile];                         // by warpgroup: (m, sum) of a row
  uint32_t tmem_base;
  // the CTA's range
  int r0;                                      // first request, and the weight before it
  uint32_t w0, from, to, total, ranges;
  uint32_t part[F::kThreads / 32];
};

// A place in a ring of N: the buffer, and the parity of its use.
template <int N>
struct Place {
  int b = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void next() {
    if (++b == N) {
      b = 0;
      par ^= 1u;
    }
  }
};

// Weights.  A request: heads x pairs of tiles x pages.
struct Req {
  int n, t0, base, L, nb, rows, pairs;
  uint32_t gw, hw, weight;                     // of a group of two tiles; a head; the request
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
  q.rows = t.n * a.G;
  // (small trees over NVFP4 pools are the dense decode's)
  const bool ours = t.n > 0 && !(F::kFp4 && q.rows <= kTreeDenseRows);
  q.nb = ours ? (q.L + kBlock - 1) / kBlock : 0;
  const int tiles = (q.rows + kTile - 1) / kTile;
  q.pairs = (tiles + 1) / 2;
  q.gw = (uint32_t)(q.nb * F::kW2 + F::kHead);
  q.hw = q.nb == 0 ? 0
                   : (uint32_t)(tiles / 2) * q.gw + (tiles & 1) * (uint32_t)(q.nb * F::kW1 + F::kHead);
  q.weight = q.hw * (uint32_t)a.Hkv;
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
// page belongs to the range in which its weight starts, a group's own weight before
// its first page.
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
      const uint32_t x = w - wr;
      h = (int)(x / q.hw);
      const uint32_t y = x - h * q.hw;
      pair = min((int)(y / q.gw), q.pairs - 1);
      rows = min(kPairRows, q.rows - pair * kPairRows);
      tiles = rows > kTile ? 2 : 1;
      const uint32_t step = tiles == 2 ? F::kW2 : F::kW1;
      const uint32_t g0 = wr + h * q.hw + pair * q.gw + F::kHead;              // of page 0
      j0 = w > g0 ? (int)((w - g0 + step - 1) / step) : 0;
      j1 = end > g0 ? (int)min((uint32_t)q.nb, (end - g0 + step - 1) / step) : 0;
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
// Lane i of the warp's quarter, 64 columns.
__device__ __forceinline__ void tmem_st64(uint32_t taddr, const uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x64.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%"
      "23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%"
      "43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%"
      "63,%64"
      "};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(r[32]), "r"(r[33]), "r"(r[34]), "r"(r[35]), "r"(r[36]), "r"(r[37]),
      "r"(r[38]), "r"(r[39]), "r"(r[40]), "r"(r[41]), "r"(r[42]), "r"(r[43]),
      "r"(r[44]), "r"(r[45]), "r"(r[46]), "r"(r[47]), "r"(r[48]), "r"(r[49]),
      "r"(r[50]), "r"(r[51]), "r"(r[52]), "r"(r[53]), "r"(r[54]), "r"(r[55]),
      "r"(r[56]), "r"(r[57]), "r"(r[58]), "r"(r[59]), "r"(r[60]), "r"(r[61]),
      "r"(r[62]), "r"(r[63])
      : "memory");
}
// Waits for this thread's TMEM loads; the registers pass through it, so that no use
// of them moves before it.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
        "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
        "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
        "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
        "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 32 bytes of a row: a whole sector in one store where the address allows it (a
// thread has a row of its own, and half sectors cost as much as whole ones).
__device__ __forceinline__ void store32(void* p, const uint32_t (&h)[8], bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(h[0]), "r"(h[1]),
                 "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// ---------------------------------------------------------------- e4m3 scores
// D[tmem] (+)= A[smem] * B[smem]^T of e4m3 operands, one K step of 32.
template <bool kAcc>
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint32_t alo, uint32_t ahi,
                                          uint32_t blo, uint32_t bhi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .b64 a, b;\n .reg .pred p;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n}" ::"r"(d_tmem),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "n"(kAcc ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ float exp2_of(int e) { return __int_as_float((e + 127) << 23); }

// Largest magnitudes of the even and of the odd ones of eight bf16, as their bits.
__device__ __forceinline__ uint32_t largest(const uint4& v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                  __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
// The exponent e of a query row's scale from its largest magnitudes: they lie in
// [2^7, 2^8) of 2^e.  (Not below -107: scales stay normal numbers.  A row with an
// element that is not finite is NaN, whatever its scale.)
__device__ __forceinline__ int row_exponent(uint32_t top) {
  const int x = (int)max(top & 0xffffu, top >> 16);
  return max((x >> 7) - 127, -100) - 7;
}

// Eight elements of a bf16 query row (sixteen lanes hold the row) as hi + lo of two
// e4m3 values times 2^e, the row's largest magnitude scaled into [128, 256).  bf16
// has 8 significant bits and e4m3 4: hi takes the first four, what is left is a
// multiple of 2^-7 of at most 2^-4 (of the element's power of two), which lo holds
// exactly down to e4m3's smallest step, 2^-9: an element is off by at most 2^-10,
// 2^-17 of the row's largest.  Elements that are not finite become NaN.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ void split_e4m3(const uint4& v, uint2& q_hi, uint2& q_lo) {
  uint32_t top = largest(v);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float scale = exp2_of(-row_exponent(top));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // times 0 is NaN where it is not finite, and adds nothing elsewhere; the eight
    // bits fit fp16's eleven, below 2^-16 apart, and so does what hi leaves
    const float a = bf16lo(w[i]), b = bf16hi(w[i]);
    const uint32_t x = pack_f16(fmaf(a, 0.f, a * scale), fmaf(b, 0.f, b * scale));
    h[i] = e4m3x2_of_f16x2(x);
    const uint32_t y = e4m3x2_to_f16x2((uint16_t)h[i]);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x),
                              *reinterpret_cast<const __half2*>(&y));
    l[i] = e4m3x2_of_f16x2(*reinterpret_cast<const uint32_t*>(&r));
  }
  q_hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  q_lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
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

// A chunk of a page's slot: 16 bytes of the tile it becomes (bf16, whose tile it is
// already), or 16 dims that become two such chunks (e4m3, NVFP4).  Eight (sixteen)
// lanes take the same chunk of eight (sixteen) rows, which the swizzles of the raw
// tile (72-byte rows) and of the operand spread over all banks.
template <int KV>
struct Chunk {
  static constexpr bool kBf16 = KV == MSA_KV_BF16;
  static constexpr int kOut = kBf16 ? 1 : 2, kChunks = kTileBytes / 16 / kOut / kConvThreads;
  uint4 w;                     // as read (NVFP4: 8 bytes, and the scale)
  int key, c;                  // row, and chunk of the row (of kOut operand chunks)

  __device__ __forceinline__ void load(const uint8_t* raw, int x) {
    if constexpr (kBf16) {
      key = (x >> 3) & (kBlock - 1);
      c = (x & 7) ^ (key & 7) | (x >> 10) << 3;
      w = *reinterpret_cast<const uint4*>(raw + x * 16);
    } else if constexpr (KV == MSA_KV_FP8_E4M3) {
      key = (x & 7) | ((x >> 6) << 3);
      c = (x >> 3) & 7;
      w = *reinterpret_cast<const uint4*>(raw + key * 128 + ((c ^ (key & 7)) << 4));
    } else {
      key = (x & 15) | ((x >> 7) << 4);
      c = (x >> 4) & 7;
      const uint8_t* row = raw + key * kFp4Row;
      const uint2 y = *reinterpret_cast<const uint2*>(row + 8 * c);
      w.x = y.x;
      w.y = y.y;
      w.z = row[kHeadDim / 2 + c];
    }
  }
  // eight fp16 values of operand chunk k
  __device__ __forceinline__ void convert(int k, uint32_t (&h)[4]) const {
    if constexpr (kBf16) {
      to_f16(w, h);
    } else if constexpr (KV == MSA_KV_FP8_E4M3) {
      const uint32_t u[2] = {k ? w.z : w.x, k ? w.w : w.y};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        h[2 * e] = e4m3x2_to_f16x2((uint16_t)u[e]);
        h[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(u[e] >> 16));
      }
    } else {
      const uint32_t s = e4m3_scale_f16x2(w.z);
      e2m1x8_to_f16x2(k ? w.y : w.x, h);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = hmul2_u32(h[e], s);
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile, int k, const uint32_t (&h)[4]) const {
    *reinterpret_cast<uint4*>(tile + swz_tma(key, kOut * c + k)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
};

// One page's K or V slot -> the operand tile at `tile` (K-major rows, 128-byte
// swizzle), by a group of converter threads; a bf16 tile in place.  kEdge: a page of
// values with an end or nodes in it: rows from `ntok` on become 0; of rows from `all`
// on (which not every query row sees: 0 * NaN is not 0) elements that are not finite
// become 0 and are noted in `bad` by node.  Returns whether a value left the fp16
// range.  (The pages without edges are most, and their loop has to stay small: the
// roles' loops together have to fit the instruction cache.)
template <int KV, bool kEdge>
__device__ __forceinline__ bool convert_page(const uint8_t* raw, uint8_t* tile, int tid, int ntok,
                                             int all, unsigned long long* bad) {
  using C = Chunk<KV>;
  constexpr int kAhead = kEdge ? 1 : 4;
  bool ovf = false;
  uint32_t top = 0;                            // bf16: largest magnitudes
#pragma unroll 1
  for (int i = 0; i < C::kChunks; i += kAhead) {
    C chunk[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) chunk[e].load(raw, tid + kConvThreads * (i + e));
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
#pragma unroll
      for (int k = 0; k < C::kOut; ++k) {
        uint32_t h[4];
        chunk[e].convert(k, h);
        if (kEdge) {
          const int key = chunk[e].key;
          if (key >= ntok) {
            h[0] = h[1] = h[2] = h[3] = 0u;
          } else {
            if (KV == MSA_KV_BF16) ovf |= any_inf(h);
            if (key >= all && clear_non_finite(h)) atomicOr(bad, 1ull << (key - all));
          }
        } else if (KV == MSA_KV_BF16) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t m = h[q] & 0x7fff7fffu;
            const __half2 y = __hmax2(*reinterpret_cast<const __half2*>(&top),
                                      *reinterpret_cast<const __half2*>(&m));
            top = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
        chunk[e].store(tile, k, h);
      }
    }
  }
  return ovf | f16x2_has_inf(top);
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
__global__ void __launch_bounds__(Form<KV>::kThreads, 1)
tree_attention_kernel(WsView ws, TreeArgs a, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v) {
  using F = Form<KV>;
  constexpr int kThreads = F::kThreads, kLoadWarp = F::kLoadWarp, kMmaWarp = F::kMmaWarp,
                kIdleWarp = F::kIdleWarp;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) Shared<KV> sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);         // uniform
  if (tid == 0) {
    for (int i = 0; i < F::kKeys; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_ready[i], 4);
      mbar_init(&sh.k_empty[i], 2);            // both MMA warps, or one twice
    }
    for (int i = 0; i < F::kVals; ++i) {
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_ready[i], 4);
      mbar_init(&sh.v_empty[i], 2);
    }
    for (int i = 0; i < F::kRawKeys; ++i) {
      mbar_init(&sh.kr_full[i], 1);
      mbar_init(&sh.kr_empty[i], 4);
    }
    for (int i = 0; i < F::kRawVals; ++i) {
      mbar_init(&sh.vr_full[i], 1);
      mbar_init(&sh.vr_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.q_free[i], 2);             // both MMA warps
      mbar_init(&sh.s_ready[i], 1);
      mbar_init(&sh.p_ready[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.turn[i], 1);
      mbar_init(&sh.mid[i], 1);
      mbar_init(&sh.fin[i], 1);
    }
    for (int i = 0; i < kBads; ++i) sh.bad[i] = 0;
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
    regs_down<F::kMiscRegs>();
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loader
      // The pages of a segment 32 at a time (a lane each).
      Walk<KV> wk;
      wk.open(ws, a, sh);
      Place<F::kFp4 ? at_least(F::kRawKeys) : F::kKeys> kp;
      Place<F::kBf16 ? F::kVals : at_least(F::kRawVals)> vp;
      int keys = 0, vals = 0;                  // copied
      bool going = true;                       // after a wait gave up nothing more is copied
      // one page's slot (kind 0 keys, 1 values) into `dst`, once `empty` says so
      auto copy = [&](const Walk<KV>& wk, int j, int page, int kind, uint64_t* empty, uint64_t* full,
                      uint32_t par, uint8_t* dst) {
        going = __all_sync(0xffffffffu, mbar_wait(empty, par ^ 1u, ws.hdr));
        if (!going) return;
        if (elect_one()) {
          if (page < 0) {
            mbar_arrive(full);
          } else if constexpr (F::kFp4) {
            const int64_t slot = ((int64_t)page * a.Hkv + wk.h) * 2 + kind;
            const int rows = min(kBlock, wk.q.L - j * kBlock);
            const uint32_t bytes = (uint32_t)((rows + 1) & ~1) * kFp4Row;       // 16 divides it
            mbar_arrive_expect_tx(full, bytes);
            bulk_load(dst, (kind ? a.v_pool : a.k_pool) + slot * (kBlock * kFp4Row), bytes, full);
          } else {
            const int y = (page * a.Hkv + wk.h) * kBlock;
            const void* map = kind ? (const void*)&tmap_v : (const void*)&tmap_k;
            if constexpr (F::kE4m3) {
              mbar_arrive_expect_tx(full, F::kRawBytes);
              tma_load_2d(dst, map, 0, y, full);
            } else {
              mbar_arrive_expect_tx(full, kTileBytes);
              tma_load_2d(dst, map, 0, y, full);
              tma_load_2d(dst + kTileBytes / 2, map, 64, y, full);
            }
          }
        }
        __syncwarp();
      };
      while (going && wk.next(ws, a)) {
        int mine = -1;
        for (int j = wk.j0; going && j < wk.j1; ++j) {
          const int k = (j - wk.j0) & 31;
          if (k == 0)
            mine = j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + j + lane] : -1;
          const int page = __shfl_sync(0xffffffffu, mine, k);
          if constexpr (F::kFp4)
            copy(wk, j, page, 0, &sh.kr_empty[kp.b], &sh.kr_full[kp.b], kp.par,
                 smem + F::kRawAt + kp.b * F::kRawBytes);
          else
            copy(wk, j, page, 0, &sh.k_empty[kp.b], &sh.k_full[kp.b], kp.par,
                 smem + F::kKeyAt + kp.b * F::kKeyBytes);
          if (!going) break;
          kp.next();
          ++keys;
          if constexpr (F::kBf16)
            copy(wk, j, page, 1, &sh.v_empty[vp.b], &sh.v_full[vp.b], vp.par,
                 smem + F::kValAt + vp.b * kTileBytes);
          else
            copy(wk, j, page, 1, &sh.vr_empty[vp.b], &sh.vr_full[vp.b], vp.par,
                 smem + F::kRawAt + (F::kRawKeys + vp.b) * F::kRawBytes);
          if (!going) break;
          vp.next();
          ++vals;
        }
      }
      // The copies land before the CTA retires (the converters and the MMAs wait for them
      // too, unless a wait gave up).
      if (lane == 0) {
        auto drain = [&](uint64_t* bars, int n, int b, uint32_t par, int arms) {
          for (int i = 0; i < n; ++i)          // its last use: of this round before b, else the last
            if (i < arms) mbar_drain(&bars[i], i < b ? par : par ^ 1u);
        };
        drain(F::kFp4 ? sh.kr_full : sh.k_full, F::kFp4 ? F::kRawKeys : F::kKeys, kp.b, kp.par,
              keys);
        drain(F::kBf16 ? sh.v_full : sh.vr_full, F::kBf16 ? F::kVals : F::kRawVals, vp.b, vp.par,
              vals);
      }
    } else if (warp < kIdleWarp) {
      // ---------------------------------------------------------------- MMAs
      // A warp per softmax warpgroup w, on the items of w: O += P V, then the next S
      // once that has read the P which it overwrites.  The same wait orders O for
      // the softmax: where an S is there, O holds the items before it.  The two
      // warps take turns, an item's P V and the next S together: left to themselves
      // they fall into step, both in the tensor cores, then both in the softmax.
      const int w = warp - kMmaWarp;
      // (the fields of e4m3 x e4m3 read as those of fp16 x fp16)
      const uint32_t idesc_s = idesc_f16(F::kBf16 ? 1 : 0, kTile, kBlock),
                     idesc_o = idesc_f16_bmn(0, kTile, kHeadDim);
      const uint64_t d0 = kstep_desc(smem_u32(smem), 0, kTile),
                     v0 = sdesc_sw128_mn(smem_u32(smem), kTileBytes / 2);
      const uint32_t lo = (uint32_t)d0, hi = (uint32_t)(d0 >> 32), v_lo = (uint32_t)v0,
                     v_hi = (uint32_t)(v0 >> 32);
      const uint32_t ts = tmem + w * 128, to = tmem + 256 + w * 128;
      Walk<KV> wk;
      wk.open(ws, a, sh);
      Place<F::kKeys> kp;                      // of the next page
      Place<F::kVals> vp;
      int k0 = 0, mine = 0, qsel = 0;          // first item of the segment; items of w so far
      uint32_t q_phase = 0;                    // bit b: uses of Q buffer b, odd or even
      uint32_t mids = 0;
      constexpr int kMid = 2;
      while (wk.next(ws, a)) {
        const bool two = wk.tiles == 2;
        const int pages = wk.j1 - wk.j0, odd = (w ^ k0) & 1;
        const int qb = two ? odd : qsel;       // this warp's Q
        const int step = two ? 1 : 2;
        if (!two) qsel ^= 1;
        auto issue_s = [&](int kb, int p, bool pass) {
          tc_fence_after();
          if (elect_one()) {
            const uint32_t qd = lo + qb * (kTileBytes >> 4),
                           kd = lo + ((F::kKeyAt + kb * F::kKeyBytes) >> 4);
            if constexpr (F::kE4m3) {          // Q as two e4m3 tiles, 32 dims a step
#pragma unroll
              for (int ks = 0; ks < 8; ++ks) {
                const uint32_t qs = qd + (ks >> 2) * (kTileBytes >> 5) + (ks & 3) * 2,
                               kk = kd + (ks & 3) * 2;
                if (ks == 0) umma_e4m3<false>(ts, qs, hi, kk, hi, idesc_s);
                else umma_e4m3<true>(ts, qs, hi, kk, hi, idesc_s);
                if (ks == kMid && pass) umma_commit(&sh.mid[w]);
              }
            } else {
              umma_ss<false>(ts, qd, hi, kd, hi, idesc_s);
#pragma unroll
              for (int ks = 1; ks < 8; ++ks) {
                const uint32_t o = (ks >> 2) * (kTileBytes >> 5) + (ks & 3) * 2;
                umma_ss<true>(ts, qd + o, hi, kd + o, hi, idesc_s);
                if (ks == kMid && pass) umma_commit(&sh.mid[w]);
              }
            }
            umma_commit(&sh.s_ready[w]);
            umma_commit(&sh.k_empty[kb]);
            if (!two) umma_commit(&sh.k_empty[kb]);              // (counts both warps)
            if (p + step >= pages) umma_commit(&sh.q_free[qb]);  // its last S
          }
          __syncwarp();
          if (pass) {
            // MMAs of two warps would take turns one by one: the turn goes on when
            // these are so far that the other's first follows their last
            mbar_wait(&sh.mid[w], mids & 1u, ws.hdr);
            ++mids;
            __syncwarp();
            if (elect_one()) mbar_arrive(&sh.turn[w ^ 1]);
            __syncwarp();
          }
        };
        auto wait = [&](uint64_t* bar, uint32_t par) {
          mbar_wait(bar, par, ws.hdr);
          __syncwarp();
        };
        auto k_bar = [&](int b) { return F::kFp4 ? &sh.k_ready[b] : &sh.k_full[b]; };
        int p = two ? 0 : odd, taken = 0;      // pages that kp and vp have passed
        const bool any = p < pages;
        auto go = [&](int page) {              // to a page of the segment
          for (; taken < page; ++taken) {
            kp.next();
            vp.next();
          }
        };
        if (any) {                             // the first S of the segment, without a turn
          go(p);
          wait(k_bar(kp.b), kp.par);
          wait(&sh.q_full[qb], q_phase >> qb & 1u);
          if (mine > 0) wait(&sh.o_done[w], (uint32_t)(mine - 1) & 1u);
          issue_s(kp.b, p, false);
        }
        for (; p < pages; p += step) {
          const bool next = p + step < pages;
          const int vb = vp.b;
          wait(&sh.v_ready[vb], vp.par);
          go(next ? p + step : p);
          wait(&sh.p_ready[w], (uint32_t)mine & 1u);
          if (mine > 0 || w == 1)              // phase n of a turn: the other's n-th pass
            wait(&sh.turn[w], (uint32_t)(w ? mine : mine - 1) & 1u);
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vd = v_lo + ((F::kValAt + vb * kTileBytes) >> 4);
            if (p < step) umma_ts<false>(to, ts, vd, v_hi, idesc_o);   // O of the segment begins
            else umma_ts<true>(to, ts, vd, v_hi, idesc_o);
#pragma unroll
            for (int ks = 1; ks < 8; ++ks)
              umma_ts<true>(to, ts + 8 * ks, vd + 128 * ks, v_hi, idesc_o);
            umma_commit(&sh.o_done[w]);
            umma_commit(&sh.v_empty[vb]);
            if (!two) umma_commit(&sh.v_empty[vb]);
          }
          __syncwarp();
          // Keys that are not there yet are not waited for in one's turn.  (Asked
          // after the turn came: the other warp's S of the page before is done, and
          // with it the phase before the one that is asked for.)
          const bool here =
              next && __shfl_sync(0xffffffffu, (int)mbar_test_wait(k_bar(kp.b), kp.par), 0);
          if (!here && elect_one()) mbar_arrive(&sh.turn[w ^ 1]);
          __syncwarp();
          if (next) {
            if (!here) wait(k_bar(kp.b), kp.par);
            wait(&sh.o_done[w], (uint32_t)mine & 1u);
            issue_s(kp.b, p + step, here);
          }
          ++mine;
        }
        go(pages);
        // a Q buffer that this warp did not read: seen all the same, so that none of
        // its phases passes this warp by
        for (int b = 0; b < 2; ++b) {
          if (!two && b != qb) continue;
          if (!any || b != qb) {
            wait(&sh.q_full[b], q_phase >> b & 1u);
            if (elect_one()) mbar_arrive(&sh.q_free[b]);
            __syncwarp();
          }
          q_phase ^= 1u << b;
        }
        k0 += pages * wk.tiles;
      }
      // every MMA issued here has completed before TMEM goes and the smem is left
      if (elect_one()) umma_commit(&sh.fin[w]);
      __syncwarp();
      mbar_drain(&sh.fin[w], 0);
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
        uint4* row = reinterpret_cast<uint4*>(a.out + (int64_t)t * a.Hq * kHeadDim);
        for (int x = lane; x < a.Hq * (kHeadDim / 8); x += 32) row[x] = make_uint4(0, 0, 0, 0);
        for (int x = lane; x < a.Hq; x += 32) a.lse[(int64_t)t * a.Hq + x] = -INFINITY;
      }
    }
  } else if (warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    regs_down<F::kConvRegs>();
    // Four warps convert the values (and load Q), four more the keys of NVFP4 pages
    // (and load Q there).
    const int ct = (tid - kConvWarp * 32) & (kConvThreads - 1);
    const bool keys = F::kFp4 && warp < kConvWarp + 4;
    Walk<KV> wk;
    wk.open(ws, a, sh);
    Place<F::kKeys> kp;
    Place<F::kVals> vp;
    Place<at_least(F::kRawKeys)> krp;
    Place<at_least(F::kRawVals)> vrp;
    int seg = 0, qsel = 0;
    uint32_t q_used = 0, q_phase = 0;          // bit b: Q buffer b was used; its uses, odd or even
    auto done = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // Q rows of tile t of the segment into buffer b, zero past the last
    auto load_q = [&](int t, int b) {
      if (q_used >> b & 1u) mbar_wait(&sh.q_free[b], (q_phase >> b & 1u) ^ 1u, ws.hdr);
      q_used |= 1u << b;
      q_phase ^= 1u << b;
      bool ovf = false;
      const int first = wk.pair * kPairRows + t * kTile, rows = wk.rows - t * kTile;
      uint8_t* dst = smem + b * kTileBytes;
      // All copies in flight at once, straight to their places as bf16 rows; then, where
      // the scores are no bf16 products, in place: a warp has two rows at a time, and
      // the two e4m3 rows of a Q row take the place of its two halves.
      constexpr int kN = kTile * 16 / kConvThreads;
#pragma unroll 4
      for (int i = 0; i < kN; ++i) {
        const int x = ct + kConvThreads * i, row = x >> 4, ch = x & 15;
        const bool in = row < rows;
        cp_async16(smem_u32(dst + kmaj_off(row, ch, kTile)),
                   a.q + (in ? a.q_row(wk.q.t0, wk.h, first + row) : 0) * kHeadDim + 8 * ch,
                   in ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      if constexpr (!F::kBf16) {
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < kN; ++i) {
          const int x = ct + kConvThreads * i, row = x >> 4, ch = x & 15;
          uint4* place = reinterpret_cast<uint4*>(dst + kmaj_off(row, ch, kTile));
          const uint4 v = *place;
          if constexpr (F::kE4m3) {
            uint2 q_hi, q_lo;
            split_e4m3(v, q_hi, q_lo);
            __syncwarp();                      // the rows are read
            uint8_t* at = dst + row * 128 + (((ch >> 1) ^ (row & 7)) << 4) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(at) = q_hi;
            *reinterpret_cast<uint2*>(at + kTileBytes / 2) = q_lo;
          } else {
            uint32_t h[4];
            to_f16(v, h);
            ovf |= any_inf(h);
            *place = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
      if (F::kFp4 && __any_sync(0xffffffffu, ovf) && lane == 0)
        set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
      done(&sh.q_full[b]);
    };
    while (wk.next(ws, a)) {
      if (!F::kFp4 || keys) {
#pragma unroll 1
        for (int t = 0; t < wk.tiles; ++t) load_q(t, wk.tiles == 2 ? t : qsel);
      }
      if (wk.tiles == 1) qsel ^= 1;
      if (!keys && ct == 0) sh.bad[(seg + kBads / 2) & (kBads - 1)] = 0;
      // ---- pages
      unsigned long long* bad = &sh.bad[seg & (kBads - 1)];
      int mine = -1;
      bool ovf = false;
      for (int j = wk.j0; j < wk.j1; ++j) {
        const int k = (j - wk.j0) & 31;
        if (k == 0)
          mine = j + lane < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + j + lane] : -1;
        const bool usable = __shfl_sync(0xffffffffu, mine, k) >= 0;
        const int ntok = usable ? wk.q.L - j * kBlock : 0;       // keys that exist
        const int all = usable ? wk.q.base - j * kBlock : 0;     // and that every row sees
        if (keys) {
          if constexpr (F::kFp4) {
            mbar_wait(&sh.kr_full[krp.b], krp.par, ws.hdr);
            mbar_wait(&sh.k_empty[kp.b], kp.par ^ 1u, ws.hdr);
            convert_page<KV, false>(smem + F::kRawAt + krp.b * F::kRawBytes,
                                    smem + F::kKeyAt + kp.b * kTileBytes, ct, 0, 0, nullptr);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.kr_empty[krp.b]);
            done(&sh.k_ready[kp.b]);
            krp.next();
            kp.next();
          }
          continue;
        }
        uint8_t* tile = smem + F::kValAt + vp.b * kTileBytes;
        if constexpr (F::kBf16) {
          mbar_wait(&sh.v_full[vp.b], vp.par, ws.hdr);
          ovf |= all >= kBlock ? convert_page<KV, false>(tile, tile, ct, 0, 0, nullptr)
                               : convert_page<KV, true>(tile, tile, ct, ntok, all, bad);
        } else {
          mbar_wait(&sh.vr_full[vrp.b], vrp.par, ws.hdr);
          mbar_wait(&sh.v_empty[vp.b], vp.par ^ 1u, ws.hdr);
          const uint8_t* src = smem + F::kRawAt + (F::kRawKeys + vrp.b) * F::kRawBytes;
          if (all >= kBlock) convert_page<KV, false>(src, tile, ct, 0, 0, nullptr);
          else convert_page<KV, true>(src, tile, ct, ntok, all, bad);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.vr_empty[vrp.b]);
          vrp.next();
        }
        done(&sh.v_ready[vp.b]);
        vp.next();
      }
      if (F::kBf16 && __any_sync(0xffffffffu, ovf) && lane == 0)
        set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
      ++seg;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // Control flow depends on the plan's data alone (never on what a wait saw),
    // so that the named barriers match even after a wait gave up.
    regs_up<F::kSoftRegs>();
    constexpr int kBar = 1, kCount = kSoftWarps * 32;
    constexpr int kC = 32;                     // columns at a time
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lanes + wg * 128, to = lanes + 256 + wg * 128;
    Walk<KV> wk;
    wk.open(ws, a, sh);
    int k0 = 0, seg = 0;                       // k0: first item of the segment
    int4 split = make_int4(0, 0, 0, 0);
    while (wk.next(ws, a)) {
      const bool two = wk.tiles == 2;
      const int pages = wk.j1 - wk.j0, odd = (wg ^ k0) & 1;
      const int t = two ? odd : 0;             // this warpgroup's tile
      float sc = a.scale_log2;                 // exponent of a score
      float m = -INFINITY, l = 0.f;
      uint64_t mask = 0;                       // what the row sees of the nodes
      const int n = t * kTile + row;           // row of the pair
      const bool on = n < wk.rows;
      if (on) {
        const int i = a.node_of(wk.pair * kPairRows + n);
        mask = a.mask ? (uint64_t)a.mask[wk.q.t0 + i] : ~0ull >> (63 - i);
        if (wk.q.n < 64) mask &= (1ull << wk.q.n) - 1;
        if constexpr (F::kE4m3) {              // the scale of the row's Q, from the row itself
          const uint4* q = reinterpret_cast<const uint4*>(
              a.q + a.q_row(wk.q.t0, wk.h, wk.pair * kPairRows + n) * kHeadDim);
          uint32_t top = 0;
#pragma unroll 4
          for (int c = 0; c < 16; ++c) top = __vmaxu2(top, largest(q[c]));
          sc = a.scale_log2 * exp2_of(row_exponent(top));
        }
      }
      int mine = -1, have = -1;
      bool first = true, fast = false;         // first: page of this warpgroup's
      for (int p = two ? 0 : odd; p < pages; p += two ? 1 : 2) {
        const int k = two ? k0 + 2 * p + t : k0 + p, j = wk.j0 + p;
        if (p >> 5 != have) {
          have = p >> 5;
          const int jj = wk.j0 + 32 * have + lane;
          mine = jj < wk.j1 ? ws.block_table[(int64_t)wk.r * a.max_blocks + jj] : -1;
        }
        const bool usable = __shfl_sync(0xffffffffu, mine, p & 31) >= 0;
        const int d = wk.q.base - j * kBlock;  // keys before the nodes
        mbar_wait(&sh.s_ready[wg], (uint32_t)(k >> 1) & 1u, ws.hdr);
        tc_fence_after();
        const bool plain = usable && d >= kBlock;
        const uint64_t sl = f2(sc, sc);
        uint64_t sum0 = 0, sum1 = 0;
        float mx[2];
        auto most = [&](const uint32_t (&x)[kC]) {
#pragma unroll
          for (int i = 0; i < kC; i += 4) {
            mx[0] = fmax3(mx[0], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            mx[1] = fmax3(mx[1], __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
        };
        uint32_t pk[64];
        // A row's m, and with it its bits, goes by the row alone: where a warp takes
        // the slow path for one row, the others keep theirs and compute the same.
        bool good = false, tried = false, kept = false;
        if (plain && first) {
          // a page that begins a row: the maximum of its first columns stands for all
          uint32_t x[kC];
          tmem_ld32(ts, x);
          tmem_wait32(x);
          mx[0] = mx[1] = -INFINITY;
          most(x);
          m = fmaxf(mx[0], mx[1]);
          fast = __all_sync(0xffffffffu, fabsf(m) * sc < kNear);
        }
        if (plain && fast) {
          // One pass, with m as it is and -m scale + bias rounded to fp32 (fast: off
          // by less than 2^-18): P stays in registers until its sum says that no
          // probability is beyond fp16.
          const float c0 = fmaf(-m, sc, kBias);
          const uint64_t cc = f2(c0, c0);
          auto prob1 = [&](const uint32_t (&x)[kC], uint32_t* y) {
#pragma unroll
            for (int i = 0; i < kC / 2; i += 2) {
              float p0, p1, p2, p3;
              f2_split(fma_f2(f2u(x[2 * i], x[2 * i + 1]), sl, cc), p0, p1);
              f2_split(fma_f2(f2u(x[2 * i + 2], x[2 * i + 3]), sl, cc), p2, p3);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              p2 = ex2_approx(p2);
              p3 = ex2_approx(p3);
              sum0 = add_f2(sum0, f2(p0, p1));
              sum1 = add_f2(sum1, f2(p2, p3));
              y[i] = pack_f16(p0, p1);
              y[i + 1] = pack_f16(p2, p3);
            }
          };
          uint32_t xa[kC], xb[kC];
          if constexpr (F::kFp4) {             // fewer registers: no loads ahead
#pragma unroll
            for (int c = 0; c < kBlock; c += kC) {
              tmem_ld32(ts + c, xa);
              tmem_wait32(xa);
              prob1(xa, pk + c / 2);
            }
          } else {
            tmem_ld32(ts, xa);
#pragma unroll
            for (int c = 0; c < kBlock; c += 2 * kC) {
              tmem_wait32(xa);
              tmem_ld32(ts + c + kC, xb);
              prob1(xa, pk + c / 2);
              tmem_wait32(xb);
              if (c + 2 * kC < kBlock) tmem_ld32(ts + c + 2 * kC, xa);
              prob1(xb, pk + (c + kC) / 2);
            }
          }
          float s0, s1;
          f2_split(add_f2(sum0, sum1), s0, s1);
          tried = true;
          kept = s0 + s1 < kMaxSum;            // (not so for NaN)
          good = __all_sync(0xffffffffu, kept);
        }
        if (good) {
          tmem_st64(ts, pk);                   // over S
        } else {
          // Two passes: the row's maximum over what it sees, then P.  (Loops: this is
          // for pages with an end or nodes in them, and where m moves.)
          auto see = [&](uint32_t (&x)[kC], int c) {             // columns c ..
            if (plain) return;
            const int e = d - c;
            uint32_t vis;
            if (!usable) vis = 0;
            else if (e >= 32) vis = ~0u;
            else if (e > 0) vis = ((1u << e) - 1) | (uint32_t)(mask << e);
            else vis = e > -64 ? (uint32_t)(mask >> -e) : 0;
#pragma unroll
            for (int i = 0; i < kC; ++i)
              if (!(vis >> i & 1)) x[i] = 0xff800000u;
          };
          uint32_t x[kC], y[kC];
          mx[0] = mx[1] = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kBlock; c += 2 * kC) {
            tmem_ld32(ts + c, x);
            tmem_ld32(ts + c + kC, y);
            tmem_wait32(x);
            tmem_wait32(y);
            see(x, c);
            see(y, c + kC);
            most(x);
            most(y);
          }
          const float top = fmaxf(mx[0], mx[1]);
          // the difference, exact near m; -inf - -inf is NaN: no move
          const bool move = tried ? !kept : (top - m) * sc > kSlack;
          if (__any_sync(0xffffffffu, move)) {
            const float mn = move ? fmaxf(m, top) : m;
            const float alpha = mn == -INFINITY ? 1.f : ex2_approx((m - mn) * sc);
            m = mn;
            l *= alpha;
            if (!first) {                      // (S was issued after the last P V of this O)
#pragma unroll 1
              for (int c = 0; c < kHeadDim; c += 32) {
                tmem_ld32(to + c, x);
                tmem_wait32(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * alpha);
                tmem_st32(to + c, x);
              }
            }
          }
          // P = 2^((s - m) scale + bias); m close to 0: as in the one pass
          const bool near = fabsf(m) * sc < kNear;
          const float ref = near || m == -INFINITY ? 0.f : -m;
          const float add = near ? fmaf(-m, sc, kBias) : kBias;
          const uint64_t rf = f2(ref, ref), ad = f2(add, add);
          sum0 = sum1 = 0;
#pragma unroll 1
          for (int c = 0; c < kBlock; c += kC) {
            tmem_ld32(ts + c, x);
            tmem_wait32(x);
            see(x, c);
            uint32_t p[kC / 2];
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
              float p0, p1;
              f2_split(fma_f2(add_f2(f2u(x[2 * i], x[2 * i + 1]), rf), sl, ad), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              if (i & 1) sum1 = add_f2(sum1, f2(p0, p1));
              else sum0 = add_f2(sum0, f2(p0, p1));
              p[i] = pack_f16(p0, p1);
            }
            tmem_st16(ts + c / 2, p);          // over columns that were read
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[wg]);
        {
          float s0, s1;
          f2_split(add_f2(sum0, sum1), s0, s1);
          l += s0 + s1;
        }
        first = false;
        fast = __all_sync(0xffffffffu, fabsf(m) * sc < kNear);
      }

      // ---- the segment's result: whole rows, or a partial
      const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.starts ? 1 : 0);
      const int items = pages * wk.tiles, kl = k0 + items - 1;   // the last item, and the one
                                                                 // before it in the other slot
      float* part = a.o_part + (slot * kHeadDim / 4 * a.rows + n) * 4;       // + dim * rows
      const int64_t out_row = on ? a.q_row(wk.q.t0, wk.h, wk.pair * kPairRows + n) : 0;
      __nv_bfloat16* out = a.out + out_row * kHeadDim;
      // Two tiles: this warpgroup's O, all dims.  One: both warpgroups' results of a
      // row, joined, half its dims each.  (A small loop: it runs once a segment, from
      // a cold instruction cache.)
      int dim0 = 0, dims = kHeadDim;
      uint32_t t0 = to, t1 = 0;                // the O's columns; the other O's
      float f0 = 1.f, f1 = 0.f;
      if (two) {
        const int mine_l = (kl & 1) == wg ? kl : kl - 1;
        mbar_wait(&sh.o_done[wg], (uint32_t)(mine_l >> 1) & 1u, ws.hdr);
      } else {
        sh.ml[wg][row] = make_float2(m, l);
        named_bar_sync(kBar, kCount);
        const int wl = kl & 1;                 // the warpgroup of the last item
        mbar_wait(&sh.o_done[wl], (uint32_t)(kl >> 1) & 1u, ws.hdr);
        const float2 ml = sh.ml[wl][row], mo = sh.ml[wl ^ 1][row];
        m = ml.x;
        l = ml.y;
        dim0 = 64 * wg;
        dims = 64;
        t0 = lanes + 256 + wl * 128;
        if (pages > 1) {
          mbar_wait(&sh.o_done[wl ^ 1], (uint32_t)((kl - 1) >> 1) & 1u, ws.hdr);
          t1 = lanes + 256 + (wl ^ 1) * 128;
          m = fmaxf(ml.x, mo.x);
          f1 = 1.f;
          if (m != -INFINITY) {
            f0 = ex2_approx((ml.x - m) * sc);
            f1 = ex2_approx((mo.x - m) * sc);
          }
          l = ml.y * f0 + mo.y * f1;
        }
      }
      tc_fence_after();
      const bool joined = !two && pages > 1;
      const float inv = !wk.whole ? 1.f : (l == 0.f ? 0.f : a.v_scale / l);
#pragma unroll 1
      for (int c = dim0; c < dim0 + dims; c += 16) {
        uint32_t o[16], q[16];
        tmem_ld16(t0 + c, o);
        if (joined) tmem_ld16(t1 + c, q);
        tmem_wait16(o);
        if (joined) {
          tmem_wait16(q);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + __uint_as_float(q[i]) * f1);
        }
        if (!two && c == dim0 + 48) {          // O and ml may be overwritten from here on
          tc_fence_before();
          named_bar_sync(kBar, kCount);
        }
        if (!on) continue;
        if (wk.whole) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            h[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          store32(out + c, h, a.out32);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(part + (int64_t)(c + 4 * i) * a.rows) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (on && (two || wg == 0)) {
        if (wk.whole)
          a.lse[out_row] = l == 0.f ? -INFINITY : (m * sc + log2f(l) - kBias) * kLn2;
        else
          a.ml_part[slot * a.rows + n] = make_float2(F::kE4m3 ? m * (sc / a.scale_log2) : m, l);
      }
      // rare: values that are not finite, of nodes that the row sees
      for (unsigned long long b = on ? sh.bad[seg & (kBads - 1)] & mask : 0; b; b &= b - 1) {
        const int u = wk.q.base + __ffsll((long long)b) - 1;
        const int page = ws.block_table[(int64_t)wk.r * a.max_blocks + u / kBlock];
        for (int dim = dim0; dim < dim0 + dims; ++dim) {
          const float v = value_of<KV>(a.v_pool, page, a.Hkv, wk.h, u % kBlock, dim);
          if (fabsf(v) < INFINITY) continue;
          if (wk.whole) {
            __nv_bfloat16* y = a.out + out_row * kHeadDim + dim;
            *y = __float2bfloat16_rn(__bfloat162float(*y) + v);
          } else {
            part[(int64_t)(dim & ~3) * a.rows + (dim & 3)] += v;
          }
        }
      }
      tc_fence_before();
      if (wk.starts && !wk.whole) {            // the range ends inside this group
        const int c1 = (int)range_of(sh.total, sh.ranges, wk.last);
        split = make_int4(c1 - (int)blockIdx.x + 1, wk.q.t0, wk.h, wk.pair << 16 | wk.rows);
      }
      k0 += items;
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
// then takes its share of (group, 32 rows).  A lane has a row, as the partials are
// laid out.  Up to kFew partials: a warp takes 16 of the 128 dims, all loads in
// flight at once.  More: a block takes 32 dims, its warps every eighth partial,
// and joins their sums in shared memory.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32, kFew = 4;
constexpr int kMergeChunks = (kMaxCtas + kMergeThreads - 1) / kMergeThreads;
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(TreeArgs a, int ctas) {
  __shared__ int4 list[kMaxCtas];
  __shared__ int owner[kMaxCtas];
  __shared__ int counts[kMergeChunks * kMergeWarps];
  __shared__ union {
    float sums[kMergeWarps][32][33];           // [warp][row][dim], and l
    uint4 stage[32][17];                       // rows of 256 bytes
  } u;
  auto& sums = u.sums;
  auto& stage = u.stage;
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
  // the groups of few partials, then the others by quarters of their dims
  const int tiles = (a.rows + 31) / 32, items = n * tiles;
  for (int item = blockIdx.x; item < 5 * items; item += gridDim.x) {
    const bool few = item < items;
    const int it = few ? item : (item - items) >> 2, quarter = few ? 0 : (item - items) & 3;
    const int gi = it / tiles, row0 = (it - gi * tiles) * 32;
    const int4 g = list[gi];
    const int rows = g.w & 0xffff, np = g.x, row = row0 + lane;
    if (row0 >= rows || few != (np <= kFew)) continue;           // (the whole block)
    const int64_t c0 = owner[gi];
    const bool on = row < rows;
    // partial i: the second slot of c0, the first of c0 + i
    auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };
    auto ml_of = [&](int i) {
      return on ? a.ml_part[slot(i) * a.rows + row] : make_float2(-INFINITY, 0.f);
    };
    auto o_of = [&](int i, int chunk) {
      return on ? *reinterpret_cast<const float4*>(
                      a.o_part + ((slot(i) * (kHeadDim / 4) + chunk) * a.rows + row) * 4)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto weight = [&](float m, float M) {
      return M == -INFINITY ? 1.f : ex2_approx((m - M) * a.scale_log2);
    };
    auto lse_of = [&](float M, float l) {
      return l == 0.f ? -INFINITY : (M * a.scale_log2 + log2f(l) - kBias) * kLn2;
    };
    const int64_t hq = on ? a.q_row(g.y, g.z, (g.w >> 16) * kPairRows + row) : 0;
    if (np <= kFew) {
      float2 ml[kFew];
      float4 v[kFew][4];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        ml[i] = i < np ? ml_of(i) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[i][c] = i < np ? o_of(i, 4 * warp + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < kFew; ++i) M = fmaxf(M, ml[i].x);
      float4 o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        if (i >= np) continue;
        const float f = weight(ml[i].x, M);
        l = fmaf(f, ml[i].y, l);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          o[c].x = fmaf(f, v[i][c].x, o[c].x);
          o[c].y = fmaf(f, v[i][c].y, o[c].y);
          o[c].z = fmaf(f, v[i][c].z, o[c].z);
          o[c].w = fmaf(f, v[i][c].w, o[c].w);
        }
      }
      const float inv = l == 0.f ? 0.f : a.v_scale / l;
#pragma unroll
      for (int c = 0; c < 4; c += 2)           // 16 dims of 32 rows, out through shared memory
        stage[lane][2 * warp + c / 2] =
            make_uint4(pack_bf16(o[c].x * inv, o[c].y * inv), pack_bf16(o[c].z * inv, o[c].w * inv),
                       pack_bf16(o[c + 1].x * inv, o[c + 1].y * inv),
                       pack_bf16(o[c + 1].z * inv, o[c + 1].w * inv));
      if (warp == 0 && on) a.lse[hq] = lse_of(M, l);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {            // a warp's four rows, 16 lanes a row
        const int r = 4 * warp + k;
        const int64_t to = __shfl_sync(0xffffffffu, hq, r);
        if (row0 + r < rows && lane < 16)
          reinterpret_cast<uint4*>(a.out + to * kHeadDim)[lane] = stage[r][lane];
      }
      __syncthreads();
    } else {
      float M = -INFINITY;
#pragma unroll 8
      for (int i = 0; i < np; ++i) M = fmaxf(M, ml_of(i).x);
      float4 o[8];
      float l = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int i = warp; i < np; i += kMergeWarps) {
        const float2 ml = ml_of(i);
        float4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = o_of(i, 8 * quarter + c);
        const float f = weight(ml.x, M);
        l = fmaf(f, ml.y, l);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          o[c].x = fmaf(f, v[c].x, o[c].x);
          o[c].y = fmaf(f, v[c].y, o[c].y);
          o[c].z = fmaf(f, v[c].z, o[c].z);
          o[c].w = fmaf(f, v[c].w, o[c].w);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        sums[warp][lane][4 * c] = o[c].x;
        sums[warp][lane][4 * c + 1] = o[c].y;
        sums[warp][lane][4 * c + 2] = o[c].z;
        sums[warp][lane][4 * c + 3] = o[c].w;
      }
      sums[warp][lane][32] = l;
      __syncthreads();
      // thread: row tid / 8, 4 dims; the warps' sums in order
      const int r = tid >> 3, d = (tid & 7) * 4;
      float y[4] = {0.f, 0.f, 0.f, 0.f}, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += sums[w][r][d + e];
        ll += sums[w][r][32];
      }
      const int64_t to = __shfl_sync(0xffffffffu, hq, r);
      const float Mr = __shfl_sync(0xffffffffu, M, r);
      if (row0 + r < rows) {
        const float inv = ll == 0.f ? 0.f : a.v_scale / ll;
        *reinterpret_cast<uint2*>(a.out + to * kHeadDim + 32 * quarter + d) =
            make_uint2(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv));
        if (quarter == 0 && (tid & 7) == 0) a.lse[to] = lse_of(Mr, ll);
      }
      __syncthreads();
    }
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
  msa_status st = launch_pdl(tree_attention_kernel<KV>, dim3((unsigned)grid), dim3(F::kThreads),
                             F::kSmem, s, v, a, tk, tv);
  if (st != MSA_OK) return st;
  int64_t blocks = grid * ((a.rows + 31) / 32) * 4;
  if (blocks > 4 * sm_count()) blocks = 4 * sm_count();
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
  const size_t n = align_up(2 * (size_t)kMaxCtas * rows * kHeadDim * 4) +
                   align_up(2 * (size_t)kMaxCtas * rows * 8) + align_up(kMaxCtas * sizeof(int4));
  // the two kernels of an NVFP4 step run after one another
  return cfg->kv_dtype == MSA_KV_NVFP4 ? std::max(n, tree_dense_scratch(*cfg)) : n;
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
  a.v_scale = bf16 ? 1.f : cfg->v_scale;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.G = a.Hq / a.Hkv;
  a.g_magic = ((1u << 20) + a.G - 1) / a.G;    // exact for rows up to 1024 and G <= 16
  a.max_blocks = cfg->max_blocks_per_req;
  a.rows = part_rows(*cfg);
  a.out32 = ((uintptr_t)out & 31) == 0;
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
    default: break;
  }
  // NVFP4: the small trees, then the others (either may have none: the host does not
  // know the trees' sizes)
  const msa_status st4 =
      tree_dense_attention(*cfg, v, q, k_pages, v_pages, tree_mask, scratch, out, lse, s);
  if (st4 != MSA_OK) return st4;
  return launch_tree<MSA_KV_NVFP4>(v, a, pool_rows, units, s);
}
