// msa_rope_cache_write: the step's new queries and keys rotated by their
// positions, and keys, values and index keys stored into the paged pools, in
// one pass.
//
// sglang minimax_sparse_backend.py (MiniMaxSparseAttnBackend.forward_decode and
// forward_extend) receives q, k, idx_q and idx_k after the model's rotary
// embedding and stores the keys with set_fused_kv_index_buffer before the
// attention; here the embedding and the store are one launch over the
// projection's output.
//
// Mathematics.  For a head row x and the angles' cosines c_i and sines s_i of
// its position, i < r/2 (r = rotary_dim), the pair (x_a, x_b) = (x_i,
// x_{i + r/2}), or (x_2i, x_2i+1) when interleaved, becomes
//     y_a = x_a c_i - x_b s_i,   y_b = x_b c_i + x_a s_i,
// every product, difference and sum one IEEE fp32 operation (no contraction,
// so that the quantised codes do not depend on the compiler); dims from r on
// are copied.  Queries are rounded to bf16 once; keys go from fp32 straight to
// the pool's type (bf16, e4m3 or NVFP4 codes: kv_quant.cuh).
//
// Work split.  Eight threads own a row (a head of a token), each two 16-byte
// chunks: the two halves of its eight pairs, so a rotation needs no exchange
// between threads, and rows may be rotated in place.  Dims that are only
// copied, and interleaved pairs, give a thread two neighbouring chunks.  A CTA
// takes 32 rows of one token, so the smallest steps spread over the machine
// and every load of the step is in flight at once.
#include "kv_quant.cuh"

namespace msa {
namespace {

constexpr int kRowThreads = 8;
constexpr int kRowsPerCta = 32;

struct RopeArgs {
  int Hq, Hkv, d, max_blocks, kv, interleaved;
  int rot, idx_rot;              // rotary dims of the heads and of the index heads
  int64_t num_positions, pool_slots;
  int64_t qs, ks, vs, iqs, iks, ivs;    // elements between tokens
  float k_scale, v_scale;
  const float* cs;               // [num_positions, rot]: cosines, then sines
  const float* idx_cs;
  const int64_t* positions;      // or null: the plan's
  const int64_t* loc;            // or null: the plan's
  const __nv_bfloat16 *q, *k, *v, *iq, *ik, *iv;
  __nv_bfloat16 *q_out, *iq_out;
  uint8_t *k_pages, *v_pages;    // may be one allocation (NVFP4)
  __nv_bfloat16 *ik_pages, *iv_pages;
};

// Not the non-coherent path: q_out may be q.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

__global__ void __launch_bounds__(kRowsPerCta* kRowThreads)
rope_write_kernel(WsView ws, RopeArgs a) {
  const int t = blockIdx.x;
  const int sub = threadIdx.x & (kRowThreads - 1);
  int row = blockIdx.y * kRowsPerCta + (threadIdx.x >> 3);
  griddep_launch_dependents();
  griddep_wait();            // the plan of this step, and readers of the last one
  if (t >= ws.hdr->num_tokens) return;
  const int r = ws.tok_req[t];
  if (r < 0) return;         // idle request: nothing to rotate or store
  const int plan_pos = ws.tok_pos[t];

  // the row's kind, head and source: q | k | v | idx_q | idx_k | idx_v
  enum { kQ, kK, kV, kIq, kIk, kIv, kNone };
  int kind = kNone, h = row;
  const __nv_bfloat16* src = nullptr;
  if (h < a.Hq) {
    kind = kQ;
    src = a.q + t * a.qs;
  } else {
    h -= a.Hq;
    const int n = h / a.Hkv;
    h -= n * a.Hkv;
    if (n == 0) kind = kK, src = a.k + t * a.ks;
    else if (n == 1) kind = kV, src = a.v + t * a.vs;
    else if (n == 2 && a.iq != nullptr) kind = kIq, src = a.iq + t * a.iqs;
    else if (n == 3 && a.ik != nullptr) kind = kIk, src = a.ik + t * a.iks;
    else if (n == 4 && a.iv != nullptr) kind = kIv, src = a.iv + t * a.ivs;
  }
  const bool idx = kind >= kIq;
  const int width = idx ? a.d : kHeadDim;
  const bool on = kind != kNone && sub < width / 16;
  const int rot = (kind == kV || kind == kIv) ? 0 : (idx ? a.idx_rot : a.rot);
  const bool turn = sub < rot / 16;
  const bool split = turn && !a.interleaved;
  // this thread's two chunks of eight elements
  const int ca = split ? sub : 2 * sub, cb = split ? sub + rot / 16 : 2 * sub + 1;

  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
  const int64_t pos = a.positions != nullptr ? a.positions[t] : plan_pos;
  if (pos < 0 || pos >= a.num_positions) {     // beyond the table: the token is skipped
    if (threadIdx.x == 0) set_error(ws.hdr, MSA_DEVERR_POSITION);
    return;
  }
  if (on) {
    src += h * width;
    const uint4 wa = ld_once(src + 8 * ca), wb = ld_once(src + 8 * cb);
    bf16x8_to_f32(wa, x);
    bf16x8_to_f32(wb, y);
    if (turn) {
      const float4* tab =
          reinterpret_cast<const float4*>((idx ? a.idx_cs : a.cs) + pos * rot + 8 * sub);
      const float4 c0 = __ldg(tab), c1 = __ldg(tab + 1);
      const float4 s0 = __ldg(tab + rot / 8), s1 = __ldg(tab + rot / 8 + 1);
      const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i], w = y[i];
          x[i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
          y[i] = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
          const float u2 = y[2 * i], w2 = y[2 * i + 1];
          y[2 * i] = __fsub_rn(__fmul_rn(u2, c[i + 4]), __fmul_rn(w2, s[i + 4]));
          y[2 * i + 1] = __fadd_rn(__fmul_rn(w2, c[i + 4]), __fmul_rn(u2, s[i + 4]));
        }
      }
    }
  }
  // largest magnitudes of the 16-element blocks of the two chunks: the
  // neighbour's chunks when the halves are split (rot / 16 is even), else both
  // chunks are one block
  float ma = 0.f, mb = 0.f;
  if (a.kv == MSA_KV_NVFP4) {
    const float pa = amax8(x), pb = amax8(y);
    const float na = __shfl_xor_sync(0xffffffffu, pa, 1);
    const float nb = __shfl_xor_sync(0xffffffffu, pb, 1);
    ma = split ? fmaxf(pa, na) : fmaxf(pa, pb);
    mb = split ? fmaxf(pb, nb) : ma;
  }
  if (!on) return;

  if (kind == kQ) {
    __nv_bfloat16* dst = a.q_out + ((int64_t)t * a.Hq + h) * kHeadDim;
    reinterpret_cast<uint4*>(dst)[ca] = pack8(x);
    reinterpret_cast<uint4*>(dst)[cb] = pack8(y);
    return;
  }
  if (kind == kIq) {
    __nv_bfloat16* dst = a.iq_out + ((int64_t)t * a.Hkv + h) * a.d;
    reinterpret_cast<uint4*>(dst)[ca] = pack8(x);
    reinterpret_cast<uint4*>(dst)[cb] = pack8(y);
    return;
  }
  int64_t slot;
  if (a.loc != nullptr) {
    slot = a.loc[t];
  } else {
    const int page = ws.block_table[(int64_t)r * a.max_blocks + plan_pos / kBlock];
    slot = page < 0 ? -1 : (int64_t)page * kBlock + plan_pos % kBlock;
  }
  if (slot < 0 || slot >= a.pool_slots) {
    if (sub == 0) set_error(ws.hdr, MSA_DEVERR_PAGE_RANGE);
    return;
  }
  const int64_t line = (slot / kBlock * a.Hkv + h) * kBlock + slot % kBlock;
  if (idx) {
    uint4* dst = reinterpret_cast<uint4*>((kind == kIk ? a.ik_pages : a.iv_pages) + line * a.d);
    dst[ca] = pack8(x);
    dst[cb] = pack8(y);
  } else {
    const int half = kind == kV;
    uint8_t* pool = half ? a.v_pages : a.k_pages;
    const float g = half ? a.v_scale : a.k_scale;
    if (a.kv == MSA_KV_BF16) {
      uint4* dst = reinterpret_cast<uint4*>(pool) + line * 16;
      dst[ca] = pack8(x);
      dst[cb] = pack8(y);
    } else if (a.kv == MSA_KV_NVFP4) {
      const int64_t l4 = ((slot / kBlock * a.Hkv + h) * 2 + half) * kBlock + slot % kBlock;
      uint8_t* dst = pool + l4 * kFp4Row;
      uint8_t sa, sb;
      const uint32_t wa = nvfp4_codes8(x, ma, g, sa), wb = nvfp4_codes8(y, mb, g, sb);
      reinterpret_cast<uint32_t*>(dst)[ca] = wa;
      reinterpret_cast<uint32_t*>(dst)[cb] = wb;
      if (!split) {
        dst[kHeadDim / 2 + sub] = sa;
      } else if ((sub & 1) == 0) {
        dst[kHeadDim / 2 + ca / 2] = sa;
        dst[kHeadDim / 2 + cb / 2] = sb;
      }
    } else {
      uint2* dst = reinterpret_cast<uint2*>(pool) + line * 16;
      dst[ca] = make_uint2(e4m3x2_of(x[0], x[1], g) | e4m3x2_of(x[2], x[3], g) << 16,
                           e4m3x2_of(x[4], x[5], g) | e4m3x2_of(x[6], x[7], g) << 16);
      dst[cb] = make_uint2(e4m3x2_of(y[0], y[1], g) | e4m3x2_of(y[2], y[3], g) << 16,
                           e4m3x2_of(y[4], y[5], g) | e4m3x2_of(y[6], y[7], g) << 16);
    }
  }
  // the step's later kernels read these rows with TMA (async proxy)
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

bool rows_ok(const void* p, int64_t stride, int64_t row) {
  return aligned16(p) && stride >= row && stride % 8 == 0;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_rope_cache_write(const msa_config* cfg, void* ws, const msa_rope* rope,
                                           const void* q, const void* k, const void* v,
                                           const void* idx_q, const void* idx_k,
                                           const void* idx_v, const int64_t* positions,
                                           const int64_t* out_cache_loc, void* q_out,
                                           void* idx_q_out, void* k_pages, void* v_pages,
                                           void* idx_k_pages, void* idx_v_pages,
                                           msa_stream_t stream) {
  msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (!ws || !rope || !rope->cos_sin || !q || !k || !v || !q_out || !k_pages || !v_pages ||
      (idx_q != nullptr && idx_q_out == nullptr) || (idx_k != nullptr && idx_k_pages == nullptr) ||
      (idx_v != nullptr && idx_v_pages == nullptr))
    return MSA_ERR_INVALID_ARG;
  const bool idx = idx_q != nullptr || idx_k != nullptr;
  const int rot = rope->rotary_dim, idx_rot = idx ? rope->idx_rotary_dim : 0;
  if (rot <= 0 || rot > cfg->head_dim || idx_rot < 0 || idx_rot > cfg->index_dim ||
      rope->num_positions < 1)
    return MSA_ERR_INVALID_ARG;
  if (rot % 32 != 0 || idx_rot % 32 != 0) return MSA_ERR_UNSUPPORTED;
  const float* idx_cs = rope->idx_cos_sin;
  if (idx_cs == nullptr) {       // the heads' table serves the index heads too
    if (idx_rot != 0 && idx_rot != rot) return MSA_ERR_INVALID_ARG;
    idx_cs = rope->cos_sin;
  }
  const int64_t Hq = cfg->num_q_heads, Hkv = cfg->num_kv_heads, d = cfg->index_dim;
  if (!rows_ok(q, rope->q_stride, Hq * kHeadDim) || !rows_ok(k, rope->k_stride, Hkv * kHeadDim) ||
      !rows_ok(v, rope->v_stride, Hkv * kHeadDim) ||
      (idx_q && !rows_ok(idx_q, rope->idx_q_stride, Hkv * d)) ||
      (idx_k && !rows_ok(idx_k, rope->idx_k_stride, Hkv * d)) ||
      (idx_v && !rows_ok(idx_v, rope->idx_v_stride, Hkv * d)))
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(rope->cos_sin) || !aligned16(idx_cs) || !aligned16(q_out) ||
      !aligned16(k_pages) || !aligned16(v_pages) || (idx_q && !aligned16(idx_q_out)) ||
      (idx_k && !aligned16(idx_k_pages)) || (idx_v && !aligned16(idx_v_pages)))
    return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0) return MSA_OK;
  RopeArgs a;
  a.Hq = cfg->num_q_heads;
  a.Hkv = cfg->num_kv_heads;
  a.d = cfg->index_dim;
  a.max_blocks = cfg->max_blocks_per_req;
  a.kv = cfg->kv_dtype;
  a.interleaved = rope->interleaved != 0;
  a.rot = rot;
  a.idx_rot = idx_rot;
  a.num_positions = rope->num_positions;
  a.pool_slots = (int64_t)cfg->num_pages * kBlock;
  a.qs = rope->q_stride;
  a.ks = rope->k_stride;
  a.vs = rope->v_stride;
  a.iqs = rope->idx_q_stride;
  a.iks = rope->idx_k_stride;
  a.ivs = rope->idx_v_stride;
  const bool scaled = cfg->kv_dtype != MSA_KV_BF16;
  a.k_scale = scaled ? cfg->k_scale : 1.f;
  a.v_scale = scaled ? cfg->v_scale : 1.f;
  a.cs = rope->cos_sin;
  a.idx_cs = idx_cs;
  a.positions = positions;
  a.loc = out_cache_loc;
  a.q = (const __nv_bfloat16*)q;
  a.k = (const __nv_bfloat16*)k;
  a.v = (const __nv_bfloat16*)v;
  a.iq = (const __nv_bfloat16*)idx_q;
  a.ik = (const __nv_bfloat16*)idx_k;
  a.iv = (const __nv_bfloat16*)idx_v;
  a.q_out = (__nv_bfloat16*)q_out;
  a.iq_out = (__nv_bfloat16*)idx_q_out;
  a.k_pages = (uint8_t*)k_pages;
  a.v_pages = (uint8_t*)v_pages;
  a.ik_pages = (__nv_bfloat16*)idx_k_pages;
  a.iv_pages = (__nv_bfloat16*)idx_v_pages;
  const int64_t kinds = idx_v ? 5 : (idx_k ? 4 : (idx_q ? 3 : 2));   // row groups past q
  const int64_t chunks = (Hq + kinds * Hkv + kRowsPerCta - 1) / kRowsPerCta;
  if (chunks > 65535) return MSA_ERR_UNSUPPORTED;
  return launch_pdl(rope_write_kernel, dim3((unsigned)T, (unsigned)chunks),
                    dim3(kRowsPerCta * kRowThreads), 0, (cudaStream_t)stream,
                    view_of(*cfg, ws), a);
}
