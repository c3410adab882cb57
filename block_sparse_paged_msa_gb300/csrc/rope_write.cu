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
// copied, and interleaved pairs, give a thread two neighbouring chunks.  The
// rows of all tokens are one list (q | k | v | idx_q | idx_k | idx_v per
// token), 16 of it to a CTA whatever the head counts are.  What bounds it is the
// number of loads in flight: one row a thread at ten CTAs an SM moves the 407 MB
// of 8192 tokens (64 + 8 heads, bf16) in 69.0 us, 5.9 TB/s, 0.87 of the measured
// copy bandwidth; one token takes 2.0 us.  1.4 and 0.2 us of that wait for the
// step's token count before the first row is read (the grid is the config's, the
// inputs end with the step).  Before that wait, at 67.6 us: CTAs of 32 rows 71
// us, of 8 rows 100 us, two rows a thread 86 us, without the streaming stores 73.
#include "kv_quant.cuh"

namespace msa {
namespace {

constexpr int kRowThreads = 8;
constexpr int kSlots = 16;     // threads / kRowThreads of a CTA
constexpr int kKinds = 6;      // q, k, v, idx_q, idx_k, idx_v

// x / d for x < 2^31 by one multiplication.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d_) : d(d_), shift(0) {
    while ((1u << shift) < d) ++shift;         // ceil(log2 d)
    mul = (uint32_t)((((uint64_t)1 << (31 + shift)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
    return (uint32_t)(((uint64_t)x * mul) >> (31 + shift));
  }
};

// One kind of row: where it comes from, its rotation, where it goes.
struct Kind {
  const __nv_bfloat16* src;    // null: the step has none
  int64_t stride;              // elements between tokens
  const float* cs;             // [num_positions, rot]: cosines, then sines
  uint8_t* dst;                // rows by token, or a pool
  int width, rot;
  int pool;                    // kv dtype of the pool, -1 = rows by token (bf16)
  int fp4_slot;                // NVFP4: 0 = keys, 1 = values
  float scale;
};

struct RopeArgs {
  FastDiv R;                   // rows a token
  uint32_t items;              // tokens * rows
  int Hq, Hkv, max_blocks, interleaved;
  int64_t num_positions, pool_slots;
  const int64_t* positions;    // or null: the plan's
  const int64_t* loc;          // or null: the plan's
  Kind kinds[kKinds];
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

__global__ void __launch_bounds__(kSlots* kRowThreads, 10)
rope_write_kernel(WsView ws, const __grid_constant__ RopeArgs a) {
  const int sub = threadIdx.x & (kRowThreads - 1);
  griddep_launch_dependents();
  const uint32_t item = blockIdx.x * kSlots + (threadIdx.x >> 3);
  const int t = (int)a.R(item);
  int h = (int)(item - (uint32_t)t * a.R.d), kind = 0, heads = a.Hq;
  if (h >= a.Hq) {
    h -= a.Hq;
    heads = a.Hkv;
    kind = 1 + (h >= a.Hkv) + (h >= 2 * a.Hkv) + (h >= 3 * a.Hkv) + (h >= 4 * a.Hkv);
    h -= (kind - 1) * a.Hkv;
  }
  const Kind& kd = a.kinds[kind];
  const int width = kd.width, rot = kd.rot;
  const bool turn = sub < rot / 16, split = turn && !a.interleaved;
  // this thread's two chunks of eight elements
  const int ca = split ? sub : 2 * sub, cb = split ? sub + rot / 16 : 2 * sub + 1;
  bool live = item < a.items && kd.src != nullptr && sub < width / 16;
  griddep_wait();              // the projection, the plan, readers of the last step
  // the inputs have rows for the step's tokens only, the grid for the config's
  live = live && t < ws.hdr->num_tokens;
  uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
  int req = -1, plan_pos = 0;
  int64_t pos = 0, slot = 0;
  if (live) {
    const __nv_bfloat16* src = kd.src + t * kd.stride + h * width;
    xa = ld_once(src + 8 * ca);
    xb = ld_once(src + 8 * cb);
    req = ws.tok_req[t];       // -1: idle
    plan_pos = ws.tok_pos[t];
    pos = a.positions != nullptr ? a.positions[t] : plan_pos;
    if (a.loc != nullptr && kd.pool >= 0) slot = a.loc[t];
    live = req >= 0;
    if (live && (uint64_t)pos >= (uint64_t)a.num_positions) {     // beyond the table: skipped
      set_error(ws.hdr, MSA_DEVERR_POSITION);
      live = false;
    }
  }
  float x[8], y[8];
  bf16x8_to_f32(xa, x);
  bf16x8_to_f32(xb, y);
  if (live && turn) {
    const float4* tab = reinterpret_cast<const float4*>(kd.cs + pos * rot + 8 * sub);
    const float4 c0 = __ldg(tab), c1 = __ldg(tab + 1);
    const float4 s0 = __ldg(tab + rot / 8), s1 = __ldg(tab + rot / 8 + 1);
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (split) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = x[i], q = y[i];
        x[i] = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, s[i]));
        y[i] = __fadd_rn(__fmul_rn(q, c[i]), __fmul_rn(p, s[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = x[2 * i], q = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, s[i]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(q, c[i]), __fmul_rn(p, s[i]));
        const float p2 = y[2 * i], q2 = y[2 * i + 1];
        y[2 * i] = __fsub_rn(__fmul_rn(p2, c[i + 4]), __fmul_rn(q2, s[i + 4]));
        y[2 * i + 1] = __fadd_rn(__fmul_rn(q2, c[i + 4]), __fmul_rn(p2, s[i + 4]));
      }
    }
  }
  // largest magnitudes of the 16-element blocks of the two chunks: the
  // neighbour's chunks when the halves are split (rot / 16 is even), else both
  // chunks are one block
  float ma = 0.f, mb = 0.f;
  if (__any_sync(0xffffffffu, kd.pool == MSA_KV_NVFP4)) {   // the shuffles are warp-wide
    const float pa = amax8(x), pb = amax8(y);
    const float na = __shfl_xor_sync(0xffffffffu, pa, 1);
    const float nb = __shfl_xor_sync(0xffffffffu, pb, 1);
    ma = split ? fmaxf(pa, na) : fmaxf(pa, pb);
    mb = split ? fmaxf(pb, nb) : ma;
  }
  if (!live) return;
  int64_t line;                // destination row
  if (kd.pool < 0) {
    line = (int64_t)t * heads + h;
  } else {
    if (a.loc == nullptr) {
      const int page = ws.block_table[(int64_t)req * a.max_blocks + plan_pos / kBlock];
      slot = page < 0 ? -1 : (int64_t)page * kBlock + plan_pos % kBlock;
    }
    if ((uint64_t)slot >= (uint64_t)a.pool_slots) {
      set_error(ws.hdr, MSA_DEVERR_PAGE_RANGE);
      return;
    }
    int64_t head = (slot >> 7) * heads + h;
    if (kd.pool == MSA_KV_NVFP4) head = 2 * head + kd.fp4_slot;   // a slot each for K and V
    line = head * kBlock + (slot & (kBlock - 1));
  }
  static_assert(kBlock == 128, "slot arithmetic");
  if (kd.pool == MSA_KV_NVFP4) {
    uint8_t* dst = kd.dst + line * kFp4Row;
    uint8_t sa, sb;
    const uint32_t wa = nvfp4_codes8(x, ma, kd.scale, sa), wb = nvfp4_codes8(y, mb, kd.scale, sb);
    reinterpret_cast<uint32_t*>(dst)[ca] = wa;
    reinterpret_cast<uint32_t*>(dst)[cb] = wb;
    if (!split) {
      dst[kHeadDim / 2 + sub] = sa;
    } else if ((sub & 1) == 0) {
      dst[kHeadDim / 2 + ca / 2] = sa;
      dst[kHeadDim / 2 + cb / 2] = sb;
    }
  } else if (kd.pool == MSA_KV_FP8_E4M3) {
    const float g = kd.scale;
    uint2* dst = reinterpret_cast<uint2*>(kd.dst + line * width);
    dst[ca] = make_uint2(e4m3x2_of(x[0], x[1], g) | e4m3x2_of(x[2], x[3], g) << 16,
                         e4m3x2_of(x[4], x[5], g) | e4m3x2_of(x[6], x[7], g) << 16);
    dst[cb] = make_uint2(e4m3x2_of(y[0], y[1], g) | e4m3x2_of(y[2], y[3], g) << 16,
                         e4m3x2_of(y[4], y[5], g) | e4m3x2_of(y[6], y[7], g) << 16);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(kd.dst + line * (2 * width));
    __stcs(dst + ca, pack8(x));
    __stcs(dst + cb, pack8(y));
  }
  // the step's later kernels read the pools with TMA (async proxy)
  if (kd.pool >= 0) asm volatile("fence.proxy.async.global;" ::: "memory");
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
  if (((uintptr_t)ws & 255) != 0 || !aligned16(rope->cos_sin) || !aligned16(idx_cs) ||
      !aligned16(q_out) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (idx_q && !aligned16(idx_q_out)) || (idx_k && !aligned16(idx_k_pages)) ||
      (idx_v && !aligned16(idx_v_pages)))
    return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0) return MSA_OK;
  const int64_t kinds = idx_v ? 5 : (idx_k ? 4 : (idx_q ? 3 : 2));   // row groups past q
  const int64_t rows = Hq + kinds * Hkv;
  if (T * rows >= (int64_t)1 << 31) return MSA_ERR_UNSUPPORTED;      // rows count in 31 bits
  const bool scaled = cfg->kv_dtype != MSA_KV_BF16;
  const int D = cfg->head_dim, di = cfg->index_dim, kv = cfg->kv_dtype;
  auto kind = [](const void* src, int64_t stride, const float* cs, void* dst, int width, int rot,
                 int pool, int fp4_slot, float scale) {
    return Kind{(const __nv_bfloat16*)src, stride, cs, (uint8_t*)dst, width, rot, pool, fp4_slot,
                scale};
  };
  RopeArgs a;
  a.R = FastDiv((uint32_t)rows);
  a.items = (uint32_t)(T * rows);
  a.Hq = cfg->num_q_heads;
  a.Hkv = cfg->num_kv_heads;
  a.max_blocks = cfg->max_blocks_per_req;
  a.interleaved = rope->interleaved != 0;
  a.num_positions = rope->num_positions;
  a.pool_slots = (int64_t)cfg->num_pages * kBlock;
  a.positions = positions;
  a.loc = out_cache_loc;
  a.kinds[0] = kind(q, rope->q_stride, rope->cos_sin, q_out, D, rot, -1, 0, 1.f);
  a.kinds[1] = kind(k, rope->k_stride, rope->cos_sin, k_pages, D, rot, kv, 0,
                    scaled ? cfg->k_scale : 1.f);
  a.kinds[2] = kind(v, rope->v_stride, nullptr, v_pages, D, 0, kv, 1, scaled ? cfg->v_scale : 1.f);
  a.kinds[3] = kind(idx_q, rope->idx_q_stride, idx_cs, idx_q_out, di, idx_rot, -1, 0, 1.f);
  a.kinds[4] = kind(idx_k, rope->idx_k_stride, idx_cs, idx_k_pages, di, idx_rot, MSA_KV_BF16, 0,
                    1.f);
  a.kinds[5] = kind(idx_v, rope->idx_v_stride, nullptr, idx_v_pages, di, 0, MSA_KV_BF16, 0, 1.f);
  const unsigned grid = (a.items + kSlots - 1) / kSlots;
  return launch_pdl(rope_write_kernel, dim3(grid), dim3(kSlots * kRowThreads), 0,
                    (cudaStream_t)stream, view_of(*cfg, ws), a);
}
