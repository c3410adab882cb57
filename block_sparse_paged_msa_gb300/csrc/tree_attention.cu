// msa_tree_attention: full-context attention of the nodes of a draft tree over a
// paged cache of bf16, e4m3 or NVFP4 rows.
//
// One warp per (node, query head): 32 keys at a time, a lane a key for the
// scores, a lane four dims for the weighted sum of the values, running maximum
// and sum in fp32.
#include "msa_device.cuh"
#include "tree.cuh"

namespace msa {
namespace {

struct TreeArgs {
  int Hkv, Hq, G, max_blocks, kv;
  float scale, v_scale;
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *v_pool;
  const int64_t* mask;
  __nv_bfloat16* out;
  float* lse;
};

// Eight consecutive dims (chunk c of 16) of a cache row.
__device__ __forceinline__ void row8(const uint8_t* row, int kv, int c, float (&f)[8]) {
  uint32_t h[4];
  if (kv == MSA_KV_BF16) {
    const uint4 w = reinterpret_cast<const uint4*>(row)[c];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(u[i]);
      f[2 * i + 1] = bf16hi(u[i]);
    }
    return;
  }
  if (kv == MSA_KV_FP8_E4M3) {
    const uint2 w = reinterpret_cast<const uint2*>(row)[c];
    h[0] = e4m3x2_to_f16x2((uint16_t)w.x);
    h[1] = e4m3x2_to_f16x2((uint16_t)(w.x >> 16));
    h[2] = e4m3x2_to_f16x2((uint16_t)w.y);
    h[3] = e4m3x2_to_f16x2((uint16_t)(w.y >> 16));
  } else {
    e2m1x8_to_f16x2(reinterpret_cast<const uint32_t*>(row)[c], h);
    const uint32_t s = e4m3_scale_f16x2(row[kHeadDim / 2 + c / 2]);
    for (int i = 0; i < 4; ++i) h[i] = hmul2_u32(h[i], s);
  }
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

__global__ void __launch_bounds__(128) tree_attention_kernel(WsView ws, TreeArgs a) {
  __shared__ float qs[4][kHeadDim];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t item = (int64_t)blockIdx.x * 4 + w;
  const int t = (int)(item / a.Hq), hq = (int)(item % a.Hq), h = hq / a.G;
  if (t >= ws.hdr->num_tokens) return;
  const int r = ws.tok_req[t];
  Tree tr = {0, 0, 0, false};
  if (r >= 0) tr = tree_of(ws, r);
  if (tr.too_large && lane == 0) set_error(ws.hdr, MSA_DEVERR_TREE);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (tr.n > 0) {
    const int node = t - tr.t0;
    uint64_t mask = a.mask ? (uint64_t)a.mask[t] : ~0ull >> (63 - node);
    if (tr.n < 64) mask &= (1ull << tr.n) - 1;
    for (int d = lane; d < kHeadDim; d += 32) qs[w][d] = __bfloat162float(a.q[item * kHeadDim + d]);
    if (a.kv != MSA_KV_BF16)
      for (int d = lane; d < kHeadDim; d += 32)
        if (fabsf(qs[w][d]) >= 65520.f) set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
    __syncwarp();
    const int L = tr.base + tr.n;
    const int rb = a.kv == MSA_KV_BF16 ? 256 : (a.kv == MSA_KV_FP8_E4M3 ? 128 : kFp4Row);
    const int slots = a.kv == MSA_KV_NVFP4 ? 2 : 1;
    for (int u0 = 0; u0 < L; u0 += 32) {
      const int page = ws.block_table[(int64_t)r * a.max_blocks + u0 / kBlock];
      if (page < 0) continue;
      const int64_t at = (((int64_t)page * a.Hkv + h) * slots) * kBlock + u0 % kBlock;
      const int u = u0 + lane;
      const bool seen = u < tr.base || (u < L && (mask >> (u - tr.base) & 1));
      float s = -INFINITY;
      if (seen) {
        s = 0.f;
        const uint8_t* k = a.k_pool + (at + lane) * rb;
        for (int c = 0; c < 16; ++c) {
          float f[8];
          row8(k, a.kv, c, f);
          for (int i = 0; i < 8; ++i) s = fmaf(f[i], qs[w][8 * c + i], s);
        }
        s *= a.scale;
      }
      float mx = s;
      for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m, mx);
      const float p = seen ? expf(s - mn) : 0.f;
      const float al = m == -INFINITY ? 0.f : expf(m - mn);
      if (mn != -INFINITY) {
        m = mn;
        l = l * al;
        for (int i = 0; i < 4; ++i) o[i] *= al;
      }
      l += p;
      const unsigned on = __ballot_sync(0xffffffffu, seen);
      for (int k = 0; k < 32; ++k) {
        if (!(on >> k & 1)) continue;
        const float pk = __shfl_sync(0xffffffffu, p, k);
        float f[8];
        row8(a.v_pool + (at + (slots - 1) * kBlock + k) * rb, a.kv, lane / 2, f);
        for (int i = 0; i < 4; ++i) {
          const float v = f[(lane & 1) * 4 + i];
          o[i] = fmaf(pk, v, o[i]);
          if (fabsf(v) >= 65520.f) set_error(ws.hdr, MSA_DEVERR_FP16_RANGE);
        }
      }
    }
  }
  for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
  reinterpret_cast<uint2*>(a.out + item * kHeadDim)[lane] =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (lane == 0) a.lse[item] = l == 0.f ? -INFINITY : m + logf(l);
}

bool tree_supported(const msa_config& c) {
  return (int64_t)c.max_batch * c.max_blocks_per_req * c.num_kv_heads < (1 << 27) &&
         (int64_t)c.num_pages * c.num_kv_heads < (1 << 24);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" size_t msa_tree_attention_scratch_bytes(const msa_config* cfg) {
  if (check_config(cfg) != MSA_OK || !tree_supported(*cfg)) return 0;
  return 256;
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
  a.scale = cfg->softmax_scale * (bf16 ? 1.f : cfg->k_scale);
  if (!(a.scale * kLog2e > 0.f && a.scale * kLog2e < INFINITY)) return MSA_ERR_INVALID_ARG;
  const int64_t T = max_tokens_of(*cfg);
  if (T <= 0 || cfg->max_batch == 0) return MSA_OK;
  a.Hkv = cfg->num_kv_heads;
  a.Hq = cfg->num_q_heads;
  a.G = a.Hq / a.Hkv;
  a.max_blocks = cfg->max_blocks_per_req;
  a.kv = cfg->kv_dtype;
  a.v_scale = bf16 ? 1.f : cfg->v_scale;
  a.q = (const __nv_bfloat16*)q;
  a.k_pool = (const uint8_t*)k_pages;
  a.v_pool = (const uint8_t*)v_pages;
  a.mask = tree_mask;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  return launch_pdl(tree_attention_kernel, dim3((unsigned)((T * a.Hq + 3) / 4)), dim3(128), 0,
                    (cudaStream_t)stream, view_of(*cfg, ws), a);
}
