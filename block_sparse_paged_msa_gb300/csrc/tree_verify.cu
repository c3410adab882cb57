// msa_tree_verify: which drafted tokens of a tree stand, against the target's
// probabilities and given random numbers, and the token after them.
//
// Mathematics.  From node x the children are tried in order.  A child y that was
// drawn from q stands with probability min(1, w(y) / (Z q(y))), w / Z being what
// is left of the target p; a refusal leaves w' = max(w - Z q, 0), Z' = sum w'.
// Since w = max(p - A q, 0) with A the sum of the earlier Z, w' = max(p - (A + Z)
// q, 0): the whole state of a node is the number A, and a refusal costs one pass
// over the rows p and q.  A child that is given (q is 1 at y) stands with
// probability w(y) / Z; a refusal takes w(y) out of both, and needs no pass.
// Emitted tokens are distributed as p in both cases.
//
// Precision.  A drawn token is a comparison of prefix sums over up to hundreds
// of thousands of probabilities with a random number: with sums of 24 bits one
// draw in some tens would take a neighbour.  Weights and their sums per thread
// are pairs of floats (two-sum, about 48 bits; an fp64 addition has a 60th of
// the rate here), the few sums of warps fp64.
//
// Work split.  A cluster of kC blocks per request: each takes a contiguous part
// of the vocabulary, its warps contiguous parts of that.  The walk over the tree
// needs single entries only, fetched for all nodes at once; every block walks by
// itself.  Sums of warps are written to all blocks of the cluster through
// distributed shared memory, one cluster barrier a pass; every warp then finds
// by the same arithmetic whose part holds the drawn token, and that warp goes
// through its part again (from L2) for the token itself.
#include <cooperative_groups.h>

#include "msa_device.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kVThreads = 256, kVWarps = kVThreads / 32;
constexpr int kMaxC = 8;                       // blocks of a cluster
constexpr int kMaxParts = kMaxC * kVWarps;     // warps of a cluster

struct VerifyArgs {
  const int32_t *parents, *tokens;
  const void *target, *draft;
  int64_t target_stride, draft_stride;
  int32_t vocab;
  const float *uniform, *uniform_final;
  int32_t *accepted, *num, *out;
};

// A sum of floats as an unevaluated pair.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {         // two-sum
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// max(p - A q, 0) as a pair; A = ah + al.
template <bool DRAWN>
__device__ __forceinline__ void weight(float p, float q, float ah, float al, float& hi, float& lo) {
  if (!DRAWN) {
    hi = fmaxf(p, 0.f);
    if (p != p) hi = p;                        // a NaN shows in the sum
    lo = 0.f;
    return;
  }
  const float h = __fmul_rn(ah, q), e = __fmaf_rn(ah, q, -h);       // h + e = ah q
  const float d = __fsub_rn(p, h), b = __fsub_rn(d, p);             // d + f = p - h
  const float f = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(h, b));
  const float g = __fsub_rn(f, __fmaf_rn(al, q, e));
  const float s = __fadd_rn(d, g);
  lo = __fsub_rn(g, __fsub_rn(s, d));
  hi = s;
  if (s <= 0.f) hi = lo = 0.f;
}

// Up to V consecutive elements from `at` (V of them where it is 16-byte aligned
// and they lie within [0, vocab); others read as 0).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* row, int64_t at, int vocab, bool aligned,
                                         float (&x)[V]) {
  if (aligned && at >= 0 && at + V <= vocab) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (V == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(u[i]);
        x[2 * i + 1] = bf16hi(u[i]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    x[i] = at + i >= 0 && at + i < vocab ? to_f(row[at + i]) : 0.f;
}

template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kVThreads) tree_verify_kernel(WsView ws, VerifyArgs a, int C) {
  constexpr int V = 16 / sizeof(T);
  __shared__ double sums[2][kMaxParts];
  __shared__ int par[kTreeNodes], tok[kTreeNodes];
  __shared__ float uni[kTreeNodes], pt[kTreeNodes], qt[kTreeNodes];
  __shared__ unsigned long long kids[kTreeNodes];
  __shared__ int gone[kTreeNodes];             // refused tokens of the last node
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / C, rank = blockIdx.x - r * C;
  const int part = rank * kVWarps + warp, parts = C * kVWarps;
  griddep_launch_dependents();
  griddep_wait();
  if (r >= ws.hdr->batch) return;              // (the whole cluster, as below)
  const Tree tr = tree_of(ws, r);
  if (tr.n == 0) {
    if (rank == 0) {
      if (tid < kTreeNodes) {
        a.accepted[(int64_t)r * kTreeNodes + tid] = -1;
        a.out[(int64_t)r * kTreeNodes + tid] = -1;
      }
      if (tid == 0) {
        a.num[r] = 0;
        if (tr.too_large) set_error(ws.hdr, MSA_DEVERR_TREE);
      }
    }
    return;
  }
  auto target = [&](int x) { return (const T*)a.target + (tr.t0 + x) * a.target_stride; };
  auto draft = [&](int x) { return (const T*)a.draft + (tr.t0 + x) * a.draft_stride; };
  if (tid < kTreeNodes) kids[tid] = 0;
  __syncthreads();
  if (tid < tr.n) {
    const int p = a.parents[tr.t0 + tid], y = a.tokens[tr.t0 + tid];
    const bool child = p >= 0 && p < tid, known = y >= 0 && y < a.vocab;
    par[tid] = child ? p : -1;
    tok[tid] = y;
    uni[tid] = a.uniform[tr.t0 + tid];
    pt[tid] = child && known ? fmaxf(to_f(target(p)[y]), 0.f) : 0.f;
    qt[tid] = DRAWN && child && known ? to_f(draft(p)[y]) : 1.f;
    if (child) atomicOr(&kids[p], 1ull << tid);
    if (rank == 0 && ((child && !known) || p < -1 || p >= tid)) set_error(ws.hdr, MSA_DEVERR_TREE);
  }
  __syncthreads();

  // A pass over row x: this warp's part of sum w, with A = ah + al, then all
  // parts' to all blocks; `buf` alternates.
  int buf = 0;
  const int NVmax = a.vocab / V + 2;           // vectors of a row, its ragged ends included
  const int per = ((NVmax + parts - 1) / parts + 31) & ~31;      // of a warp, whole rounds
  auto span = [&](const T* row) { return (int)(((uintptr_t)row / sizeof(T)) & (V - 1)); };
  auto pass = [&](int x, float ah, float al, int ngone) {
    const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
    const int sh = span(p);                    // vector v: elements V v - sh ..
    const bool qa = DRAWN && span(q) == sh;
    Pair s = {0.f, 0.f};
#pragma unroll 4
    for (int v0 = part * per; v0 < (part + 1) * per; v0 += 32) {
      const int64_t at = (int64_t)(v0 + lane) * V - sh;
      if ((int64_t)v0 * V - sh >= a.vocab) break;
      float xp[V], xq[V];
      load_vec<T, V>(p, at, a.vocab, true, xp);
      if (DRAWN) load_vec<T, V>(q, at, a.vocab, qa, xq);
      for (int k = 0; k < ngone; ++k) {
        const int64_t d = gone[k] - at;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (d == i) xp[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float hi, lo;
        weight<DRAWN>(xp[i], DRAWN ? xq[i] : 0.f, ah, al, hi, lo);
        s.add(hi);
        if (DRAWN) s.lo += lo;
      }
    }
    double t = s.value();
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    buf ^= 1;
    if (lane < C) *cluster.map_shared_rank(&sums[buf][part], lane) = t;
    cluster.sync();
  };
  // Inclusive prefix sums of the parts, the same numbers in every warp: this
  // lane's parts are 2 lane, 2 lane + 1.
  auto prefix = [&](double& s0, double& s1, double& total) {
    const double a0 = 2 * lane < parts ? sums[buf][2 * lane] : 0.0;
    const double a1 = 2 * lane + 1 < parts ? sums[buf][2 * lane + 1] : 0.0;
    double t = a0 + a1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    total = __shfl_sync(0xffffffffu, t, 31);
    const double before = __shfl_up_sync(0xffffffffu, t, 1);
    s0 = (lane ? before : 0.0) + a0;
    s1 = t;
  };

  int x = 0, len = 1, ngone = 0;
  double A = 0.0, Z = 1.0, s0, s1, total = 0.0;
  unsigned long long path = 1;
  bool have = false;                           // sums of the current residual are there
  for (;;) {
    unsigned long long m = kids[x];
    int next = -1;
    A = 0.0;
    Z = 1.0;
    ngone = 0;
    have = false;
    while (m) {
      const int c = __ffsll((long long)m) - 1;
      m &= m - 1;
      double w;
      if (DRAWN) {
        w = fmax((double)pt[c] - A * (double)qt[c], 0.0);
      } else {
        w = pt[c];
        for (int k = 0; k < ngone; ++k)
          if (gone[k] == tok[c]) w = 0.0;
      }
      if ((double)uni[c] * (double)qt[c] * Z < w) {
        next = c;
        break;
      }
      if (DRAWN) {
        A += Z;
        const float ah = (float)A;
        pass(x, ah, (float)(A - (double)ah), 0);
        prefix(s0, s1, total);
        Z = total;
        have = true;
      } else {
        Z -= w;
        __syncthreads();
        if (tid == 0) gone[ngone] = tok[c];
        ++ngone;
        __syncthreads();
      }
    }
    if (next < 0) break;
    x = next;
    path |= 1ull << x;
    ++len;
  }
  float ah = (float)A, al = (float)(A - (double)ah);
  if (!have) {
    pass(x, ah, al, ngone);
    prefix(s0, s1, total);
  }
  if (total == 0.0 && (A != 0.0 || ngone > 0)) {                 // nothing left: the target itself
    ah = al = 0.f;
    ngone = 0;
    pass(x, 0.f, 0.f, 0);
    prefix(s0, s1, total);
  }
  const bool sound = total > 0.0 && total < INFINITY;

  // ---- whose part holds the token, and where in it
  const double aim = (double)a.uniform_final[r] * total;
  const unsigned b0 = __ballot_sync(0xffffffffu, s0 > aim && 2 * lane < parts);
  const unsigned b1 = __ballot_sync(0xffffffffu, s1 > aim && 2 * lane + 1 < parts);
  int owner = parts;
  if (b0 | b1) {
    const int i0 = b0 ? 2 * (__ffs(b0) - 1) : parts, i1 = b1 ? 2 * (__ffs(b1) - 1) + 1 : parts;
    owner = min(i0, i1);
  } else {                                     // uniform_final near 1: the last part with weight
    const unsigned w0 = __ballot_sync(0xffffffffu, 2 * lane < parts && sums[buf][2 * lane] > 0.0);
    const unsigned w1 =
        __ballot_sync(0xffffffffu, 2 * lane + 1 < parts && sums[buf][2 * lane + 1] > 0.0);
    owner = max(w0 ? 2 * (31 - __clz(w0)) : 0, w1 ? 2 * (31 - __clz(w1)) + 1 : 0);
  }
  if (rank == 0 && warp == 0) {
    // the path, from the root; its nodes' tokens, then the drawn one
    for (int j = lane; j < kTreeNodes; j += 32) {
      const bool on = path >> j & 1ull;
      const int at = __popcll(path & ((1ull << j) - 1ull));
      if (on) a.accepted[(int64_t)r * kTreeNodes + at] = j;
      if (j >= len) a.accepted[(int64_t)r * kTreeNodes + j] = -1;
      if (on && at > 0) a.out[(int64_t)r * kTreeNodes + at - 1] = tok[j];
      if (j >= len) a.out[(int64_t)r * kTreeNodes + j] = -1;
    }
    if (lane == 0) {
      a.num[r] = len;
      if (!sound) {
        a.out[(int64_t)r * kTreeNodes + len - 1] = -1;
        set_error(ws.hdr, MSA_DEVERR_PROBS);
      }
    }
  }
  if (!sound || part != owner) return;
  const double e0 = __shfl_sync(0xffffffffu, owner & 1 ? s0 : s1, owner & 1 ? owner / 2
                                                                             : max(owner / 2 - 1, 0));
  double run = owner == 0 ? 0.0 : e0;          // sum of the parts before
  const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
  const int sh = span(p);
  const bool qa = DRAWN && span(q) == sh;
  int got = -1, last = -1;
  for (int v0 = part * per; v0 < (part + 1) * per; v0 += 32) {
    const int64_t at = (int64_t)(v0 + lane) * V - sh;
    if ((int64_t)v0 * V - sh >= a.vocab) break;
    float xp[V], xq[V];
    load_vec<T, V>(p, at, a.vocab, true, xp);
    if (DRAWN) load_vec<T, V>(q, at, a.vocab, qa, xq);
    for (int k = 0; k < ngone; ++k) {
      const int64_t d = gone[k] - at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (d == i) xp[i] = 0.f;
    }
    double w[V], t = 0.0;
    int top = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float hi, lo;
      weight<DRAWN>(xp[i], DRAWN ? xq[i] : 0.f, ah, al, hi, lo);
      w[i] = (double)hi + (double)lo;
      t += w[i];
      if (hi > 0.f) top = i;
    }
    double inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + inc > aim);
    const unsigned pos = __ballot_sync(0xffffffffu, top >= 0);
    if (pos) {
      const int l = 31 - __clz(pos);
      const int i = __shfl_sync(0xffffffffu, top, l);
      last = (int)((int64_t)(v0 + l) * V - sh + i);
    }
    if (hit) {
      const int l = __ffs(hit) - 1;
      const double before = __shfl_up_sync(0xffffffffu, inc, 1);
      int i_hit = -1;
      if (lane == l) {
        double c = run + (lane ? before : 0.0);
        int i = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {          // the first that passes; else the last with weight
          c += w[k];
          if (i_hit < 0 && c > aim) i_hit = k;
        }
        (void)i;
        if (i_hit < 0) i_hit = top;
      }
      i_hit = __shfl_sync(0xffffffffu, i_hit, l);
      got = i_hit >= 0 ? (int)((int64_t)(v0 + l) * V - sh + i_hit) : last;
      break;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (got < 0) got = last;
  if (lane == 0) a.out[(int64_t)r * kTreeNodes + len - 1] = got;
}

template <typename T, bool DRAWN>
msa_status launch_verify(const WsView& v, const VerifyArgs& a, int batch, cudaStream_t s) {
  const int C = kMaxC;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)batch * C);
  lc.blockDim = dim3(kVThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, tree_verify_kernel<T, DRAWN>, v, a, C) == cudaSuccess
             ? MSA_OK
             : MSA_ERR_CUDA;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_tree_verify(const msa_config* cfg, void* ws, const int32_t* parents,
                                      const int32_t* tokens, const msa_tree_probs* probs,
                                      const float* uniform, const float* uniform_final,
                                      int32_t* accepted, int32_t* num_accepted,
                                      int32_t* out_tokens, msa_stream_t stream) {
  const msa_status st = check_config(cfg);
  if (st != MSA_OK) return st;
  if (!ws || ((uintptr_t)ws & 255) != 0 || !probs) return MSA_ERR_INVALID_ARG;
  if (probs->vocab < 1 || (probs->dtype != 0 && probs->dtype != 1) ||
      probs->target_stride < probs->vocab ||
      (probs->draft && probs->draft_stride < probs->vocab))
    return MSA_ERR_INVALID_ARG;
  if (probs->vocab > (1 << 28)) return MSA_ERR_UNSUPPORTED;
  if (max_tokens_of(*cfg) <= 0 || cfg->max_batch == 0) return MSA_OK;
  if (!parents || !tokens || !probs->target || !uniform || !uniform_final || !accepted ||
      !num_accepted || !out_tokens)
    return MSA_ERR_INVALID_ARG;
  const uintptr_t size = probs->dtype == 0 ? 4 : 2;
  if (((uintptr_t)probs->target | (uintptr_t)probs->draft) & (size - 1)) return MSA_ERR_INVALID_ARG;
  if (((uintptr_t)parents | (uintptr_t)tokens | (uintptr_t)uniform | (uintptr_t)uniform_final |
       (uintptr_t)accepted | (uintptr_t)num_accepted | (uintptr_t)out_tokens) & 3)
    return MSA_ERR_INVALID_ARG;
  VerifyArgs a;
  a.parents = parents;
  a.tokens = tokens;
  a.target = probs->target;
  a.draft = probs->draft;
  a.target_stride = probs->target_stride;
  a.draft_stride = probs->draft_stride;
  a.vocab = probs->vocab;
  a.uniform = uniform;
  a.uniform_final = uniform_final;
  a.accepted = accepted;
  a.num = num_accepted;
  a.out = out_tokens;
  const WsView v = view_of(*cfg, ws);
  cudaStream_t s = (cudaStream_t)stream;
  if (probs->dtype == 0)
    return probs->draft ? launch_verify<float, true>(v, a, cfg->max_batch, s)
                        : launch_verify<float, false>(v, a, cfg->max_batch, s);
  return probs->draft ? launch_verify<__nv_bfloat16, true>(v, a, cfg->max_batch, s)
                      : launch_verify<__nv_bfloat16, false>(v, a, cfg->max_batch, s);
}
