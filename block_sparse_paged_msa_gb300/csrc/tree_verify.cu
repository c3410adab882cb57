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
// draw in some tens would take a neighbour.  Weights, sums, A and Z are pairs of
// floats (two-sum, about 47 bits).  fp64 has a 60th of the rate here: with no more
// than the sums of warps and the walk in it, its pipe was what bounded the kernel.
//
// Work split.  A cluster of eight blocks per request: each takes a contiguous part
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

constexpr int kVThreads = 512, kVWarps = kVThreads / 32;
constexpr int kMaxC = 8;                       // blocks of a cluster
constexpr int kParts = kMaxC * kVWarps;        // warps of a cluster
constexpr int kMine = kParts / 32;             // of them a lane looks after

struct VerifyArgs {
  const int32_t *parents, *tokens;
  const void *target, *draft;
  int64_t target_stride, draft_stride;
  int32_t vocab;
  const float *uniform, *uniform_final;
  int32_t *accepted, *num, *out;
};

// A number as an unevaluated sum of two floats.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {         // two-sum; lo is left to grow
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
};
__device__ __forceinline__ Pair tidy(float hi, float lo) {         // |lo| to half a step of hi
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  a.add(b.hi);
  return tidy(a.hi, __fadd_rn(a.lo, b.lo));
}
__device__ __forceinline__ Pair operator*(Pair a, float x) {
  const float h = __fmul_rn(a.hi, x);
  return tidy(h, __fmaf_rn(a.lo, x, __fmaf_rn(a.hi, x, -h)));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) {
  return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) < 0.f;
}
__device__ __forceinline__ Pair shfl(Pair a, int l) {
  return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)};
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
// The inclusive prefix sums over the lanes.
__device__ __forceinline__ Pair scan(Pair t, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = shfl_up(t, o);
    if (lane >= o) t = t + y;
  }
  return t;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// max(p - A q, 0).
template <bool DRAWN>
__device__ __forceinline__ Pair weight(float p, float q, Pair A) {
  if (!DRAWN) return {p != p ? p : fmaxf(p, 0.f), 0.f};              // a NaN shows in the sum
  const float h = __fmul_rn(A.hi, q), e = __fmaf_rn(A.hi, q, -h);   // h + e = A.hi q
  const float d = __fsub_rn(p, h), b = __fsub_rn(d, p);             // d + f = p - h
  const float f = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(h, b));
  Pair w = tidy(d, __fsub_rn(f, __fmaf_rn(A.lo, q, e)));
  if (w.hi <= 0.f) w = {0.f, 0.f};
  return w;
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
__global__ void __launch_bounds__(kVThreads) tree_verify_kernel(WsView ws, VerifyArgs a) {
  constexpr int V = 16 / sizeof(T);
  __shared__ Pair sums[2][kParts];
  __shared__ int par[kTreeNodes], tok[kTreeNodes];
  __shared__ float uni[kTreeNodes], pt[kTreeNodes], qt[kTreeNodes];
  __shared__ unsigned long long kids[kTreeNodes];
  __shared__ int gone[kTreeNodes];             // refused tokens of the last node
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / kMaxC, rank = blockIdx.x - r * kMaxC;
  const int part = rank * kVWarps + warp;
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

  // A pass over row x: this warp's part of sum w, then all
  // parts' to all blocks; `buf` alternates.
  int buf = 0;
  const int NVmax = a.vocab / V + 2;           // vectors of a row, its ragged ends included
  const int per = ((NVmax + kParts - 1) / kParts + 31) & ~31;    // of a warp, whole rounds
  auto span = [&](const T* row) { return (int)(((uintptr_t)row / sizeof(T)) & (V - 1)); };
  auto pass = [&](int x, Pair A, int ngone) {
    const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
    const int sh = span(p);                    // vector v: elements V v - sh ..
    const bool qa = DRAWN && span(q) == sh;
    Pair s = {0.f, 0.f};
#pragma unroll (DRAWN ? 4 : 8)
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
        const Pair w = weight<DRAWN>(xp[i], DRAWN ? xq[i] : 0.f, A);
        s.add(w.hi);
        if (DRAWN) s.lo += w.lo;
      }
    }
    Pair t = tidy(s.hi, s.lo);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
      t = t + Pair{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)};
    buf ^= 1;
    if (lane < kMaxC) *cluster.map_shared_rank(&sums[buf][part], lane) = t;
    cluster.sync();
  };
  // Inclusive prefix sums of the parts, the same numbers in every warp: this lane's
  // are kMine from kMine * lane on.
  auto prefix = [&](Pair (&s)[kMine], Pair& total) {
    s[0] = sums[buf][kMine * lane];
#pragma unroll
    for (int i = 1; i < kMine; ++i) s[i] = s[i - 1] + sums[buf][kMine * lane + i];
    const Pair inc = scan(s[kMine - 1], lane), before = shfl_up(inc, 1);
    total = shfl(inc, 31);
    if (lane > 0) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) s[i] = before + s[i];
    }
  };

  int x = 0, len = 1, ngone = 0;
  Pair A = {0.f, 0.f}, Z = {1.f, 0.f}, s[kMine], total = {0.f, 0.f};
  unsigned long long path = 1;
  bool have = false;                           // sums of the current residual are there
  for (;;) {
    unsigned long long m = kids[x];
    int next = -1;
    A = {0.f, 0.f};
    Z = {1.f, 0.f};
    ngone = 0;
    have = false;
    while (m) {
      const int c = __ffsll((long long)m) - 1;
      m &= m - 1;
      Pair w = weight<DRAWN>(pt[c], qt[c], A);
      if (!DRAWN) {
        for (int k = 0; k < ngone; ++k)
          if (gone[k] == tok[c]) w = {0.f, 0.f};
      }
      if (Z * qt[c] * uni[c] < w) {
        next = c;
        break;
      }
      if (DRAWN) {
        A = A + Z;
        pass(x, A, 0);
        prefix(s, total);
        Z = total;
        have = true;
      } else {
        Z = Z + Pair{-w.hi, -w.lo};
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
  if (!have) {
    pass(x, A, ngone);
    prefix(s, total);
  }
  if (total.hi == 0.f && (A.hi != 0.f || ngone > 0)) {           // nothing left: the target itself
    A = {0.f, 0.f};
    ngone = 0;
    pass(x, A, 0);
    prefix(s, total);
  }
  const bool sound = total.hi > 0.f && total.hi < INFINITY;

  // ---- whose part holds the token, and where in it
  const Pair aim = total * a.uniform_final[r];
  // the first part whose prefix passes the aim; uniform_final near 1: the last one
  // with weight
  int mine = kMine, weighty = -1;
  Pair e0 = {0.f, 0.f};                        // the prefix before that part
#pragma unroll
  for (int i = kMine - 1; i >= 0; --i) {
    if (aim < s[i]) mine = i;
    if (weighty < 0 && sums[buf][kMine * lane + i].hi > 0.f) weighty = i;
  }
  const unsigned past = __ballot_sync(0xffffffffu, mine < kMine);
  const unsigned any = __ballot_sync(0xffffffffu, weighty >= 0);
  int owner;
  if (past) {
    const int l = __ffs(past) - 1;
    owner = kMine * l + __shfl_sync(0xffffffffu, mine, l);
  } else {
    const int l = any ? 31 - __clz(any) : 0;
    owner = kMine * l + max(__shfl_sync(0xffffffffu, weighty, l), 0);
  }
  {
    const int before = max(owner - 1, 0);
    Pair v = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (before % kMine == i) v = s[i];
    v = shfl(v, before / kMine);
    if (owner > 0) e0 = v;
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
  // This warp's part once more, from L2: a lane sums the vectors of a stretch of its
  // own, then the stretch that holds the token is gone through, a lane a vector at a
  // time.
  const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
  const int sh = span(p);
  const bool qa = DRAWN && span(q) == sh;
  auto weights = [&](int v, Pair (&w)[V], int& top) {          // of vector v; its last weighty
    const int64_t at = (int64_t)v * V - sh;
    float xp[V], xq[V];
    load_vec<T, V>(p, at, a.vocab, true, xp);
    if (DRAWN) load_vec<T, V>(q, at, a.vocab, qa, xq);
    for (int k = 0; k < ngone; ++k) {
      const int64_t d = gone[k] - at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (d == i) xp[i] = 0.f;
    }
    Pair t = {0.f, 0.f};
    top = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = weight<DRAWN>(xp[i], DRAWN ? xq[i] : 0.f, A);
      t.add(w[i].hi);
      t.lo += w[i].lo;
      if (w[i].hi > 0.f) top = i;
    }
    return tidy(t.hi, t.lo);
  };
  const int each = per / 32;                   // vectors of a lane's stretch
  Pair w[V], t = {0.f, 0.f};
  int top, last = -1;                          // last: the last vector with weight
#pragma unroll 4
  for (int k = 0; k < each; ++k) {
    const int v = part * per + lane * each + k;
    t = t + weights(v, w, top);
    if (top >= 0) last = v;
  }
  Pair inc = scan(t, lane);
  unsigned hit = __ballot_sync(0xffffffffu, aim < e0 + inc);
  unsigned heavy = __ballot_sync(0xffffffffu, last >= 0);
  int l = hit ? __ffs(hit) - 1 : (heavy ? 31 - __clz(heavy) : 0);
  // the sum before stretch l, and its vectors 32 at a time
  Pair run = shfl(inc, max(l - 1, 0));
  run = l > 0 ? e0 + run : e0;
  const int v_last = __shfl_sync(0xffffffffu, last, l);
  const int v0 = part * per + l * each;
  int got = -1;
  for (int k = 0; k < each && got < 0; k += 32) {
    const bool on = k + lane < each;
    t = on ? weights(v0 + k + lane, w, top) : Pair{0.f, 0.f};
    inc = scan(t, lane);
    hit = __ballot_sync(0xffffffffu, on && aim < run + inc);
    if (hit) {
      const int f = __ffs(hit) - 1;
      const Pair b = shfl_up(inc, 1);
      int i_hit = -1;
      if (lane == f) {
        Pair c = lane ? run + b : run;
#pragma unroll
        for (int i = 0; i < V; ++i) {          // the first that passes; else the last with weight
          c = c + w[i];
          if (i_hit < 0 && aim < c) i_hit = i;
        }
        if (i_hit < 0) i_hit = top;
      }
      i_hit = __shfl_sync(0xffffffffu, i_hit, f);
      if (i_hit >= 0) got = (int)((int64_t)(v0 + k + f) * V - sh + i_hit);
      break;
    }
    run = run + shfl(inc, 31);
  }
  if (got < 0 && v_last >= 0) {                // rounding, or uniform_final near 1
    weights(v_last, w, top);
    got = (int)((int64_t)v_last * V - sh + top);
  }
  if (lane == 0) a.out[(int64_t)r * kTreeNodes + len - 1] = got;
}

template <typename T, bool DRAWN>
msa_status launch_verify(const WsView& v, const VerifyArgs& a, int batch, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kMaxC;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)batch * kMaxC);
  lc.blockDim = dim3(kVThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, tree_verify_kernel<T, DRAWN>, v, a) == cudaSuccess
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
