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
// Work split.  A cluster of blocks per request: each takes a contiguous part of the
// vocabulary, its warps contiguous parts of that.  The walk over the tree needs single
// entries only, fetched for all nodes at once; the first warp of every block walks, all
// alike (sixteen warps that did it took three times as long: their issue slots).  A
// refused given token's siblings of the same token lose their weight before the walk,
// and in a pass the refused tokens are looked for once in several rounds of loads
// (compared with every element they cost as much as the sums).  Sums of warps are
// written to all blocks of the cluster through distributed shared memory, one cluster
// barrier a pass, and one before the first (a block that has not started has no shared
// memory yet; the wait lies behind the nodes' loads, later it costs the same); the first
// warp finds whose part holds the drawn token, and that warp goes through its part again
// (from L2) for the token itself.
//
// What bounds it.  One request of 4 nodes, 32000 tokens: 6.5 us on the GPU, the chain
// header - nodes - their entries - row - barrier - owner's part.  64 requests of 16
// nodes, 131072 tokens (34 MB): 18 us, of them 5 to 7 for the rows (the two-sums' FMA
// pipe).  24 requests with drawn drafts, 100003 tokens: 26 to 29 us, by the paths taken:
// up to five passes of 4.3 us one after the other.
#include <cooperative_groups.h>

#include "msa_device.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kVThreads = 512, kVWarps = kVThreads / 32;

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

// The two halves of a cluster barrier: every thread of the cluster's blocks, once each.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// 16 bytes of probabilities as V numbers.
template <int V>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[V]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (V == 4) {
      x[i] = __uint_as_float(u[i]);
    } else {
      x[2 * i] = bf16lo(u[i]);
      x[2 * i + 1] = bf16hi(u[i]);
    }
  }
}
// V consecutive elements from `at`, one by one; those outside [0, vocab) read as 0.
template <typename T, int V>
__device__ __forceinline__ void load_slow(const T* row, int at, int vocab, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    x[i] = at + i >= 0 && at + i < vocab ? to_f(row[at + i]) : 0.f;
}

// kC blocks a cluster: eight while all clusters are resident at once, fewer for more
// requests (launch_verify).
template <typename T, bool DRAWN, int kC>
__global__ void __launch_bounds__(kVThreads, 2) tree_verify_kernel(WsView ws, VerifyArgs a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kParts = kC * kVWarps;         // warps of a cluster
  constexpr int kMine = kParts / 32;           // of them a lane looks after
  constexpr int kDeep = 16 / V;               // rounds of loads in flight
  __shared__ Pair sums[2][kParts];
  __shared__ int tok[kTreeNodes];
  __shared__ float uni[kTreeNodes], pt[kTreeNodes], qt[kTreeNodes];
  __shared__ unsigned long long kids[kTreeNodes];
  __shared__ int gone[kTreeNodes];             // refused tokens of the last node
  __shared__ struct {                          // what the first warp has the others do
    int row, ngone;                            // a pass over that row; -1: no more
    Pair A;
    int owner, x, len;                         // then the owner's search
    Pair aim, before;
  } todo;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / kC, rank = blockIdx.x - r * kC;
  const int part = rank * kVWarps + warp;
  // this block has started: the others may write to its shared memory
  cluster_arrive();
  griddep_launch_dependents();
  griddep_wait();
  if (r >= ws.hdr->batch) {                    // (the whole cluster, as below)
    cluster_wait();
    return;
  }
  const Tree tr = tree_of(ws, r);
  if (tr.n == 0) {
    cluster_wait();
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
  int parent = -1;
  if (tid < tr.n) {
    const int p = a.parents[tr.t0 + tid], y = a.tokens[tr.t0 + tid];
    const bool child = p >= 0 && p < tid, known = y >= 0 && y < a.vocab;
    if (child) parent = p;
    tok[tid] = y;
    uni[tid] = a.uniform[tr.t0 + tid];
    pt[tid] = child && known ? fmaxf(to_f(target(p)[y]), 0.f) : 0.f;
    qt[tid] = DRAWN && child && known ? to_f(draft(p)[y]) : 1.f;
    if (child) atomicOr(&kids[p], 1ull << tid);
    if (rank == 0 && ((child && !known) || p < -1 || p >= tid)) set_error(ws.hdr, MSA_DEVERR_TREE);
  }
  __syncthreads();
  if (!DRAWN && parent >= 0) {                 // a token that was refused has nothing left
    for (unsigned long long m = kids[parent] & ((1ull << tid) - 1ull); m; m &= m - 1)
      if (tok[__ffsll((long long)m) - 1] == tok[tid]) pt[tid] = 0.f;
  }
  __syncthreads();
  cluster_wait();                              // and so have the others

  // A row in vectors of 16 bytes, aligned ones: vector v holds elements V v - sh ..;
  // 32 of them, a lane each, are a round, and a part has `per` vectors, whole rounds.
  // (vocab is up to 2^28: elements are counted in 32 bits.)
  auto span = [&](const T* row) { return (int)(((uintptr_t)row / sizeof(T)) & (V - 1)); };
  auto per_of = [&](int sh) {
    const int n = (a.vocab + sh + V - 1) / V;
    return ((n + kParts - 1) / kParts + 31) & ~31;
  };
  auto drop = [&](float (&xp)[V], int at, int ngone) {           // the refused tokens
    for (int k = 0; k < ngone; ++k) {
      const int d = gone[k] - at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (d == i) xp[i] = 0.f;
    }
  };
  // whether one of them lies in [lo, hi): few rounds have any
  auto any_gone = [&](int lo, int hi, int ngone) {
    bool in = false;
    for (int k = lane; k < ngone; k += 32) in |= gone[k] >= lo && gone[k] < hi;
    return __any_sync(0xffffffffu, in) != 0;
  };

  // Sums of max(p - A q, 0) as pairs, two elements at a time in packed floats.
  const uint64_t minus = f2(-1.f, -1.f);
  auto less = [&](uint64_t x, uint64_t y) { return fma_f2(y, minus, x); };       // x - y
  struct Sum {
    uint64_t hi, lo;
  };
  auto add = [&](Sum& s, const float (&xp)[V], const float (&xq)[V], Pair A) {
    const uint64_t ah = f2(A.hi, A.hi), nh = f2(-A.hi, -A.hi), nl = f2(-A.lo, -A.lo);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      uint64_t d = f2(xp[i], xp[i + 1]), g = 0;
      float d0, d1;
      if constexpr (DRAWN) {                   // d + g = p - A q (as in weight())
        const uint64_t p = d, q = f2(xq[i], xq[i + 1]);
        const uint64_t h = mul_f2(ah, q), ne = fma_f2(nh, q, h);
        d = less(p, h);
        const uint64_t b = less(d, p);
        const uint64_t f = less(less(p, less(d, b)), add_f2(h, b));
        g = add_f2(f, fma_f2(nl, q, ne));
        float t0, t1, g0, g1;
        f2_split(add_f2(d, g), t0, t1);
        f2_split(d, d0, d1);
        f2_split(g, g0, g1);
        if (t0 <= 0.f) d0 = g0 = 0.f;
        if (t1 <= 0.f) d1 = g1 = 0.f;
        g = f2(g0, g1);
      } else {
        d0 = xp[i] < 0.f ? 0.f : xp[i];        // a NaN shows in the sum
        d1 = xp[i + 1] < 0.f ? 0.f : xp[i + 1];
      }
      d = f2(d0, d1);
      const uint64_t t = add_f2(s.hi, d), b = less(t, s.hi);     // two-sum; lo is left to grow
      s.lo = add_f2(s.lo, add_f2(less(s.hi, less(t, b)), less(d, b)));
      if (DRAWN) s.lo = add_f2(s.lo, g);
      s.hi = t;
    }
  };
  auto joined = [&](const Sum& s) {
    float h0, h1, l0, l1;
    f2_split(s.hi, h0, h1);
    f2_split(s.lo, l0, l1);
    return tidy(h0, l0) + tidy(h1, l1);
  };

  // A pass over row x: this warp's part of sum w, then all
  // parts' to all blocks; `buf` alternates.
  int buf = 0;
  auto pass = [&](int x, Pair A, int ngone) {
    const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
    const int sh = span(p), per = per_of(sh);
    const bool qa = !DRAWN || span(q) == sh;
    // a round that lies within the row, as vectors of both rows
    auto whole = [&](int v0) {
      const int at = v0 * V - sh;
      return qa && at >= 0 && at + 32 * V <= a.vocab;
    };
    Sum s = {0, 0};
    const int from = part * per, to = from + per;
    // kDeep rounds' loads in flight; of others zeros
#pragma unroll 1
    for (int v0 = from; v0 < to; v0 += 32 * kDeep) {
      const int at0 = (v0 + lane) * V - sh;
      if (v0 * V - sh >= a.vocab) break;
      uint4 rp[kDeep], rq[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        rp[u] = rq[u] = make_uint4(0, 0, 0, 0);
        if (v0 + 32 * u < to && whole(v0 + 32 * u)) {
          rp[u] = __ldg(reinterpret_cast<const uint4*>(p + at0 + 32 * V * u));
          if (DRAWN) rq[u] = __ldg(reinterpret_cast<const uint4*>(q + at0 + 32 * V * u));
        }
      }
      const int some = any_gone(v0 * V - sh, v0 * V - sh + 32 * V * kDeep, ngone) ? ngone : 0;
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        float xp[V], xq[V];
        unpack<V>(rp[u], xp);
        unpack<V>(rq[u], xq);
        drop(xp, at0 + 32 * V * u, some);
        add(s, xp, xq, A);
      }
    }
#pragma unroll 1
    for (int v0 = from; v0 < to; v0 += 32) {   // the ragged rounds
      const int at = (v0 + lane) * V - sh;
      if (v0 * V - sh >= a.vocab) break;
      if (whole(v0)) continue;
      float xp[V], xq[V];
      load_slow<T, V>(p, at, a.vocab, xp);
      if (DRAWN) load_slow<T, V>(q, at, a.vocab, xq);
      else unpack<V>(make_uint4(0, 0, 0, 0), xq);
      drop(xp, at, ngone);
      add(s, xp, xq, A);
    }
    Pair t = joined(s);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
      t = t + Pair{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)};
    buf ^= 1;
    if (lane < kC) *cluster.map_shared_rank(&sums[buf][part], lane) = t;
    cluster.sync();
  };
  // Inclusive prefix sums of the parts, the same numbers in every block: this lane's
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

  // The first warp walks (all blocks' alike); the others do the passes that it asks for.
  int x = 0, len = 1, ngone = 0;
  Pair A = {0.f, 0.f}, Z = {1.f, 0.f}, s[kMine], total = {0.f, 0.f};
  unsigned long long path = 1, m = kids[0];
  bool have = false;                           // the last sums are of the residual as it is
  for (bool end = false;;) {
    if (warp == 0) {
      bool need = false;                       // a pass
      while (!need && m && !end) {
        const int c = __ffsll((long long)m) - 1;
        m &= m - 1;
        const Pair w = DRAWN ? weight<DRAWN>(pt[c], qt[c], A) : Pair{pt[c], 0.f};
        if ((DRAWN ? Z * qt[c] * uni[c] : Z * uni[c]) < w) {
          x = c;
          path |= 1ull << x;
          ++len;
          m = kids[x];
          A = {0.f, 0.f};
          Z = {1.f, 0.f};
          have = false;
        } else if (DRAWN) {
          A = A + Z;
          need = have = true;
        } else {
          Z = Z + Pair{-w.hi, -w.lo};
        }
      }
      if (!need && !end) {                     // no child is left
        end = true;
        if (!have) {
          need = true;
          if (!DRAWN) {
            ngone = __popcll(kids[x]);
            for (int j = lane; j < kTreeNodes; j += 32)
              if (kids[x] >> j & 1ull) gone[__popcll(kids[x] & ((1ull << j) - 1ull))] = tok[j];
          }
        }
      }
      if (!need && total.hi == 0.f && (A.hi != 0.f || ngone > 0)) {
        A = {0.f, 0.f};                        // nothing left: the target itself
        ngone = 0;
        need = true;
      }
      if (lane == 0) {
        todo.row = need ? x : -1;
        todo.A = A;
        todo.ngone = ngone;
      }
    }
    __syncthreads();
    const int row = todo.row;
    if (row < 0) break;
    pass(row, todo.A, todo.ngone);             // (a cluster barrier at its end)
    if (warp == 0) {
      prefix(s, total);
      Z = total;
    }
  }
  if (warp == 0) {
    // ---- whose part holds the token
    const bool sound = total.hi > 0.f && total.hi < INFINITY;
    const Pair aim = total * a.uniform_final[r];
    // the first part whose prefix passes the aim; uniform_final near 1: the last one
    // with weight
    int mine = kMine, weighty = -1;
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
    const int before = max(owner - 1, 0);
    Pair v = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (before % kMine == i) v = s[i];
    v = shfl(v, before / kMine);
    if (lane == 0) {
      todo.owner = sound ? owner : -1;
      todo.aim = aim;
      todo.before = owner > 0 ? v : Pair{0.f, 0.f};
      todo.ngone = ngone;
      todo.x = x;
      todo.A = A;
      todo.len = len;
    }
    if (rank == 0) {
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
  }
  __syncthreads();
  if (part != todo.owner) return;
  const Pair aim = todo.aim, e0 = todo.before; // e0: the prefix before the part
  x = todo.x;
  A = todo.A;
  ngone = todo.ngone;
  len = todo.len;
  // This warp's part once more, from L2: a lane sums the vectors of a stretch of its
  // own, then the stretch that holds the token is gone through, a lane a vector at a
  // time.
  const T *p = target(x), *q = DRAWN ? draft(x) : nullptr;
  const int sh = span(p), per = per_of(sh), from = part * per;
  const bool qa = !DRAWN || span(q) == sh;
  if (!any_gone(from * V - sh, (from + per) * V - sh, ngone)) ngone = 0;
  // the elements of vector v, without the refused ones
  auto load = [&](int v, uint4& rp, uint4& rq) {       // zeros unless it is within the rows
    const int at = v * V - sh;
    rp = rq = make_uint4(0, 0, 0, 0);
    const bool in = qa && at >= 0 && at + V <= a.vocab;
    if (in) {
      rp = __ldg(reinterpret_cast<const uint4*>(p + at));
      if (DRAWN) rq = __ldg(reinterpret_cast<const uint4*>(q + at));
    }
    return in;
  };
  auto elements = [&](int v, bool in, const uint4& rp, const uint4& rq, float (&xp)[V],
                      float (&xq)[V]) {
    unpack<V>(rp, xp);
    unpack<V>(rq, xq);
    if (!in) {
      load_slow<T, V>(p, v * V - sh, a.vocab, xp);
      if (DRAWN) load_slow<T, V>(q, v * V - sh, a.vocab, xq);
    }
    drop(xp, v * V - sh, ngone);
  };
  auto weights = [&](int v, Pair (&w)[V], int& top) {          // and the last that is not 0
    uint4 rp, rq;
    float xp[V], xq[V];
    const bool in = load(v, rp, rq);
    elements(v, in, rp, rq, xp, xq);
    Pair t = {0.f, 0.f};
    top = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = weight<DRAWN>(xp[i], xq[i], A);
      t.add(w[i].hi);
      t.lo += w[i].lo;
      if (w[i].hi > 0.f) top = i;
    }
    return tidy(t.hi, t.lo);
  };
  const int each = per / 32;                   // vectors of a lane's stretch
  Sum sum = {0, 0};
#pragma unroll 1
  for (int k = 0; k < each; k += kDeep) {
    const int v = from + lane * each + k;
    uint4 rp[kDeep], rq[kDeep];
    bool in[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) in[u] = load(v + u, rp[u], rq[u]);
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (k + u >= each) continue;             // (loaded, not used)
      float xp[V], xq[V];
      elements(v + u, in[u], rp[u], rq[u], xp, xq);
      add(sum, xp, xq, A);
    }
  }
  Pair inc = scan(joined(sum), lane);
  unsigned hit = __ballot_sync(0xffffffffu, aim < e0 + inc);
  // the sum before the stretch, and its vectors 32 at a time
  const int l = hit ? __ffs(hit) - 1 : 0;
  Pair run = shfl(inc, max(l - 1, 0));
  run = l > 0 ? e0 + run : e0;
  const int v0 = from + l * each, v1 = hit ? v0 + each : from + per;
  Pair w[V];
  int got = -1, top;
  for (int k = 0; hit && k < each; k += 32) {
    const bool on = k + lane < each;
    const Pair t = on ? weights(v0 + k + lane, w, top) : Pair{0.f, 0.f};
    inc = scan(t, lane);
    const unsigned here = __ballot_sync(0xffffffffu, on && aim < run + inc);
    const Pair b = shfl_up(inc, 1);
    if (here) {
      const int f = __ffs(here) - 1;
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
      if (i_hit >= 0) got = (v0 + k + f) * V - sh + i_hit;
      break;
    }
    run = run + shfl(inc, 31);
  }
  // Rounding between the sums, or uniform_final near 1: the last with weight, of the
  // stretch or of the part.
  for (int k = (v1 - v0 - 1) / 32 * 32; got < 0 && k >= 0; k -= 32) {
    top = -1;
    if (v0 + k + lane < v1) weights(v0 + k + lane, w, top);
    const unsigned heavy = __ballot_sync(0xffffffffu, top >= 0);
    if (!heavy) continue;
    const int f = 31 - __clz(heavy);
    got = (v0 + k + f) * V - sh + __shfl_sync(0xffffffffu, top, f);
  }
  if (lane == 0) a.out[(int64_t)r * kTreeNodes + len - 1] = got;
}

template <typename T, bool DRAWN, int kC>
msa_status launch_clusters(const WsView& v, const VerifyArgs& a, int batch, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kC;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)batch * kC);
  lc.blockDim = dim3(kVThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, tree_verify_kernel<T, DRAWN, kC>, v, a) == cudaSuccess
             ? MSA_OK
             : MSA_ERR_CUDA;
}

// Two blocks an SM are resident: the largest clusters of which all are (64 requests of
// 131072 tokens: clusters of four 28 us, of eight in two waves 30, of two 44; 24 of
// 100003, drawn: of eight 28, of four 38).
template <typename T, bool DRAWN>
msa_status launch_verify(const WsView& v, const VerifyArgs& a, int batch, cudaStream_t s) {
  const int resident = 2 * sm_count();
  if (8 * (int64_t)batch <= resident) return launch_clusters<T, DRAWN, 8>(v, a, batch, s);
  if (4 * (int64_t)batch <= resident) return launch_clusters<T, DRAWN, 4>(v, a, batch, s);
  return launch_clusters<T, DRAWN, 2>(v, a, batch, s);
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
