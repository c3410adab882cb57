"""msa_tree_plan, msa_tree_verify, msa_tree_commit, and a whole step that verifies
draft trees.  What they return are whole numbers and moved bytes: equal to the
oracle's, but for tokens drawn so near a border that 64 bits decide otherwise
(none in these cases: the borders' distances are checked)."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from block_sparse_paged_msa_gb300 import ops
from oracle_io import to_np
from tree_util import Step, config

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p


# ------------------------------------------------------------ refusals (CPU)
def test_plan_refused_on_the_host():
    cfg, fn = config(8, 1, 2, 8, 16, 8), ops.lib().msa_tree_plan
    good = [256, 4, 8, 8]                        # ws parents mask positions

    def call(c, a):
        return fn(ctypes.byref(c), *[P(x) for x in a], None)

    for i in range(3):
        assert call(cfg, good[:i] + [None] + good[i + 1:]) == INVALID, i
    for i, v in ((0, 128), (1, 2), (2, 4), (3, 4)):
        assert call(cfg, good[:i] + [v] + good[i + 1:]) == INVALID, i
    assert call(config(8, 1, 2, 8, 16, 8, head_dim=64), good) == UNSUPPORTED
    assert call(config(8, 1, 0, 8, 16, 8), good) == 0


def test_verify_refused_on_the_host():
    cfg, fn = config(8, 1, 2, 8, 16, 8), ops.lib().msa_tree_verify
    good = [256, 4, 4, None, 4, 4, 4, 4, 4]      # ws parents tokens probs u uf accepted num out

    def probs(**kw):
        f = {**dict(target=16, draft=None, vocab=100, dtype=0, target_stride=100, draft_stride=0),
             **kw}
        return ops.MsaTreeProbs(*[f[k] for k, _ in ops.MsaTreeProbs._fields_])

    def call(c, a, p):
        a = [P(x) for x in a]
        a[3] = None if p is None else ctypes.byref(p)
        return fn(ctypes.byref(c), *a, None)

    for i in (0, 1, 2, 4, 5, 6, 7, 8):
        assert call(cfg, good[:i] + [None] + good[i + 1:], probs()) == INVALID, i
        assert call(cfg, good[:i] + [130] + good[i + 1:], probs()) == INVALID, i
    assert call(cfg, good, None) == INVALID
    for kw in (dict(target=None), dict(target=18), dict(vocab=0), dict(vocab=-3), dict(dtype=2),
               dict(target_stride=99), dict(draft=16), dict(draft=18, draft_stride=100),
               dict(dtype=1, target=17)):
        assert call(cfg, good, probs(**kw)) == INVALID, kw
    assert call(cfg, good, probs(vocab=1 << 29, target_stride=1 << 29)) == UNSUPPORTED
    assert call(config(8, 1, 0, 8, 16, 8), good, probs()) == 0


def test_commit_refused_on_the_host():
    cfg, fn = config(8, 1, 2, 8, 16, 8), ops.lib().msa_tree_commit

    def arr(*x):
        return (ctypes.c_void_p * len(x))(*x)

    def call(c=cfg, ws=256, acc=4, num=4, n=2, k=arr(16, 32), v=arr(48, 64), ik=None, iv=None):
        return fn(ctypes.byref(c), P(ws), P(acc), P(num), n, k, v, ik, iv, None)

    assert call(ws=None) == call(ws=128) == call(acc=None) == call(acc=2) == call(num=None) == 1
    assert call(num=6) == call(n=-1) == call(k=None) == call(v=None) == INVALID
    assert call(k=arr(16, None)) == call(v=arr(16, 40)) == call(ik=arr(16, 8)) == INVALID
    assert call(iv=arr(None, 16)) == INVALID
    # a pool in one list twice
    assert call(k=arr(16, 16)) == call(v=arr(64, 64)) == call(ik=arr(80, 80)) == INVALID
    assert call(n=0) == 0 and call(c=config(8, 1, 0, 8, 16, 8)) == 0
    with pytest.raises(ValueError):
        msa.tree_commit(cfg, None, None, None, [], [])


@pytest.mark.parametrize("n", [5, 12])
def test_lists_of_pools_that_do_not_fit(n):
    """The lists' tensors are checked together where they are alike, else one by
    one: the same tensors pass, and the others are named."""
    good = [torch.zeros((3, 2, 4, 8), dtype=torch.bfloat16) for _ in range(n)]
    more = torch.zeros((4, 2, 4, 8), dtype=torch.bfloat16)
    args = "pools", (torch.bfloat16, torch.int16), (3, 2, 4, 8), -1
    for pools in (good, tuple(good), good[:1], good + [more], good + [more.view(torch.int16)]):
        assert ops._expect_all(pools, *args).tolist() == [x.data_ptr() for x in pools]
    for bad in (good + [more[:2]], good + [good[0].float()], [good[0].float()], good + [None],
                [None], ["x"], good + [more.transpose(2, 3)], good + [more[:3, :, :, :4]]):
        with pytest.raises(ValueError, match="pools"):
            ops._expect_all(bad, *args)
    with pytest.raises(ValueError, match="pools"):
        ops._expect_all(good, *args[:3], 0)


# ------------------------------------------------------------ oracle pins (CPU)
def test_oracle_masks_by_hand():
    #       0
    #     1   2
    #    3 4   5
    assert oracle.tree_masks([-1, 0, 0, 1, 1, 2]) == [1, 3, 5, 11, 19, 37]
    assert oracle.tree_masks([-1, -1, 1]) == [1, 2, 6]


@pytest.mark.parametrize("drawn", [False, True])
def test_oracle_verification_keeps_the_target_distribution(drawn):
    """Exact expectation: over a grid of random numbers, the first emitted token
    is distributed as the target's row 0, whatever was drafted."""
    p = np.array([0.5, 0.25, 0.125, 0.125])
    q = np.array([0.125, 0.5, 0.25, 0.125])
    n = 16
    grid = (np.arange(n) + 0.5) / n
    total = np.zeros(4)
    pairs = [(a, b) for a in range(4) for b in range(4)] if drawn else [(1, 2)]
    for a, b in pairs:
        weight = q[a] * q[b] if drawn else 1.0
        for u1 in grid:
            for u2 in grid:
                for uf in grid:
                    path, new = oracle.tree_verify([-1, 0, 0], [0, a, b], np.tile(p, (3, 1)),
                                                   np.tile(q, (3, 1)) if drawn else None,
                                                   [0.0, u1, u2], uf)
                    total[new[0]] += weight / n ** 3
    # the grid's own error: a threshold is met within half a cell in each variable
    assert np.abs(total - p).max() <= 3 * 0.5 / n


def test_oracle_commit_moves_in_order():
    pool = np.arange(4 * 1 * 4 * 1).reshape(4, 1, 4, 1)
    oracle.tree_commit(pool, 10, 6, [3, 0, 2], [0, 2, 3, 5], 4)
    # positions 4, 6, 7, 9 -> 4, 5, 6, 7 (page 0 row 0.., position 9 = page 2 row 1)
    assert pool[0, 0, :, 0].tolist() == [0, 2, 3, 9] and pool[2, 0, :, 0].tolist() == [8, 9, 10, 11]


# ------------------------------------------------------------ the plan (GPU)
def _planned(s, d=None):
    d = d or msa.TreeAttention(s.cfg)
    msa.plan(s.cfg, s.seq_lens, s.block_table, d.ws, s.cu)
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 3, 40])
def test_plan(width):
    nodes = [1, 64, 2, 0, 33, 7, 64, 5]
    lens = [1, 64, 1000, 0, 128, 20, 5000, 0]
    s = Step(8, 1, lens, nodes, width=width, seed=width, max_batch=10, extra_tokens=4)
    d = _planned(s)
    d.tree_mask.fill_(9)
    d.positions.fill_(9)
    msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask, d.positions)
    assert msa.check_device_error(d.ws) == 0
    masks, pos = [], []
    for L, n, p in zip(lens, nodes, s.parents_of):
        m = oracle.tree_masks(p)
        masks += m if L else [0] * n
        pos += [L - n + bin(x).count("1") - 1 for x in m] if L else [-1] * n
    assert [m % (1 << 64) for m in d.tree_mask.tolist()] == masks + [9] * 4
    assert d.positions.tolist() == pos + [9] * 4
    again = d.tree_mask.clone()
    d.tree_mask.zero_()
    msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask)
    assert torch.equal(d.tree_mask[:s.T], again[:s.T])


@pytest.mark.gpu
def test_plan_flags_what_is_no_tree():
    s = Step(8, 1, [50, 90, 20], [4, 65, 3], seed=1)
    d = _planned(s)
    for bad in (3, 1, -2, 1 << 30, -(1 << 31)):   # of node 1
        s.parents[1] = bad
        msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask, d.positions)
        assert msa.check_device_error(d.ws) == 64
        assert d.tree_mask[1] == 2 and d.positions[1] == 46
        assert d.tree_mask[0] == 1 and bool((d.tree_mask[4:69] == 0).all())
        assert bool((d.positions[4:69] == -1).all())


# ------------------------------------------------------ the verification (GPU)
class Probs:
    def __init__(self, s, vocab, drawn, dtype=torch.float32, pad=0, seed=1, sharp=3.0, offset=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        T, rng = len(s.parents), np.random.default_rng(seed)
        self.vocab, self.drawn = vocab, drawn

        def rows(x):
            y = torch.zeros(T * (vocab + pad) + offset, dtype=dtype, device="cuda")[offset:]
            y = y.view(T, vocab + pad)
            y.fill_(float("nan"))                # beside the rows: not read
            y[:, :vocab] = torch.softmax(x, dim=1)
            return y[:, :vocab]

        x = torch.randn((T, vocab), generator=g, device="cuda") * sharp
        self.target = rows(x)
        x = x + 0.7 * torch.randn((T, vocab), generator=g, device="cuda")
        self.draft = rows(x) if drawn else None
        best = torch.topk(x, min(vocab, 8), dim=1).indices.tolist()
        dr = self.draft.double().cpu().numpy() if drawn else None
        tokens, t0 = [], 0
        for par in s.parents_of:
            seen = {}
            for i, p in enumerate(par):
                if p < 0:
                    tokens.append(-5)            # a root's token is not read
                    continue
                k = seen[p] = seen.get(p, -1) + 1
                if drawn:
                    w = dr[t0 + p] / dr[t0 + p].sum()
                    tokens.append(int(rng.choice(vocab, p=w)))
                else:
                    tokens.append(best[t0 + p][k % len(best[t0 + p])])
            t0 += len(par)
        self.tokens = torch.tensor(tokens + [0] * (T - len(tokens)), dtype=torch.int32,
                                   device="cuda")
        self.u = torch.rand(T, generator=g, device="cuda")
        self.uf = torch.rand(s.cfg.max_batch, generator=g, device="cuda")

    def run(self, s, d=None):
        d = d or _planned(s)
        for x in (d.accepted, d.num_accepted, d.out_tokens):
            x.fill_(99)
        return d, d.verify(s.parents, self.tokens, self.target, self.u, self.uf, self.draft)

    def check(self, s, got):
        acc, num, out = (x.cpu().numpy() for x in got)
        tgt = self.target.double().cpu().numpy()
        dr = self.draft.double().cpu().numpy() if self.drawn else None
        tok, u, uf, t0 = self.tokens.tolist(), self.u.tolist(), self.uf.tolist(), 0
        for r, (L, n) in enumerate(zip(s.lens, s.nodes)):
            sl = slice(t0, t0 + n)
            t0 += n
            path, new = ([], [])
            if L and n:
                path, new = oracle.tree_verify(s.parents_of[r], tok[sl], tgt[sl],
                                               None if dr is None else dr[sl], u[sl], uf[r])
            assert num[r] == len(path), r
            assert acc[r].tolist() == path + [-1] * (64 - len(path)), r
            assert out[r].tolist() == new + [-1] * (64 - len(new)), (r, path)
        assert np.all(num[len(s.lens):] == 99) and np.all(acc[len(s.lens):] == 99)


TREES = dict(lens=[70, 64, 5, 0, 900, 33, 2], nodes=[1, 64, 5, 0, 20, 33, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("vocab,dtype,pad,offset", [
    (1, torch.float32, 0, 0), (2, torch.float32, 0, 0), (7, torch.bfloat16, 1, 1),
    (31, torch.float32, 5, 2), (257, torch.float32, 0, 1), (1000, torch.bfloat16, 3, 3),
    (4099, torch.float32, 1, 3), (32000, torch.float32, 0, 0), (50001, torch.bfloat16, 0, 0),
    (131072, torch.float32, 64, 0)])
def test_verify(vocab, dtype, pad, offset, drawn):
    for seed in range(3):
        s = Step(8, 1, **TREES, width=3 + seed, seed=seed, max_batch=9, extra_tokens=2)
        p = Probs(s, vocab, drawn, dtype, pad, seed=seed + 10, offset=offset)
        d, got = p.run(s)
        assert msa.check_device_error(d.ws) == 0
        p.check(s, got)


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_many_requests(drawn):
    """Paths of several lengths, drafts that are always and never taken."""
    rng = np.random.default_rng(4)
    nodes = rng.integers(1, 20, size=80).tolist()
    s = Step(8, 1, [n + 5 for n in nodes], nodes, width=2, seed=4)
    p = Probs(s, 3001, drawn, seed=5)
    p.u[::3] = 0.0
    p.u[1::7] = float(np.nextafter(np.float32(1), np.float32(0)))
    p.uf[::4] = 0.0
    p.uf[1::4] = float(np.nextafter(np.float32(1), np.float32(0)))
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 0
    p.check(s, got)
    assert len(set(got[1].tolist())) > 2
    p.u *= 0.01                                  # and long ones
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 0
    p.check(s, got)
    assert int(got[1].max()) > 4


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("batch", [37, 39, 75, 79, 200])
@pytest.mark.parametrize("vocab,dtype,pad", [(5003, torch.float32, 2), (20011, torch.bfloat16, 5),
                                             (66000, torch.float32, 0)])
def test_verify_batches_of_every_cluster_size(batch, vocab, dtype, pad, drawn):
    """Fewer blocks a request take more rounds each, the last ones ragged."""
    rng = np.random.default_rng(batch)
    nodes = rng.integers(1, 6, size=batch).tolist()
    s = Step(8, 1, [n + 5 for n in nodes], nodes, width=2, seed=batch)
    p = Probs(s, vocab, drawn, dtype, pad, seed=vocab)
    p.uf[::5] = float(np.nextafter(np.float32(1), np.float32(0)))
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 0
    p.check(s, got)


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("max_batch", [11, 60, 140])
def test_verify_among_requests_that_have_nothing_to_verify(max_batch, drawn):
    """Clusters of every size that leave at once (no request, an idle one, a tree that
    is too large) beside others that work, again and again."""
    nodes = [3, 0, 70, 6, 0, 1, 12, 90, 2, 0]
    lens = [40, 0, 80, 6, 0, 200, 33, 95, 9, 7]
    s = Step(8, 1, lens, nodes, masks=[1] * sum(nodes), width=2, seed=max_batch,
             max_batch=max_batch)
    p = Probs(s, 40009, drawn, pad=3, seed=max_batch + 1)
    want = None
    for _ in range(20):
        d, got = p.run(s)
        assert msa.check_device_error(d.ws) == 64
        if want is None:
            want = [x.clone() for x in got]
            for r in (1, 2, 4, 7, 9):
                assert got[1][r] == 0 and bool((got[0][r] == -1).all())
                assert bool((got[2][r] == -1).all())
            few = [0 if n > 64 else L for L, n in zip(lens, nodes)]
            s.lens = few
            p.check(s, got)
            s.lens = lens
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
def test_the_same_token_drafted_twice(drawn):
    """Given: the second of two equal siblings has nothing left to stand on.
    Drawn: it is tried against what the first left."""
    s = Step(8, 1, [20], [4], seed=1)
    s.parents_of = [[-1, 0, 0, 0]]
    s.parents.copy_(torch.tensor([-1, 0, 0, 0], dtype=torch.int32))
    p = Probs(s, 50, drawn, seed=3, sharp=1.0)
    p.tokens[1:] = p.tokens[1].clone()
    for u in (0.0, 0.01, 0.3, 0.6, 0.99):
        for uf in (0.0, 0.3, 0.999):
            p.u[1:] = torch.tensor([0.9999, u, u])
            p.uf[:] = uf
            d, got = p.run(s)
            assert msa.check_device_error(d.ws) == 0
            p.check(s, got)


@pytest.mark.gpu
def test_nothing_left_of_the_target():
    """p = q exactly, every draft refused by a random number of 1: the residual is
    empty and the token comes from the target itself."""
    s = Step(8, 1, [20, 30], [3, 3], seed=2)
    s.parents_of = [[-1, 0, 0]] * 2
    s.parents.copy_(torch.tensor([-1, 0, 0] * 2, dtype=torch.int32))
    p = Probs(s, 64, True, seed=6)
    p.target[:] = 1.0 / 64
    p.draft[:] = 1.0 / 64
    p.u[:] = 1.0
    p.uf[:] = torch.tensor([0.5, 0.999])
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 0
    assert got[1].tolist() == [1, 1] and got[2][:, 0].tolist() == [32, 63]
    # the same with given drafts that hold all of the target
    p.draft = None
    p.drawn = False
    p.target[:] = 0.0
    p.target[:, 7] = 1.0
    p.tokens[:] = 7
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 0
    assert got[1].tolist() == [1, 1] and got[2][:, 0].tolist() == [7, 7]


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0.0, float("nan"), float("inf"), -1.0])
def test_rows_that_are_no_distribution(fill):
    """No token is drawn from them; rows that the walk does not reach are not
    looked at."""
    s = Step(8, 1, [20, 30], [2, 3], seed=2, width=1)
    p = Probs(s, 500, False, seed=7)
    p.u[:] = 1.0
    p.target[1] = float("nan")                   # node 1 is not reached
    p.target[2:5] = fill                         # request 1
    d, got = p.run(s)
    assert msa.check_device_error(d.ws) == 128
    # (an infinite weight is above any random number: those drafts stand)
    num = 3 if fill == float("inf") else 1
    assert got[1].tolist() == [1, num]
    assert got[2][1, num - 1] == -1 and 0 <= got[2][0, 0] < 500


@pytest.mark.gpu
def test_tokens_and_trees_that_are_out_of_range():
    s = Step(8, 1, [20, 90], [3, 65], seed=2, width=1)
    p = Probs(s, 500, False, seed=8)
    for bad in (500, -1, 1 << 30, -(1 << 31)):
        p.tokens[1] = bad
        p.u[:] = 0.0
        d, got = p.run(s)
        assert msa.check_device_error(d.ws) == 64
        assert got[1].tolist() == [1, 0] and 0 <= got[2][0, 0] < 500
        assert bool((got[0][1] == -1).all()) and bool((got[2][1] == -1).all())


@pytest.mark.gpu
def test_verify_repeats_replays_and_other_streams():
    s = Step(8, 1, **TREES, width=3, seed=3)
    p = Probs(s, 20011, True, seed=9)
    d, got = p.run(s)
    want = [x.clone() for x in got]
    for _ in range(5):
        _, again = p.run(s, d)
        assert all(torch.equal(a, b) for a, b in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.verify(s.parents, p.tokens, p.target, p.u, p.uf, p.draft)
    p.u.copy_(torch.rand_like(p.u))
    p.uf.copy_(torch.rand_like(p.uf))
    graph.replay()
    torch.cuda.synchronize()
    p.check(s, (d.accepted, d.num_accepted, d.out_tokens))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    d.verify(s.parents, p.tokens, p.target, p.u, p.uf, p.draft, stream=st)
    st.synchronize()
    p.check(s, (d.accepted, d.num_accepted, d.out_tokens))


# ------------------------------------------------------------ the commit (GPU)
def _paths(s, seed):
    rng = np.random.default_rng(seed)
    paths = []
    for n, par in zip(s.nodes, s.parents_of):
        x, path = int(rng.integers(n)) if n else -1, []
        while x >= 0:
            path.append(x)
            x = par[x]
        paths.append(path[::-1])
    return paths


def _lists(s, paths):
    acc = torch.full((s.cfg.max_batch, 64), -1, dtype=torch.int32)
    num = torch.zeros(s.cfg.max_batch, dtype=torch.int32)
    for r, p in enumerate(paths):
        acc[r, :len(p)] = torch.tensor(p, dtype=torch.int32)
        num[r] = len(p)
    return acc.cuda(), num.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "nvfp4"])
@pytest.mark.parametrize("layers,hkv,d", [(1, 1, 64), (3, 2, 128), (50, 2, 0)])
def test_commit(kv, layers, hkv, d):
    s = Step(2 * hkv, hkv, [300, 64, 5, 0, 130, 257, 1], [20, 64, 5, 0, 6, 40, 1], kv, width=3,
             seed=layers, index_dim=d or 64)
    pages = s.cfg.num_pages
    g = torch.Generator(device="cuda").manual_seed(layers)

    def pool(*shape):
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

    if kv == "nvfp4":
        k = v = [pool(pages, 2 * hkv, 128, 72) for _ in range(layers)]
    else:
        n = 256 if kv == "bf16" else 128
        dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        k, v = ([pool(pages, hkv, 128, n).view(dt) for _ in range(layers)] for _ in range(2))
    ik, iv = ([pool(pages, hkv, 128, 2 * d).view(torch.bfloat16) for _ in range(layers)]
              for _ in range(2)) if d else (None, None)
    every = k + (v if kv != "nvfp4" else []) + (ik + iv if d else [])
    want = [x.view(torch.uint8).cpu().numpy().copy() for x in every]
    paths = _paths(s, 5)
    table = to_np(s.block_table)
    for x in want:
        for r, path in enumerate(paths):
            if s.lens[r]:
                oracle.tree_commit(x, s.lens[r], s.nodes[r], table[r], path, 128)
    e = _planned(s)
    msa.tree_commit(s.cfg, e.ws, *_lists(s, paths), k, v, ik, iv)
    assert msa.check_device_error(e.ws) == 0
    for a, b in zip(every, want):
        assert np.array_equal(a.view(torch.uint8).cpu().numpy(), b)


@pytest.mark.gpu
def test_commit_of_lists_that_are_no_paths():
    s = Step(4, 2, [300, 40, 50, 60, 70], [8, 8, 8, 8, 8], seed=2)
    keep = s.k.clone(), s.v.clone()
    for bad, num in (([0, 3, 3], 3), ([0, 5, 2], 3), ([0, 8], 2), ([-1, 2], 2), ([0], -1),
                     ([0, 2], 9), ([0, 2], 1 << 30)):
        acc, n = _lists(s, [[0, 4]] + [[0]] * 4)
        acc[1, :len(bad)] = torch.tensor(bad, dtype=torch.int32)
        n[1] = num
        d = _planned(s)
        msa.tree_commit(s.cfg, d.ws, acc, n, s.k, s.v)
        assert msa.check_device_error(d.ws) == 64
        other = torch.ones(s.cfg.num_pages, dtype=torch.bool, device="cuda")
        other[s.block_table[0][s.block_table[0] >= 0].long()] = False
        for x, y in zip((s.k, s.v), keep):
            assert torch.equal(x.view(torch.int16)[other], y.view(torch.int16)[other])
            page, row = int(s.block_table[0, 2]), (300 - 8) % 128
            assert torch.equal(x[page, :, row + 1], y[page, :, row + 4])
            x.copy_(y)


@pytest.mark.gpu
def test_commit_leaves_pages_that_the_plan_flagged():
    s = Step(4, 2, [130], [6], seed=2)
    keep = s.k.clone()
    page = int(s.block_table[0, 0])
    s.block_table[0, 1] = 5000
    d = _planned(s)
    # positions 124, 126, 129 (flagged): only 126 -> 125 moves
    msa.tree_commit(s.cfg, d.ws, *_lists(s, [[0, 2, 5]]), s.k, s.v)
    assert msa.check_device_error(d.ws) == 1
    keep[page, :, 125] = keep[page, :, 126]
    assert torch.equal(s.k.view(torch.int16), keep.view(torch.int16))


# ------------------------------------------------------------ the step (GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "nvfp4"])
def test_a_whole_step(kv):
    """Two full-attention layers of a step: tree plan, rotation by the nodes'
    depths and store, attention, verification, commit.  Then the same tokens as
    a chain on a second cache: the caches agree byte for byte afterwards, and so
    does what the path's nodes attended to; and the step as one graph."""
    hq, hkv = 8, 2
    s = Step(hq, hkv, [300, 133, 9, 0, 128], [9, 12, 7, 0, 1], kv, width=3, seed=20)
    g = torch.Generator(device="cuda").manual_seed(21)
    inv = 1.0e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = torch.arange(1024, dtype=torch.float64)[:, None] * inv
    rope = msa.Rope(torch.cat([ang.cos(), ang.sin()], dim=1).float().cuda())
    first = msa.TreeAttention(s.cfg, rope=rope)
    second = msa.TreeAttention(s.cfg, rope=rope, share=first)
    pools = [(s.k.clone(), s.v.clone()) for _ in range(2)]
    if kv == "nvfp4":
        pools = [(k, k) for k, _ in pools]
    new = [tuple(torch.randn((s.T, hkv, 128), generator=g, device="cuda").to(torch.bfloat16)
                 for _ in range(2)) for _ in range(2)]
    p = Probs(s, 700, False, seed=22)
    p.u *= 0.02                                  # (most drafts stand)
    before = [tuple(x.clone() for x in kv_) for kv_ in pools]

    def step():
        first.run(s.seq_lens, s.block_table, s.parents, s.q, *pools[0], cu_seqlens_q=s.cu,
                  new_kv=new[0])
        second.run(None, None, None, s.q, *pools[1], new_kv=new[1], planned=True)
        first.verify(s.parents, p.tokens, p.target, p.u, p.uf)
        first.commit([k for k, _ in pools], [v for _, v in pools])

    step()
    torch.cuda.synchronize()
    assert msa.check_device_error(first.ws) == 0
    num, acc = first.num_accepted.tolist(), first.accepted.tolist()
    assert max(num) > 1
    p.check(s, (first.accepted, first.num_accepted, first.out_tokens))
    done = [tuple(x.clone() for x in kv_) for kv_ in pools]
    outs = [first.out.clone(), second.out.clone()]

    # the path as a chain
    pick = [int(s.cu[r]) + i for r in range(5) for i in acc[r][:num[r]]]
    lens = [L - n + m for L, n, m in zip(s.lens, s.nodes, num)]
    cu = torch.tensor([0] + list(np.cumsum(num)), dtype=torch.int32, device="cuda")
    for l, layer in enumerate((first, second)):
        cfg = config(hq, hkv, 5, s.cfg.max_blocks_per_req, s.cfg.num_pages, len(pick), kv)
        one = msa.TreeAttention(cfg, rope=rope)
        kv_ = tuple(x.clone() for x in before[l])
        if kv == "nvfp4":
            kv_ = (kv_[0], kv_[0])
        chain = [i - 1 for m in num for i in range(m)]
        one.run(torch.tensor(lens, dtype=torch.int32, device="cuda"), s.block_table,
                torch.tensor(chain, dtype=torch.int32, device="cuda"), s.q[pick].contiguous(),
                *kv_, cu_seqlens_q=cu, new_kv=[x[pick].contiguous() for x in new[l]])
        assert msa.check_device_error(one.ws) == 0
        got, want = outs[l][pick].float(), one.out.float()
        assert float((got - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
        for r in range(5):
            for u in range(lens[r]):
                page, row = int(s.block_table[r, u // 128]), u % 128
                for a, b in zip(done[l], kv_):
                    assert torch.equal(a.view(torch.uint8)[page, :, row],
                                       b.view(torch.uint8)[page, :, row])

    # the step as one graph, over the cache as it was
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kv_, b in zip(pools, before):
        for x, y in zip(kv_, b):
            x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first.out, outs[0]) and torch.equal(second.out, outs[1])
    for kv_, b in zip(pools, done):
        for x, y in zip(kv_, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
