"""Draft trees on the paths that only large steps take: more requests than a block has
threads, several pools a block, several launches of a commit, pools past 4 GiB, trees
of both NVFP4 kernels in one step; and steps of q_len nodes without offsets.  Bounds
as in test_tree_attention.py; what is moved or counted is equal to the oracle's."""
import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from oracle_io import to_np
from test_tree import Probs, _lists, _paths, _planned
from tree_util import Step, config

KV = ["bf16", "fp8_e4m3", "nvfp4"]
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("max_batch,layers,idx", [(64, 61, "kv"), (200, 20, "k"), (100, 95, None)])
def test_commit_of_many_pools(kv, max_batch, layers, idx):
    """Blocks that take every 38th (13th, 25th) pool, pools of every kind among them,
    and lists of more pools than one launch holds."""
    hkv, d = 2, 64
    s = Step(2 * hkv, hkv, [140, 64, 5, 0, 130, 1], [20, 64, 5, 0, 6, 1], kv, width=3,
             seed=layers, index_dim=d, max_batch=max_batch)
    pages = s.cfg.num_pages
    g = torch.Generator(device="cuda").manual_seed(layers)

    def pool(*shape):
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

    if kv == "nvfp4":
        k = v = [pool(pages, 2 * hkv, 128, 72) for _ in range(layers)]
    else:
        k, v = ([pool(pages, hkv, 128, 256).view(torch.bfloat16) for _ in range(layers)]
                for _ in range(2))
    ik, iv = ([pool(pages, hkv, 128, 2 * d).view(torch.bfloat16) for _ in range(layers)]
              if x in (idx or "") else None for x in "kv")
    every = k + (v if kv != "nvfp4" else []) + (ik or []) + (iv or [])
    want = [x.view(torch.uint8).cpu().numpy().copy() for x in every]
    paths = _paths(s, 7)
    assert sum(a != j for p in paths for j, a in enumerate(p)) > 3
    table = to_np(s.block_table)
    for x in want:
        for r, path in enumerate(paths):
            if s.lens[r]:
                oracle.tree_commit(x, s.lens[r], s.nodes[r], table[r], path, 128)
    e = _planned(s)
    msa.tree_commit(s.cfg, e.ws, *_lists(s, paths), k, v, ik, iv)
    assert msa.check_device_error(e.ws) == 0
    for i, (a, b) in enumerate(zip(every, want)):
        assert np.array_equal(a.view(torch.uint8).cpu().numpy(), b), i


def _crowd(seed):
    """1310 requests: short ones of small trees, every seventh of more than 64 query
    rows a head, idle ones at the ends of every 512 and every 640 requests, a long one
    among the last."""
    rng = np.random.default_rng(seed)
    n = 1310
    nodes = rng.integers(1, 4, size=n)
    nodes[::7] = 5
    lens = np.minimum(nodes + rng.integers(0, 120, size=n), 128)
    for end in (512, 640, 1024, 1280):
        lens[end - 4:end + 5] = 0
    nodes[lens == 0] = 0
    lens[1300], nodes[1300] = 6000, 5
    return lens.tolist(), nodes.tolist()


@pytest.mark.parametrize("kv", KV)
def test_more_requests_than_a_block_has_threads(kv):
    lens, nodes = _crowd(3)
    s = Step(32, 2, lens, nodes, kv, width=2, seed=11)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.parametrize("drawn", [False, True])
def test_plan_verify_and_commit_of_many_requests(drawn):
    lens, nodes = _crowd(4)
    s = Step(4, 2, lens, nodes, width=2, seed=12)
    p = Probs(s, 301, drawn, seed=13)
    d = _planned(s)
    msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask, d.positions)
    assert [m % (1 << 64) for m in d.tree_mask.tolist()] == s.masks
    d, got = p.run(s, d)
    assert msa.check_device_error(d.ws) == 0
    p.check(s, got)
    want = s.k.view(torch.uint8).cpu().numpy().copy()
    table = to_np(s.block_table)
    num, acc = d.num_accepted.tolist(), d.accepted.tolist()
    for r, L in enumerate(lens):
        if L:
            oracle.tree_commit(want, L, nodes[r], table[r], acc[r][:num[r]], 128)
    d.commit(s.k, s.v)
    assert msa.check_device_error(d.ws) == 0
    assert np.array_equal(s.k.view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("q_len", [1, 5, 20])
def test_equal_trees_without_offsets(kv, q_len):
    """cfg.q_len nodes a request, an idle one among them, a batch below the largest."""
    lens = [300, q_len, 0, 129, 2000]
    s = Step(8, 2, lens, [q_len] * 5, kv, width=3, seed=q_len, max_batch=7, q_len=q_len,
             extra_tokens=2 * q_len)
    d = s.layer()
    s.cu = None
    msa.plan(s.cfg, s.seq_lens, s.block_table, d.ws)
    msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask, d.positions)
    masks = [0 if 2 * q_len <= t < 3 * q_len else m for t, m in enumerate(s.masks)]
    assert [m % (1 << 64) for m in d.tree_mask[:s.T].tolist()] == masks
    msa.tree_attention(s.cfg, d.ws, s.q, s.k, s.v, d.tree_mask, d.scratch, d.out, d.lse)
    assert msa.check_device_error(d.ws) == 0
    s.check(d)
    p = Probs(s, 401, False, seed=2)
    p.check(s, p.run(s, d)[1])


def test_e4m3_pages_past_4_gib():
    pages, kv = 45000, "fp8_e4m3"
    s = Step(8, 8, [700], [9], kv, seed=18)
    far = torch.tensor([pages - 1, pages - 1800, pages - 999, pages - 1001, pages - 500,
                        pages - 1872], device="cuda")
    big = [torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in (s.k, s.v)]
    for x, y in zip(big, (s.k, s.v)):
        x.view(torch.uint8)[far] = y.view(torch.uint8)[s.block_table[0].long()]
    want = s.attend()
    cfg = config(8, 8, 1, s.cfg.max_blocks_per_req, pages, s.T, kv)
    d = msa.TreeAttention(cfg)
    msa.plan(cfg, s.seq_lens, far.to(torch.int32)[None].contiguous(), d.ws, s.cu)
    msa.tree_attention(cfg, d.ws, s.q, *big, s.mask, d.scratch, d.out, d.lse)
    assert msa.check_device_error(d.ws) == 0
    assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("large", [(40, 20000), (9, 300), (64, 64)])
def test_a_large_nvfp4_tree_beside_many_small_ones(first, large):
    """One request of more than 64 rows a head, the others of fewer, over contexts of
    very different lengths."""
    rng = np.random.default_rng(large[0])
    nodes = rng.integers(1, 9, size=30).tolist()
    lens = [int(n + rng.integers(0, 1 << int(rng.integers(1, 12)))) for n in nodes]
    at = 0 if first else 30
    nodes.insert(at, large[0])
    lens.insert(at, large[1])
    s = Step(16, 2, lens, nodes, "nvfp4", width=4, seed=6)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)
