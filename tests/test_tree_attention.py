"""msa_tree_attention: attention of draft trees over a cache of any type.

Against the fp64 oracle's textbook attention over the dequantised pools, with
bounds derived from the roundings the kernel makes:

* out is one bf16 rounding of o: half a step, 2^-8 |o|; the probabilities are
  fp16 for P V: 2^-11 of the attention of |v|; values below 2^-14 (bf16 pools)
  keep fp16's subnormal steps, half of 2^-24; a score's error e shifts a
  probability by a factor within e^(2e) (its own and the sum's);
* a score is 128 exact products summed by the tensor cores, 8 accumulations of
  16 products each, every one within 2^-22 of the largest magnitude reached,
  which softmax_scale |q| |k| bounds: e = 8 * 2 * 2^-22 * max |q| |k| scale;
* with e4m3 pools an element of q is off by up to 2^-17 of its row's largest
  (two e4m3 values stand for it): 2^-17 max |q_d| sum |k_d| scale more;
* P V accumulates n / 16 times, 2^-22 each: n / 4 * 2^-24; the sum of n
  probabilities in fp32 is n / 4 per accumulator, 2^-24 each, and merges add less
  than 64 such steps;
* lse is off by e, by that sum and by 2^-22 relative of itself and of exp2 / log2."""
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
KV = ["bf16", "fp8_e4m3", "nvfp4"]


# ------------------------------------------------------------ refusals (CPU)
def _call(cfg, args):
    return ops.lib().msa_tree_attention(ctypes.byref(cfg), *[ctypes.c_void_p(x) for x in args],
                                        None)


def test_refused_on_the_host():
    cfg = config(8, 1, 2, 8, 16, 8)
    good = [256, 16, 16, 16, 8, 256, 16, 16]     # ws q k v mask scratch out lse
    for i in (0, 1, 2, 3, 5, 6, 7):
        assert _call(cfg, good[:i] + [None] + good[i + 1:]) == INVALID, i
    for i, v in ((0, 128), (1, 8), (2, 8), (3, 24), (4, 4), (5, 128), (6, 8), (7, 2)):
        assert _call(cfg, good[:i] + [v] + good[i + 1:]) == INVALID, i
    assert _call(config(8, 1, 2, 8, 16, 8, head_dim=64), good) == UNSUPPORTED
    # softmax_scale * k_scale: 0 or infinite in fp32
    assert _call(config(8, 1, 2, 8, 16, 8, "nvfp4", softmax_scale=1e-30, k_scale=1e-30),
                 good) == INVALID
    assert _call(config(8, 1, 2, 8, 16, 8, "nvfp4", softmax_scale=1e30, k_scale=1e30),
                 good) == INVALID
    # units of work and pool rows are counted in 32 bits
    assert _call(config(8, 8, 65536, 8192, 16, 8), good) == UNSUPPORTED
    assert _call(config(64, 8, 2, 8, 1 << 21, 8), good) == UNSUPPORTED
    # a step of no requests has nothing to do
    assert _call(config(8, 1, 0, 8, 16, 8), good) == 0


def test_scratch_bytes():
    for kv in KV:
        assert msa.tree_attention_scratch_bytes(config(8, 1, 2, 8, 16, 8, kv)) % 256 == 0
    with pytest.raises(msa.MsaError):
        msa.tree_attention_scratch_bytes(config(64, 8, 2, 8, 1 << 21, 8))
    with pytest.raises(msa.MsaError):
        msa.TreeAttention(config(8, 8, 65536, 8192, 16, 8), device="cpu")


def test_binding_refuses_tensors_that_do_not_fit():
    cfg = config(8, 1, 2, 8, 16, 8)
    cpu = torch.zeros((8, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        msa.tree_attention(cfg, cpu, cpu, cpu, cpu, None, cpu, cpu, cpu)
    layer = msa.TreeAttention(cfg, device="cpu", rope=msa.Rope(None))
    with pytest.raises(ValueError):              # a rope needs the step's rows
        layer.run(None, None, None, cpu, None, None)


def test_oracle_tree_attention_of_a_chain_is_the_dense_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 16)), rng.normal(size=(4, 2, 8, 16)), rng.normal(
        size=(4, 2, 8, 16))
    kw = dict(seq_lens=[13, 0, 9], q_lens=[3, 0, 2], block_table=[[2, 0], [-1, -1], [3, 1]], q=q,
              k=k, v=v, num_kv_heads=2, block_size=8, softmax_scale=0.25)
    got = oracle.tree_attention(masks=[1, 3, 7, 1, 3], **kw)
    for a, b in zip(got, oracle.dense_attention(**kw)):
        assert np.allclose(a, b, rtol=1e-13, atol=1e-13)
    # a node that sees the prefix alone
    one = oracle.tree_attention(masks=[1, 3, 0, 0, 3], **kw)
    ref = oracle.tree_attention(**{**kw, "masks": [0], "seq_lens": [11], "q_lens": [1],
                                   "q": q[2:3], "block_table": [[2, 0]]})
    assert not np.allclose(one[0][2], got[0][2])
    assert ref[0].shape == (1, 4, 16)


# ------------------------------------------------------------ parity (GPU)
LENS = [1, 2, 5, 127, 128, 129, 130, 255, 256, 257, 300, 700]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (8, 1), (16, 1), (6, 2), (16, 2)])
def test_small_trees(kv, hq, hkv):
    """Trees of 1 to 7 nodes that end at, before and after a page's end, idle
    requests among them."""
    nodes = [min(L, n) for L, n in zip(LENS, [1, 2, 3, 7, 4, 1, 5, 6, 2, 3, 7, 4])]
    s = Step(hq, hkv, LENS + [0, 0], nodes + [0, 2], kv, seed=hq * 10 + hkv, extra_tokens=3)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,nodes", [(8, 16), (8, 17), (16, 8), (16, 33), (5, 64), (16, 64),
                                      (1, 64), (3, 43)])
def test_large_trees(kv, hq, nodes):
    """From 64 query rows a head to 1024, on both sides of 128 and 256."""
    s = Step(hq, 1, [nodes, nodes + 1, 150, 128 + nodes, 900], [nodes] * 5, kv, width=9,
             seed=nodes)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_trees_of_every_size_in_one_step(kv):
    nodes = [1, 64, 2, 33, 16, 17, 5, 48]
    s = Step(16, 2, [n + 90 * i for i, n in enumerate(nodes)], nodes, kv, width=20, seed=3,
             max_batch=11, max_blocks=9, extra_tokens=5)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,nodes", [(8, 4), (8, 40)])
def test_long_contexts(kv, hq, nodes):
    """Groups that many blocks share: partials of all of them are merged."""
    s = Step(hq, 1, [20000, 7001], [nodes, nodes], kv, seed=5)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_many_requests(kv):
    """More groups than blocks, several in one block's range."""
    rng = np.random.default_rng(6)
    nodes = rng.integers(1, 12, size=90).tolist()
    lens = [int(n + rng.integers(0, 500)) for n in nodes]
    s = Step(32, 4, lens, nodes, kv, seed=6)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_any_mask(kv):
    """Masks that are no trees': nodes that see nothing but the prefix, all, not
    themselves; bits past the last node; rows without any key."""
    rng = np.random.default_rng(7)
    nodes, lens = [4, 64, 20, 5, 1], [4, 64, 90, 700, 1]
    masks = []
    for n in nodes:
        m = [int(rng.integers(0, 1 << 62)) | int(rng.integers(0, 4)) << 62 for _ in range(n)]
        m[0] = 0
        m[-1] = (1 << 64) - 1 if n > 1 else 0
        masks += m
    s = Step(8, 2, lens, nodes, kv, seed=7, masks=masks)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    seen = [m & ((1 << n) - 1) for m, n in zip(masks, [n for n in nodes for _ in range(n)])]
    s.check(d, masks=seen)
    for t in (0, 4, s.T - 1):                    # no prefix, no bits
        assert bool((d.out[t] == 0).all()) and bool(torch.isneginf(d.lse[t]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_without_masks_the_nodes_are_a_chain(kv):
    s = Step(16, 2, [300, 1, 129, 5000, 64], [1, 1, 9, 4, 64], kv, seed=8)
    d = s.attend(mask=False)
    assert msa.check_device_error(d.ws) == 0
    s.check(d, masks=[(2 << i) - 1 for n in s.nodes for i in range(n)])


@pytest.mark.gpu
def test_a_chain_equals_the_dense_decode():
    """Within the roundings of both: the same attention by two kernels."""
    s = Step(16, 2, [300, 4, 129, 6000], [4] * 4, "nvfp4", seed=9)
    d = s.attend(mask=False)
    cfg = config(16, 2, 4, s.cfg.max_blocks_per_req, s.cfg.num_pages, 0, "nvfp4", q_len=4)
    e = msa.DenseAttention(cfg)
    e.run(s.seq_lens, s.block_table, s.q, s.k, s.v)
    assert float((d.out.float() - e.out.float()).abs().max()) <= 2.0 ** -7 * float(
        e.out.float().abs().max())
    assert float((d.lse - e.lse).abs().max()) <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("nodes", [6, 40])
def test_what_a_node_does_not_see_does_not_reach_it(kv, nodes):
    """NaN in a drafted row's keys, then in its values: the nodes that see it
    get NaN, the others keep their bits."""
    s = Step(8, 2, [500, nodes, 130], [nodes] * 3, kv, seed=10, width=4)
    want = s.attend()
    node = 3
    for slot in (0, 1):
        x = (s.k, s.v)[slot]
        keep = x.clone()
        for r in range(3):
            u = s.lens[r] - nodes + node
            page = int(s.block_table[r, u // 128])
            if kv == "nvfp4":
                x[page, 2 + slot, u % 128, 64 + 3] = 0x7f        # dims 48..63 of head 1
            else:
                x.view(torch.uint8).view(*x.shape, -1)[page, 1, u % 128, 50] = 0x7f
                if kv == "bf16":
                    x[page, 1, u % 128, 50] = float("nan")
        d = s.attend()
        assert msa.check_device_error(d.ws) == 0
        sees = torch.tensor([m >> node & 1 == 1 for m in s.masks], device="cuda")
        assert bool(sees.any()) and not bool(sees.all())
        assert torch.equal(d.out[:, :4], want.out[:, :4])
        assert torch.equal(d.out[~sees], want.out[~sees])
        assert torch.equal(d.lse[~sees], want.lse[~sees])
        hit = d.out[sees][:, 4:].isnan()
        if slot == 0:
            assert bool(hit.all()) and bool(d.lse[sees][:, 4:].isnan().all())
        else:
            lo, hi = (48, 64) if kv == "nvfp4" else (50, 51)
            assert bool(hit[..., lo:hi].all())
            assert not bool(hit[..., :lo].any()) and not bool(hit[..., hi:].any())
            assert torch.equal(d.lse, want.lse)
        x.copy_(keep)


@pytest.mark.gpu
def test_an_infinite_value_that_no_other_node_sees():
    """bf16 infinities are beyond fp16: flagged; nodes that do not see them keep
    their bits all the same."""
    s = Step(8, 1, [300], [6], "bf16", seed=11, width=3)
    want = s.attend()
    u = 300 - 6 + 2
    s.v[int(s.block_table[0, u // 128]), 0, u % 128, 9] = float("-inf")
    d = s.attend()
    assert msa.check_device_error(d.ws) == 16
    sees = torch.tensor([m >> 2 & 1 == 1 for m in s.masks], device="cuda")
    assert torch.equal(d.out[~sees], want.out[~sees]) and torch.equal(d.lse, want.lse)
    assert not bool(torch.isfinite(d.out[sees][..., 9]).any())


@pytest.mark.gpu
def test_queries_beyond_fp16():
    """Flagged with NVFP4 pools; with the others they are within the range."""
    s = Step(8, 1, [300], [3], "nvfp4")
    s.q[0, 3, 5] = 1.0e5
    assert msa.check_device_error(s.attend().ws) == 16
    for kv in ("bf16", "fp8_e4m3"):
        s = Step(8, 1, [300], [3], kv)
        s.q[0, 3] *= 2.0 ** 18
        s.q[1, 2] *= 2.0 ** -40
        s.q[2, 1] = 0.0
        d = s.attend()
        assert msa.check_device_error(d.ws) == 0
        s.check(d)


@pytest.mark.gpu
def test_queries_of_very_different_elements():
    """e4m3 pools: rows whose elements span many powers of two, so that the small
    ones lose bits beside the largest."""
    s = Step(16, 2, [700, 130], [9, 30], "fp8_e4m3", seed=23)
    g = torch.Generator(device="cuda").manual_seed(24)
    e = torch.randint(-14, 4, s.q.shape, generator=g, device="cuda")
    s.q.copy_(s.q.float() * torch.exp2(e.float()))
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_an_infinite_query_stays_in_its_row(kv):
    s = Step(8, 2, [900, 30], [5, 20], kv, seed=25)
    want = s.attend()
    s.q[3, 2, 9] = float("inf")
    d = s.attend()
    assert msa.check_device_error(d.ws) == (16 if kv == "nvfp4" else 0)
    clean = torch.ones_like(d.lse, dtype=torch.bool)
    clean[3, 2] = False
    assert not bool(torch.isfinite(d.out[3, 2]).any())
    assert torch.equal(d.out[clean], want.out[clean])
    assert torch.equal(d.lse[clean], want.lse[clean])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_a_nan_query_stays_in_its_row(kv):
    s = Step(8, 2, [3000, 70, 9], [5, 20, 2], kv, seed=12)
    want = s.attend()
    rows = [(0, 1), (7, 7), (26, 0)]
    for t, h in rows:
        s.q[t, h, 17] = float("nan")
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    clean = torch.ones_like(d.lse, dtype=torch.bool)
    for t, h in rows:
        clean[t, h] = False
        assert bool(d.out[t, h].isnan().all()) and bool(d.lse[t, h].isnan())
    assert torch.equal(d.out[clean], want.out[clean])
    assert torch.equal(d.lse[clean], want.lse[clean])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_peaked_and_flat_rows(kv):
    """Scores far apart, and a row of equal scores, over many pages."""
    s = Step(8, 1, [5000], [5], kv, seed=13, q_std=8.0)
    s.q[1, 0] = 0.0
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("L", [900, 30000])
def test_equal_scores_past_24_bits(kv, L):
    """Two keys of the same huge score in different pages have half the weight
    each, where a step of fp32 is more than any bias of the exponent."""
    s = Step(4, 1, [L], [3], kv, seed=14)
    s.q.copy_(torch.where(s.q[:1, :1] < 0, -16384.0, 16384.0).expand_as(s.q))
    sign = s.q[0, 0] < 0
    v = []
    for u in (5, L - 200):
        page = int(s.block_table[0, u // 128])
        if kv == "nvfp4":
            codes = (7 + 8 * sign).to(torch.uint8)
            s.k[page, 0, u % 128, :64] = codes[0::2] + 16 * codes[1::2]
            s.k[page, 0, u % 128, 64:] = 0x7e
        else:
            big = 448.0 if kv == "fp8_e4m3" else 60000.0
            s.k[page, 0, u % 128] = torch.where(sign, -big, big).to(s.k.dtype)
        v.append(s.pools(0)[1][page, 0, u % 128])
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    want = oracle.bf16_round(((v[0] + v[1]) / 2).astype(np.float32))
    got = to_np(d.out)
    # (both halves of the sum are exact in fp32; the sum's rounding may cross a tie)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -24)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_pages_that_the_plan_flagged_are_skipped(kv):
    s = Step(8, 2, [600], [5], kv, seed=15)
    keep = s.block_table.clone()
    s.block_table[0, 2] = 9999
    d = s.attend()
    assert msa.check_device_error(d.ws) == 1
    s.block_table.copy_(keep)
    # the same sequence without that page
    short = s.block_table.clone()
    short[0, 2:4] = keep[0, 3:5]
    s.seq_lens -= 128
    s.block_table.copy_(short)
    want = s.attend()
    for a, b in ((d.out, want.out), (d.lse, want.lse)):
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())


@pytest.mark.gpu
def test_trees_that_are_too_large_are_flagged():
    s = Step(8, 1, [200, 90, 300], [3, 65, 4], masks=[1, 3, 7] + [1] * 65 + [1, 3, 7, 15],
             seed=16)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 64
    assert bool((d.out[3:68] == 0).all()) and bool(torch.isneginf(d.lse[3:68]).all())
    one = Step(8, 1, [200, 90, 300], [3, 64, 4], masks=[1, 3, 7] + [1] * 64 + [1, 3, 7, 15],
               seed=16)
    one.k, one.v, one.block_table = s.k, s.v, s.block_table
    one.q = torch.cat([s.q[:67], s.q[68:]])
    want = one.attend()
    assert torch.equal(d.out[:3], want.out[:3])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_repeats_and_graph_replays_are_bit_equal(kv):
    s = Step(16, 2, [3000, 200, 4500, 20], [20, 8, 5, 20], kv, seed=17)
    d = s.attend()
    torch.cuda.synchronize()
    first = d.out.clone(), d.lse.clone()
    for _ in range(8):
        s.attend(d)
        assert torch.equal(d.out, first[0]) and torch.equal(d.lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.attend(d)
    cu = s.cu.clone()
    for lens, nodes in (([3000, 200, 4500, 20], s.nodes), ([33, 0, 129, 20], [20, 0, 5, 2]),
                        ([0] * 4, [0] * 4), ([3000, 1, 1, 1], [53, 0, 0, 0])):
        s.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        s.cu.copy_(torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32))
        d.out.fill_(5.0)
        graph.replay()
        e = msa.TreeAttention(s.cfg)
        e.out.fill_(5.0)
        s.attend(e)
        torch.cuda.synchronize()
        assert msa.check_device_error(d.ws) == 0
        T = sum(nodes)
        assert torch.equal(d.out, e.out) and torch.equal(d.lse[:T], e.lse[:T])
        assert bool((d.out[T:] == 5.0).all())
    s.cu.copy_(cu)


@pytest.mark.gpu
def test_two_graphs_that_share_their_buffers():
    a, b = (Step(8, 2, lens, nodes, "fp8_e4m3", seed=x, max_blocks=40, extra_pages=e)
            for x, lens, nodes, e in ((30, [5000, 40, 700], [9, 9, 9], 3),
                                      (31, [20, 2900, 7], [20, 1, 6], 25)))
    assert bytes(a.cfg) == bytes(b.cfg)
    for x in (a, b):
        x.want = x.attend()
    d = a.layer()
    graphs = []
    for x in (a, b):
        x.attend(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.attend(d)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        d.out.fill_(7.0)
        graphs[i].replay()
        want = (a, b)[i].want
        assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.gpu
def test_two_calls_at_once():
    steps = [Step(8, 2, [9000, 40, 3000], [5, 5, 5], "bf16", seed=40),
             Step(16, 2, [2500, 6000], [30, 12], "nvfp4", seed=41)]
    want = [s.attend() for s in steps]
    layers = [s.layer() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, d, st in zip(steps, layers, streams):
            s.attend(d, stream=st)
    torch.cuda.synchronize()
    for d, w in zip(layers, want):
        assert msa.check_device_error(d.ws) == 0
        assert torch.equal(d.out, w.out) and torch.equal(d.lse, w.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,pages", [("bf16", 20000), ("nvfp4", 31000)])
def test_pages_past_4_gib(kv, pages):
    s = Step(8, 8, [700], [9], kv, seed=18)
    far = torch.tensor([pages - 1, pages - 1800, pages - 999, pages - 1001, pages - 500,
                        pages - 1872], device="cuda")
    k, v = s.k, s.v
    big = [torch.empty((pages, *k.shape[1:]), dtype=k.dtype, device="cuda")
           for _ in range(1 if kv == "nvfp4" else 2)]
    big = big * 2 if kv == "nvfp4" else big
    for x, y in zip(big, (k, v)):
        x[far] = y[s.block_table[0].long()]
    want = s.attend()
    cfg = config(8, 8, 1, s.cfg.max_blocks_per_req, pages, s.T, kv)
    d = msa.TreeAttention(cfg)
    msa.plan(cfg, s.seq_lens, far.to(torch.int32)[None].contiguous(), d.ws, s.cu)
    msa.tree_attention(cfg, d.ws, s.q, *big, s.mask, d.scratch, d.out, d.lse)
    assert msa.check_device_error(d.ws) == 0
    assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,kv", [("prefill", "bf16"), ("decode", "fp8_e4m3")])
def test_either_mode(mode, kv):
    s = Step(16, 2, [300, 40], [7, 12], kv, seed=19, mode=mode)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
def test_small_trees_over_nvfp4_in_graphs_and_at_once():
    """The kernel of small trees: two graphs on one layer's buffers, and two layers
    on two streams, with trees on both sides of its limit of 64 rows."""
    steps = [Step(8, 2, lens, nodes, "nvfp4", seed=x, max_blocks=45, extra_pages=e)
             for x, lens, nodes, e in ((50, [5000, 40, 700, 3], [9, 16, 1, 3], 3),
                                       (51, [20, 2900, 0, 2801], [17, 4, 0, 8], 3))]
    want = [s.attend() for s in steps]
    for s, w in zip(steps, want):
        assert msa.check_device_error(w.ws) == 0
        s.check(w)
    layers, streams = [s.layer() for s in steps], [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, d, st in zip(steps, layers, streams):
            s.attend(d, stream=st)
    torch.cuda.synchronize()
    for d, w in zip(layers, want):
        assert msa.check_device_error(d.ws) == 0
        assert torch.equal(d.out, w.out) and torch.equal(d.lse, w.lse)
    d, graphs = steps[0].layer(), []
    other = Step(8, 2, [4100, 77, 650, 128], [8, 2, 5, 14], "nvfp4", seed=52, max_blocks=45,
                 extra_pages=10)
    pair = [(steps[0], want[0]), (other, other.attend())]
    assert bytes(steps[0].cfg) == bytes(other.cfg)
    for s, _ in pair:
        s.attend(d)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.attend(d)
    for i in (0, 1, 1, 0, 1, 0, 0):
        d.out.fill_(7.0)
        graphs[i].replay()
        assert torch.equal(d.out, pair[i][1].out) and torch.equal(d.lse, pair[i][1].lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("group,hkv", [(16, 2), (3, 4), (1, 8)])
def test_trees_at_the_limit_of_small_ones(kv, group, hkv):
    """One node fewer than 64 rows a head, exactly, one more; few and many pages."""
    n = 64 // group
    nodes = [n, max(n - 1, 1), min(n + 1, 64), 1, n, min(n + 1, 64)]
    s = Step(group * hkv, hkv, [n, 400, 3000, 1, 6001, 129], nodes, kv, seed=group, width=5)
    d = s.attend()
    assert msa.check_device_error(d.ws) == 0
    s.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
def test_sequences_shorter_than_their_trees_are_flagged(kv):
    s = Step(8, 1, [200, 90, 300], [3, 12, 4], kv, seed=61)
    want = s.attend()
    s.seq_lens[1] = 11
    d = s.attend()
    assert msa.check_device_error(d.ws) == 2
    assert bool((d.out[3:15] == 0).all()) and bool(torch.isneginf(d.lse[3:15]).all())
    for part in (slice(0, 3), slice(15, 19)):
        tol = 2.0 ** -7 * float(want.out[part].float().abs().max())
        assert float((d.out[part].float() - want.out[part].float()).abs().max()) <= tol
    msa.tree_plan(s.cfg, d.ws, s.parents, d.tree_mask, d.positions)
    assert d.tree_mask[3:15].eq(0).all() and d.positions[3:15].eq(-1).all()
    assert d.tree_mask[:3].tolist() == s.masks[:3]
