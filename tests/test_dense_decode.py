"""msa_dense_decode: attention over the whole context of an NVFP4 cache.

Against the fp64 oracle's textbook attention over the dequantised pools, with
bounds derived from the roundings the kernel makes:

* out is one bf16 rounding of o: half a step, 2^-8 |o|; the probabilities are
  fp16 for P V: 2^-11 of the attention of |v|; a score's error e shifts a
  probability by a factor within e^(2e) (its own and the sum's);
* a score is 128 exact products summed by the tensor cores, 8 accumulations of
  16 products each, every one within 2^-22 of the largest magnitude reached,
  which softmax_scale |q| |k| bounds: e = 8 * 2 * 2^-22 * max |q| |k| scale;
* lse is off by e, by the fp32 sum of n probabilities (n / 16 of them in each
  thread, 2^-24 each) and by 2^-22 relative of itself and of exp2 / log2."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from block_sparse_paged_msa_gb300 import ops
from block_sparse_paged_msa_gb300 import workloads as wl
from oracle_io import to_np

INVALID, UNSUPPORTED = 1, 2


def _cfg(hq, hkv, batch, blocks, pages, q_len=1, **kw):
    kw = {**dict(kv_dtype="nvfp4", k_scale=0.75, v_scale=0.5), **kw}
    return msa.make_config(num_q_heads=hq, num_kv_heads=hkv, init_blocks=1, local_blocks=2,
                           topk_blocks=4, index_dim=64, max_batch=batch,
                           max_blocks_per_req=blocks, num_pages=pages, q_len=q_len, **kw)


# ------------------------------------------------------------ refusals (CPU)
def test_scratch_bytes_and_unsupported_configs():
    assert msa.dense_decode_scratch_bytes(_cfg(8, 1, 2, 8, 16)) % 256 == 0
    lib = ops.lib()
    for cfg in (_cfg(8, 1, 2, 8, 16, kv_dtype="bf16"), _cfg(8, 1, 2, 8, 16, kv_dtype="fp8_e4m3"),
                _cfg(16, 1, 2, 8, 16, q_len=5), _cfg(8, 1, 2, 8, 16, mode="prefill",
                                                     max_q_tokens=64)):
        assert lib.msa_dense_decode_scratch_bytes(ctypes.byref(cfg)) == 0
        with pytest.raises(msa.MsaError):
            msa.dense_decode_scratch_bytes(cfg)
        with pytest.raises(msa.MsaError):
            msa.DenseAttention(cfg, device="cpu")
    bad = _cfg(8, 1, 2, 8, 16)
    bad.head_dim = 64
    assert lib.msa_dense_decode_scratch_bytes(ctypes.byref(bad)) == 0


def test_refused_on_the_host():
    P, lib, cfg = ctypes.c_void_p, ops.lib(), _cfg(8, 1, 2, 8, 16)
    good = [256, 16, 16, 16, 256, 16, 16]     # ws q k v scratch out lse

    def call(c, args):
        return lib.msa_dense_decode(ctypes.byref(c), *[P(x) for x in args], None)

    for i in range(len(good)):
        assert call(cfg, good[:i] + [None] + good[i + 1:]) == INVALID, i
    for i, v in ((1, 8), (2, 8), (3, 24), (4, 128), (5, 8), (6, 2)):
        assert call(cfg, good[:i] + [v] + good[i + 1:]) == INVALID, i
    assert call(_cfg(8, 1, 2, 8, 16, kv_dtype="bf16"), good) == UNSUPPORTED
    assert call(_cfg(16, 1, 2, 8, 16, q_len=5), good) == UNSUPPORTED
    assert call(_cfg(8, 1, 2, 8, 16, mode="prefill", max_q_tokens=64), good) == INVALID


def test_limits_refused_on_the_host():
    P, lib = ctypes.c_void_p, ops.lib()

    def call(c):
        return lib.msa_dense_decode(ctypes.byref(c), *[P(256)] * 7, None)

    # units (pages x KV heads of the largest step) are counted in 31 bits
    assert call(_cfg(8, 8, 65536, 8192, 16)) == UNSUPPORTED
    # softmax_scale * k_scale: 0 or infinite in fp32
    assert call(_cfg(8, 1, 2, 8, 16, softmax_scale=1e-30, k_scale=1e-30)) == INVALID
    assert call(_cfg(8, 1, 2, 8, 16, softmax_scale=1e30, k_scale=1e30)) == INVALID
    # a config of no requests has nothing to do
    assert call(_cfg(8, 1, 0, 8, 16)) == 0
    assert call(_cfg(8, 1, 0, 8, 16, max_q_tokens=4)) == 0


def test_layouts_of_many_configs_are_not_kept_for_ever():
    for n in range(600):
        ops._layout(_cfg(8, 1, 2, 8, 16 + n))
    assert len(ops._LAYOUTS) <= 256


# ------------------------------------------------------------ oracle pin (CPU)
def test_oracle_dense_attention_is_the_sparse_one_over_every_block():
    spec = wl.small("nvfp4_decode", batch=2, seq_len_range=(300, 700), num_pages=16,
                    topk_blocks=64)
    w = wl.make_workload(spec)
    from oracle_io import run_oracle
    ref = run_oracle(w)
    pool = to_np(w.k_pages).astype(np.uint8)
    kv = oracle.nvfp4_dequant(pool, 128) * spec.kv_scale
    out, lse, mag = oracle.dense_attention(
        seq_lens=to_np(w.seq_lens), q_lens=to_np(w.q_lens), block_table=to_np(w.block_table),
        q=to_np(w.q), k=kv[:, 0::2], v=kv[:, 1::2], num_kv_heads=8, block_size=128,
        softmax_scale=spec.softmax_scale)
    assert np.abs(out - ref["out"]).max() < 1e-12 and np.abs(lse - ref["lse"]).max() < 1e-12
    assert np.all(mag >= np.abs(out))


# ------------------------------------------------------------ parity (GPU)
class Case:
    """A step over an NVFP4 pool of random codes (scales 2^-3 .. 1, both of
    them; pages of no request and rows past each end hold NaN scales)."""

    def __init__(self, hq, hkv, lens, q_len=1, seed=1, max_batch=None, max_blocks=None, q_std=1.0,
                 q_lens=None, extra_pages=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.q_len, self.lens = hq, hkv, q_len, lens
        B = len(lens)
        self.q_lens = [q_len] * B if q_lens is None else q_lens
        nb = [-(-L // 128) for L in lens]
        pages = sum(nb) + extra_pages
        blocks = max_blocks or max(max(nb), 1)
        self.cfg = _cfg(hq, hkv, max_batch or B, blocks, pages, q_len)
        self.pool = torch.randint(0, 256, (pages, 2 * hkv, 128, 72), generator=g, device="cuda",
                                  dtype=torch.uint8)
        self.pool[..., 64:] = torch.randint(0x20, 0x39, (pages, 2 * hkv, 128, 8), generator=g,
                                            device="cuda", dtype=torch.uint8)
        perm = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = np.full((B, blocks), -1, dtype=np.int32)
        used = 0
        for r, n in enumerate(nb):
            table[r, :n] = perm[used:used + n]
            used += n
            if lens[r] % 128:
                self.pool[table[r, n - 1], :, lens[r] % 128:, 64:] = 0x7f
        for p in perm[used:]:
            self.pool[p, :, :, 64:] = 0x7f
        self.block_table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.T = sum(self.q_lens)
        self.cu = None
        if q_lens is not None:
            self.cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32,
                                   device="cuda")
        rows = max(self.T, ops.max_tokens(self.cfg))
        self.q = (q_std * torch.randn((rows, hq, 128), generator=g, device="cuda")).to(
            torch.bfloat16)

    def layer(self):
        d = msa.DenseAttention(self.cfg)
        d.out.fill_(7.0)
        d.lse.fill_(7.0)
        return d

    def run(self, d=None):
        d = d or self.layer()
        d.run(self.seq_lens, self.block_table, self.q, self.pool, self.pool, cu_seqlens_q=self.cu)
        return d

    def check(self, d, heads=None):
        """heads: the KV heads to check (None: all)."""
        c, G = self.cfg, self.hq // self.hkv
        T = self.T
        pool = self.pool.cpu().numpy()
        out_all, lse_all = to_np(d.out), to_np(d.lse)
        assert np.all(out_all[T:] == 7.0) and np.all(lse_all[T:] == 7.0)
        for h in range(self.hkv) if heads is None else heads:
            k = np.nan_to_num(oracle.nvfp4_dequant(pool[:, 2 * h:2 * h + 1], 128)) * c.k_scale
            v = np.nan_to_num(oracle.nvfp4_dequant(pool[:, 2 * h + 1:2 * h + 2], 128)) * c.v_scale
            rows = slice(h * G, (h + 1) * G)
            q = to_np(self.q[:T, rows])
            out, lse, mag = oracle.dense_attention(
                seq_lens=self.lens, q_lens=self.q_lens, block_table=to_np(self.block_table),
                q=q, k=k, v=v, num_kv_heads=1, block_size=128, softmax_scale=c.softmax_scale)
            top = np.sqrt((k ** 2).sum(-1)).max() * np.sqrt((q ** 2).sum(-1)) * c.softmax_scale
            e = 16 * 2.0 ** -22 * top + 2.0 ** -21
            n = max(max(self.lens), 1)
            tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2 * e + (n / 16 + 64) * 2.0 ** -24
                                             )[..., None] * mag
            err = np.abs(out_all[:T, rows] - out)
            assert np.all(err <= tol), (h, float((err - tol).max()))
            fin = np.isfinite(lse)
            got = lse_all[:T, rows]
            assert np.array_equal(got[~fin], lse[~fin])
            lt = (e + (n / 16 + 64) * 2.0 ** -24)[fin] + 2.0 ** -22 * np.abs(lse[fin])
            assert np.all(np.abs(got[fin] - lse[fin]) <= lt), np.abs(got[fin] - lse[fin]).max()


LENS = [1, 2, 127, 128, 129, 255, 256, 257, 31, 33, 700]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (5, 1), (1, 1), (6, 2), (32, 4), (8, 8)])
def test_one_new_token(hq, hkv):
    c = Case(hq, hkv, LENS + [0], seed=hq * 10 + hkv)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 2), (8, 1, 3), (16, 2, 4), (16, 1, 2), (16, 1, 3),
                                          (16, 1, 4), (5, 1, 3), (1, 1, 4), (12, 1, 4),
                                          (3, 1, 21)])
def test_several_new_tokens(hq, hkv, q_len):
    lens = [max(L, q_len) for L in LENS] + [0, 130, 128 + q_len - 1]
    c = Case(hq, hkv, lens, q_len=q_len, seed=q_len)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,q_len,L", [(8, 1, 1, 40000), (16, 2, 1, 100001), (16, 1, 4, 30011)])
def test_one_long_request_split_over_the_machine(hq, hkv, q_len, L):
    c = Case(hq, hkv, [L], q_len=q_len, q_std=3.0, seed=L)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [33, 1100])
def test_many_requests(batch):
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 400, batch)]
    lens[5] = lens[-1] = 0
    c = Case(4, 2, lens, seed=batch, max_batch=batch + 7)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    c.check(d)


@pytest.mark.gpu
def test_empty_steps():
    c = Case(8, 2, [0, 0, 0])
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    assert bool((d.out == 0).all()) and bool(torch.isneginf(d.lse).all())
    # a batch of no request writes nothing
    d = c.layer()
    d.run(c.seq_lens[:0], c.block_table[:0], c.q, c.pool, c.pool)
    assert bool((d.out == 7).all()) and bool((d.lse == 7).all())


@pytest.mark.gpu
def test_a_single_key_gives_its_value():
    c = Case(16, 2, [1, 1], seed=3)
    d = c.run()
    v = oracle.nvfp4_dequant(c.pool.cpu().numpy(), 128) * c.cfg.v_scale
    table = to_np(c.block_table)
    for r in range(2):
        for h in range(2):
            want = oracle.bf16_round(v[table[r, 0], 2 * h + 1, 0].astype(np.float32))
            assert np.array_equal(to_np(d.out[r, 8 * h:8 * h + 8]), np.tile(want, (8, 1)))


@pytest.mark.gpu
def test_flagged_pages_are_skipped():
    """A page outside the pool is left out of the attention; with none left the
    row is empty."""
    c = Case(8, 1, [500, 100, 300], seed=4)
    bad = c.block_table.clone()
    bad[0, 1] = c.cfg.num_pages
    bad[1, 0] = -5
    d = c.layer()
    d.run(c.seq_lens, bad, c.q, c.pool, c.pool)
    assert msa.check_device_error(d.ws) == 1
    assert bool((d.out[1] == 0).all()) and bool(torch.isneginf(d.lse[1]).all())
    kv = np.nan_to_num(oracle.nvfp4_dequant(c.pool.cpu().numpy(), 128))
    k = np.concatenate([kv[p, 0] for p in to_np(c.block_table)[0, [0, 2, 3]]])[:500 - 128] * 0.75
    v = np.concatenate([kv[p, 1] for p in to_np(c.block_table)[0, [0, 2, 3]]])[:500 - 128] * 0.5
    out, lse = oracle.attention(to_np(c.q[0]), k, v, c.cfg.softmax_scale)
    assert np.abs(to_np(d.lse[0]) - lse).max() <= 1e-4
    assert np.abs(to_np(d.out[0]) - out).max() <= 2.0 ** -8 * np.abs(out).max() + 2.0 ** -10 * 3
    good = c.run()
    assert torch.equal(good.out[2], d.out[2])


@pytest.mark.gpu
def test_a_draft_tokens_nan_reaches_only_tokens_that_see_it():
    """NaN scales in the last token's own K or V row: earlier tokens of the
    request do not see it, and neither do other requests."""
    for slot in (0, 1):
        c = Case(8, 1, [133, 260, 129], q_len=4, seed=6)
        clean = c.run()
        page = int(c.block_table[0, 1])
        c.pool[page, slot, 132 - 128, 64 + 3] = 0x7f
        d = c.run()
        assert torch.equal(d.out[:3], clean.out[:3]) and torch.equal(d.lse[:3], clean.lse[:3])
        assert torch.equal(d.out[4:], clean.out[4:])
        hit = torch.isnan(d.out[3].float())
        assert bool(hit[:, 48:64].all())
        if slot == 0:
            assert bool(hit.all()) and bool(torch.isnan(d.lse[3]).all())
        else:
            assert not bool(hit[:, :48].any()) and not bool(hit[:, 64:].any())
            assert torch.equal(d.lse[3], clean.lse[3])


@pytest.mark.gpu
def test_request_with_too_many_tokens_is_flagged():
    """Through cu_seqlens_q a request may bring fewer tokens than q_len (none
    among them); more are refused, on the device."""
    c = Case(8, 2, [200, 300, 150, 90], q_len=2, q_lens=[1, 2, 0, 2], seed=8)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    c.check(d)
    bad = torch.tensor([0, 1, 4, 4, 5], dtype=torch.int32, device="cuda")
    d = c.layer()
    d.run(c.seq_lens, c.block_table, c.q, c.pool, c.pool, cu_seqlens_q=bad)
    assert msa.check_device_error(d.ws) == 2
    assert bool((d.out[1:4] == 0).all()) and bool(torch.isneginf(d.lse[1:4]).all())
    assert bool((d.out[5:] == 7).all())


@pytest.mark.gpu
def test_queries_beyond_fp16_are_flagged():
    c = Case(8, 1, [300])
    c.q[0, 3, 5] = 1.0e5
    d = c.run()
    assert msa.check_device_error(d.ws) == 16


@pytest.mark.gpu
def test_one_very_likely_key_among_many():
    """Scores far apart: a peak 40 above the rest, and a row of equal scores."""
    c = Case(8, 1, [5000], seed=9, q_std=8.0)
    c.q[0, 0] = 0.0
    d = c.run()
    c.check(d)


@pytest.mark.gpu
def test_repeats_and_graph_replays_are_bit_equal():
    """One captured call over the largest step; replayed for smaller batches and
    other lengths in the same buffers it equals eager calls bit for bit."""
    big = Case(16, 2, [3000, 2000, 4500, 2], q_len=2, seed=10)
    d = big.run()
    torch.cuda.synchronize()
    first = d.out.clone(), d.lse.clone()
    for _ in range(8):
        big.run(d)
        assert torch.equal(d.out, first[0]) and torch.equal(d.lse, first[1])
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        big.run(d)
    torch.cuda.current_stream().wait_stream(st)
    for lens in ([3000, 2000, 4500, 2], [17, 0, 129, 4500], [0, 0, 0, 0], [2, 2, 2, 2]):
        big.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        table = big.block_table.clone()
        if lens[3] > 2:
            table[3] = big.block_table[2]
            big.block_table.copy_(table)
        d.out.fill_(5.0)
        graph.replay()
        eager = msa.DenseAttention(big.cfg)
        big.run(eager)
        torch.cuda.synchronize()
        assert msa.check_device_error(d.ws) == 0
        assert torch.equal(d.out, eager.out) and torch.equal(d.lse, eager.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,q_len,L", [(8, 1, 1, 900), (16, 1, 1, 70000), (8, 1, 4, 5000),
                                            (16, 1, 4, 300)])
def test_scores_past_24_bits(hq, hkv, q_len, L):
    """Scores of 10^8, where a step of fp32 is more than any bias of the exponent.
    The first key is 2688 in every dim, with the signs of q; no other is larger
    than 6 there, so that this key has all the weight and the output is its
    value, rounded once.  Every row has a magnitude of its own: the rounding of
    its score, up to half a step, must not reach the weight."""
    c = Case(hq, hkv, [L], q_len=q_len, seed=21)
    c.q.copy_(torch.sign(c.q.float()) * 16384.0)
    c.q[c.q == 0] = 16384.0
    size = 16384.0 + 128.0 * torch.arange(c.T * hq, device="cuda").view(c.T, hq, 1)
    c.q.copy_(torch.sign(c.q[:1, :1].float()) * size)      # multiples of 2^7: bf16
    page = int(c.block_table[0, 0])
    sign = (to_np(c.q[0, 0]) < 0).astype(np.uint8)
    codes = 7 + 8 * sign                                   # +-6
    c.pool[page, 0, 0, :64] = torch.from_numpy(codes[0::2] + 16 * codes[1::2]).cuda()
    c.pool[page, 0, 0, 64:] = 0x7e                         # 448
    d = c.run()
    torch.cuda.synchronize()
    assert msa.check_device_error(d.ws) == 0
    v = oracle.nvfp4_dequant(c.pool[page].cpu().numpy()[None], 128)[0] * c.cfg.v_scale
    want = oracle.bf16_round(v[1, 0].astype(np.float32))
    got = to_np(d.out)
    assert np.array_equal(got, np.broadcast_to(want, got.shape))
    top = 128 * to_np(size)[..., 0] * 2688 * c.cfg.k_scale * c.cfg.softmax_scale
    # the score's products and sums, the scale and its rounding, ln 2's: 2^-24 each
    assert np.all(np.abs(to_np(d.lse) - top) <= (128 + 4) * 2.0 ** -24 * top)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,L", [(8, 900), (16, 70000)])
def test_equal_scores_past_24_bits(hq, L):
    """Two keys of the same huge score, in different pages (of one range, and of
    two that are merged), have half the weight each."""
    c = Case(hq, 1, [L], seed=22)
    size = 16384.0 + 128.0 * torch.arange(hq, device="cuda").view(1, hq, 1)
    c.q.copy_(torch.sign(c.q[:1, :1].float()) * size)
    sign = (to_np(c.q[0, 0]) < 0).astype(np.uint8)
    codes = torch.from_numpy((7 + 8 * sign)[0::2] + 16 * (7 + 8 * sign)[1::2]).cuda()
    v = []
    for u in (5, L - 200):
        page = int(c.block_table[0, u // 128])
        c.pool[page, 0, u % 128, :64] = codes
        c.pool[page, 0, u % 128, 64:] = 0x7e
        v.append(oracle.nvfp4_dequant(c.pool[page].cpu().numpy()[None], 128)[0, 1, u % 128])
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    want = oracle.bf16_round(((v[0] + v[1]) / 2 * c.cfg.v_scale).astype(np.float32))
    got = to_np(d.out)
    assert np.array_equal(got, np.broadcast_to(want, got.shape))


@pytest.mark.gpu
def test_two_graphs_that_share_their_buffers():
    """Two captured steps of one layer's buffers (workspace, scratch, output),
    replayed in any order on one stream."""
    a, b = (Case(8, 2, lens, seed=s, max_blocks=40, extra_pages=e) for s, lens, e in
            ((30, [5000, 40, 700], 3), (31, [3, 2900, 1], 25)))
    assert bytes(a.cfg) == bytes(b.cfg)
    for x in (a, b):
        x.want = x.run()
    d = a.layer()
    graphs = []
    for x in (a, b):
        x.run(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(d)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        d.out.fill_(7.0)
        graphs[i].replay()
        want = (a, b)[i].want
        assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.gpu
def test_another_stream():
    c = Case(8, 2, [5000, 40])
    want = c.run()
    torch.cuda.synchronize()
    d, st = c.layer(), torch.cuda.Stream()
    torch.cuda.synchronize()
    d.run(c.seq_lens, c.block_table, c.q, c.pool, c.pool, stream=st)
    st.synchronize()
    assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.gpu
def test_two_calls_at_once():
    """Two layers with their own buffers on two streams."""
    cases = [Case(8, 2, [9000, 40, 3000], seed=40), Case(16, 2, [2500, 6000], q_len=3, seed=41)]
    want = [c.run() for c in cases]
    layers = [c.layer() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(6):
        for c, d, st in zip(cases, layers, streams):
            d.run(c.seq_lens, c.block_table, c.q, c.pool, c.pool, stream=st)
    torch.cuda.synchronize()
    for d, w in zip(layers, want):
        assert msa.check_device_error(d.ws) == 0
        assert torch.equal(d.out, w.out) and torch.equal(d.lse, w.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (16, 2, 2)])
def test_a_nan_query_stays_in_its_row(hq, hkv, q_len):
    c = Case(hq, hkv, [6000, 70, 1 + q_len], q_len=q_len, seed=42)
    want = c.run()
    rows = [(0, 1), (q_len, hq - 1), (2 * q_len, 0)]
    for t, h in rows:
        c.q[t, h, 17] = float("nan")
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    clean = torch.ones_like(d.lse, dtype=torch.bool)
    for t, h in rows:
        clean[t, h] = False
        assert bool(d.out[t, h].isnan().all()) and bool(d.lse[t, h].isnan())
    assert torch.equal(d.out[clean], want.out[clean])
    assert torch.equal(d.lse[clean], want.lse[clean])


@pytest.mark.gpu
def test_a_captured_step_of_growing_requests():
    """One graph of rotate, append, attend; between replays the requests grow by
    a token each, across page ends, in the same buffers."""
    c = Case(8, 2, [126, 255, 1, 700], seed=43, max_blocks=8)
    free = c.cfg.num_pages - sum(-(-n // 128) for n in c.lens)
    assert free == 3                                 # the pages the first three grow into
    spare = sorted(set(range(c.cfg.num_pages)) - set(c.block_table[c.block_table >= 0].tolist()))
    table = c.block_table.clone()
    table[0, 1], table[1, 2], table[2, 1] = spare
    c.pool[spare, :, :, 64:] = 0x30
    tab = torch.randn((1024, 64), device="cuda").clamp(-1, 1)
    g = torch.Generator(device="cuda").manual_seed(44)
    new = [torch.randn((4, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
           for _ in range(2)]
    d = msa.DenseAttention(c.cfg, rope=msa.Rope(tab, interleaved=True))
    e = msa.DenseAttention(c.cfg, rope=msa.Rope(tab, interleaved=True))
    pool2 = c.pool.clone()

    def step(layer, pool):
        layer.run(c.seq_lens, table, c.q, pool, pool, new_kv=new)

    step(d, c.pool)                                  # the first step, eagerly on both
    step(e, pool2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, c.pool)
    for _ in range(6):
        c.seq_lens += 1
        for x in (*new, c.q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))
        graph.replay()
        step(e, pool2)
        torch.cuda.synchronize()
        assert msa.check_device_error(d.ws) == 0 and msa.check_device_error(e.ws) == 0
        assert torch.equal(d.out, e.out) and torch.equal(d.lse, e.lse)
        assert torch.equal(c.pool, pool2)


@pytest.mark.gpu
def test_pages_past_4_gib():
    """Pages whose byte offset in the pool passes 2^32."""
    c = Case(8, 8, [700], seed=12)
    pages = 31000                                  # 147456 bytes each
    pool = torch.empty((pages, 16, 128, 72), dtype=torch.uint8, device="cuda")
    far = torch.tensor([30999, 29200, 30001, 29999, 30500, 29128], device="cuda")
    pool[far] = c.pool[c.block_table[0].long()]
    table = far.to(torch.int32)[None].contiguous()
    cfg = _cfg(8, 8, 1, c.cfg.max_blocks_per_req, pages)
    d = msa.DenseAttention(cfg)
    d.run(c.seq_lens, table, c.q, pool, pool)
    want = c.run()
    assert msa.check_device_error(d.ws) == 0
    assert torch.equal(d.out, want.out) and torch.equal(d.lse, want.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (16, 2, 4)])
def test_rotate_append_and_attend(hq, hkv, q_len):
    """The layer: new rows rotated and quantised into the pool, then attended
    to with the rest of the context, against the oracle fed the pool after the
    write; as one captured graph it gives the same, step after step."""
    c = Case(hq, hkv, [300, 1000 + q_len, q_len, 128], q_len=q_len, seed=13)
    T = c.T
    n = 4096
    inv = 1.0e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    tab = torch.cat([ang.cos(), ang.sin()], dim=1).float().cuda()
    g = torch.Generator(device="cuda").manual_seed(14)
    kv = torch.randn((T, 2 * hkv, 128), generator=g, device="cuda").to(torch.bfloat16)
    new = (kv[:, :hkv], kv[:, hkv:])
    d = msa.DenseAttention(c.cfg, rope=msa.Rope(tab))
    before = c.pool.clone()

    def step():
        d.run(c.seq_lens, c.block_table, c.q, c.pool, c.pool, new_kv=new)

    step()
    torch.cuda.synchronize()
    assert msa.check_device_error(d.ws) == 0
    pos = [p for _, p in oracle.query_positions(c.lens, c.q_lens)]
    slots = oracle.cache_slots(c.lens, c.q_lens, to_np(c.block_table), 128)
    cs = tab[pos].cpu().numpy()
    kr = oracle.rotate_rows(to_np(new[0]), cs[:, :32], cs[:, 32:], False)
    want = oracle.cache_write_nvfp4(before.cpu().numpy(), slots, kr, c.cfg.k_scale, 0)
    want = oracle.cache_write_nvfp4(want, slots, to_np(new[1]), c.cfg.v_scale, 1)
    assert np.array_equal(c.pool.cpu().numpy(), want)
    qr = oracle.bf16_round(oracle.rotate_rows(to_np(c.q), cs[:, :32], cs[:, 32:], False))
    raw = c.q.clone()
    c.q = torch.from_numpy(qr).to(torch.bfloat16).cuda()
    c_out = d.out.clone(), d.lse.clone()
    c.check(d)
    c.q = raw
    c.pool.copy_(before)
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    d.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(c.pool.cpu().numpy(), want)
    assert torch.equal(d.out, c_out[0]) and torch.equal(d.lse, c_out[1])


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_new_rows_without_a_rope(given):
    """new_kv alone goes through cache_write; slots from the plan, or given."""
    c = Case(8, 2, [300, 129, 1], seed=15)
    g = torch.Generator(device="cuda").manual_seed(16)
    new = [torch.randn((3, 2, 128), generator=g, device="cuda").to(torch.bfloat16)
           for _ in range(2)]
    slots = oracle.cache_slots(c.lens, c.q_lens, to_np(c.block_table), 128)
    loc = torch.tensor(slots, dtype=torch.int64, device="cuda") if given else None
    want = oracle.cache_write_nvfp4(c.pool.cpu().numpy(), slots, to_np(new[0]), c.cfg.k_scale, 0)
    want = oracle.cache_write_nvfp4(want, slots, to_np(new[1]), c.cfg.v_scale, 1)
    d = c.layer()
    d.run(c.seq_lens, c.block_table, c.q, c.pool, c.pool, new_kv=new, out_cache_loc=loc)
    assert msa.check_device_error(d.ws) == 0
    assert np.array_equal(c.pool.cpu().numpy(), want)
    c.check(d)
    again = d.out.clone()
    d.out.fill_(7.0)
    d.run(None, None, c.q, c.pool, c.pool, planned=True)     # a second layer of the step
    assert torch.equal(d.out, again)


@pytest.mark.gpu
def test_sparse_and_dense_layers_share_a_plan():
    """A hybrid model's step: one plan and one workspace, a sparse layer, then a
    dense one that equals its own planned run."""
    spec = wl.small("nvfp4_decode", batch=3)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    sa = msa.SparseAttention(cfg)
    dense = msa.DenseAttention(cfg, ws=sa.ws)
    sa.run(w.seq_lens, w.block_table, w.idx_q, w.idx_k_pages, w.q, w.k_pages, w.v_pages)
    sparse = sa.out.clone()
    dense.run(w.seq_lens, w.block_table, w.q, w.k_pages, w.v_pages, planned=True)
    alone = msa.DenseAttention(cfg)
    alone.run(w.seq_lens, w.block_table, w.q, w.k_pages, w.v_pages)
    assert torch.equal(dense.out, alone.out) and torch.equal(dense.lse, alone.lse)
    sa.run(w.seq_lens, w.block_table, w.idx_q, w.idx_k_pages, w.q, w.k_pages, w.v_pages)
    assert torch.equal(sa.out, sparse)
    assert msa.check_device_error(sa.ws) == 0
