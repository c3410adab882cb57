"""msa_dense_decode where a team's range holds many pages.

The cases have more (page, head) units than twice the teams of the machine (two
to four an SM), so that a range holds several pages of a request, and several
requests one after the other: the accumulation over pages, the moves of the
reference, the wrap of the rings, the change of requests.

Bounds as in test_dense_decode.py, and one term more.  The probabilities go to
fp16 as 2^(s' - m + 7): those below 2^-14 are subnormal there and off by up to
half a step, 2^-25, whatever their size.  m is never above the row's largest
score, so the sum they are divided by is 2^7 or more: 2^-32 sum |v| in the
output.  It shows in a dim where the values of the likely keys are 0."""
import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from oracle_io import to_np
from test_dense_decode import Case


def _check(c, d, heads):
    """Rows of the KV heads `heads` against the oracle."""
    cfg, G, T = c.cfg, c.hq // c.hkv, c.T
    pool, table = c.pool.cpu().numpy(), to_np(c.block_table)
    out_all, lse_all = to_np(d.out), to_np(d.lse)
    assert np.all(out_all[T:] == 7.0) and np.all(lse_all[T:] == 7.0)
    for h in heads:
        k = np.nan_to_num(oracle.nvfp4_dequant(pool[:, 2 * h:2 * h + 1], 128)) * cfg.k_scale
        v = np.nan_to_num(oracle.nvfp4_dequant(pool[:, 2 * h + 1:2 * h + 2], 128)) * cfg.v_scale
        rows = slice(h * G, (h + 1) * G)
        q = to_np(c.q[:T, rows])
        out, lse, mag = oracle.dense_attention(
            seq_lens=c.lens, q_lens=c.q_lens, block_table=table, q=q, k=k, v=v, num_kv_heads=1,
            block_size=128, softmax_scale=cfg.softmax_scale)
        sums = np.zeros((T, 1, 128))               # sum |v| over all keys of the request
        for t, (r, p) in enumerate(oracle.query_positions(c.lens, c.q_lens)):
            if p >= 0:
                sums[t, 0] = np.abs(v[table[r, :-(-c.lens[r] // 128)].astype(int), 0]).sum((0, 1))
        top = np.sqrt((k ** 2).sum(-1)).max() * np.sqrt((q ** 2).sum(-1)) * cfg.softmax_scale
        e = 16 * 2.0 ** -22 * top + 2.0 ** -21
        n = max(max(c.lens), 1)
        tol = 2.0 ** -8 * np.abs(out) + 2.0 ** -32 * sums + (
            2.0 ** -11 + 2 * e + (n / 16 + 64) * 2.0 ** -24)[..., None] * mag
        err = np.abs(out_all[:T, rows] - out)
        assert np.all(err <= tol), (h, float((err - tol).max()))
        fin = np.isfinite(lse)
        got = lse_all[:T, rows]
        assert np.array_equal(got[~fin], lse[~fin])
        lt = (e + (n / 16 + 64) * 2.0 ** -24)[fin] + 2.0 ** -22 * np.abs(lse[fin])
        assert np.all(np.abs(got[fin] - lse[fin]) <= lt), np.abs(got[fin] - lse[fin]).max()


def _mixed(n_long, n_short, seed, lo=1000, hi=3000):
    rng = np.random.default_rng(seed)
    lens = np.concatenate([rng.integers(lo, hi, n_long), rng.integers(4, 300, n_short), [0, 128]])
    return [int(x) for x in rng.permutation(lens)]


FORMS = [(5, 1), (8, 1), (2, 3), (16, 1), (5, 3), (8, 4), (16, 2), (11, 2), (16, 4), (12, 4),
         (16, 3)]                                      # query heads a KV head, new tokens


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", FORMS)
def test_ranges_of_many_pages(group, q_len):
    hkv = 8
    c = Case(group * hkv, hkv, _mixed(48, 40, group * 8 + q_len), q_len=q_len, q_std=3.0,
             seed=100 + group * 8 + q_len)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    _check(c, d, [0, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", [(8, 1), (16, 1), (8, 4), (16, 4)])
def test_one_request_of_many_pages_a_range(group, q_len):
    """One request whose heads have more pages than a range holds."""
    c = Case(group * 8, 8, [40011], q_len=q_len, q_std=6.0, seed=120 + q_len)
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    _check(c, d, [1, 7])


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", [(16, 1), (3, 4)])
def test_a_long_step_of_nine_to_sixteen_rows(group, q_len):
    """More than 128 pages an SM."""
    c = Case(group * 8, 8, _mixed(62, 20, 7, 4200, 6000), q_len=q_len, q_std=3.0, seed=130)
    assert sum(-(-L // 128) for L in c.lens) * 8 >= 128 * 152
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    _check(c, d, [3])


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", [(8, 1), (16, 1), (8, 4), (16, 4)])
def test_flagged_pages_inside_ranges_of_many_pages(group, q_len):
    """Requests whose first page, or first three, are flagged: rows that see
    nothing for the first pages of a range, then what the other pages hold."""
    nb = [4 + r % 13 for r in range(64)]
    c = Case(group * 8, 8, [128 * n for n in nb], q_len=q_len, q_std=3.0, seed=140 + q_len)
    gone = [3 if r % 4 == 1 else r % 2 for r in range(64)]
    good = to_np(c.block_table).astype(np.int32)
    bad, rest = good.copy(), np.full_like(good, -1)
    for r, n in enumerate(gone):
        bad[r, :n] = c.cfg.num_pages + r
        rest[r, :nb[r] - n] = good[r, n:nb[r]]
    c.block_table = torch.from_numpy(bad).cuda()
    d = c.run()
    assert msa.check_device_error(d.ws) == 1
    c.block_table = torch.from_numpy(rest).cuda()
    c.lens = [128 * (n - g) for n, g in zip(nb, gone)]
    _check(c, d, [2, 6])


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", [(8, 4), (16, 4)])
def test_a_draft_tokens_nan_inside_ranges_of_many_pages(group, q_len):
    """NaN scales in the K or V row of every seventh request's last token."""
    hkv = 8
    lens = [L for L in _mixed(48, 40, 150) if L > 0]
    for slot in (0, 1):
        # scores of a few units: no key moves a reference after its range's first
        # page, so that the rows that do not see the NaN are bit-equal
        c = Case(group * hkv, hkv, lens, q_len=q_len, seed=150, q_std=0.2)
        clean = c.run()
        hit = torch.zeros((len(lens), q_len, group * hkv), dtype=torch.bool, device="cuda")
        for r in range(0, len(lens), 7):
            page = int(c.block_table[r, (lens[r] - 1) // 128])
            c.pool[page, slot::2, (lens[r] - 1) % 128, 64 + 3] = 0x7f
            hit[r, -1] = True
        d = c.run()
        assert msa.check_device_error(d.ws) == 0
        hit = hit.view(-1, group * hkv)
        assert torch.equal(d.out[~hit], clean.out[~hit])
        assert torch.equal(d.lse[~hit], clean.lse[~hit])
        nan = d.out[hit].isnan()
        assert bool(nan[:, 48:64].all())
        if slot == 0:
            assert bool(nan.all()) and bool(d.lse[hit].isnan().all())
        else:
            assert not bool(nan[:, :48].any()) and not bool(nan[:, 64:].any())
            assert torch.equal(d.lse, clean.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("group,q_len", [(8, 1), (16, 1), (8, 4), (16, 4)])
def test_equal_scores_past_24_bits_in_one_range(group, q_len):
    """Two keys of the same huge score in neighbouring pages have half the weight
    each; 64 requests of 8 pages on 4 heads, so that ranges hold several pages."""
    hkv, batch = 4, 64
    c = Case(group * hkv, hkv, [1024] * batch, q_len=q_len, seed=160)
    c.block_table[:] = c.block_table[:1].clone()
    ids = to_np(c.block_table[0]).astype(int)
    size = 16384.0 + 128.0 * (torch.arange(group * hkv, device="cuda") % 16).view(1, -1, 1)
    c.q.copy_(torch.sign(c.q[:1, :1].float()) * size)
    c.q[c.q == 0] = 16384.0
    sign = (to_np(c.q[0, 0]) < 0).astype(np.uint8)
    codes = torch.from_numpy((7 + 8 * sign)[0::2] + 16 * (7 + 8 * sign)[1::2]).cuda()
    c.pool[:, 0::2] = 0
    for j in (2, 3):
        c.pool[int(ids[j]), 0::2, 9, :64] = codes
        c.pool[int(ids[j]), 0::2, 9, 64:] = 0x7e
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    pool = c.pool[torch.from_numpy(ids[2:4]).cuda()].cpu().numpy()
    v = oracle.nvfp4_dequant(pool, 128)[:, 1::2, 9]                        # [2, hkv, 128]
    want = oracle.bf16_round((np.repeat(v.mean(0), group, 0) * c.cfg.v_scale).astype(np.float32))
    got = to_np(d.out)
    assert np.array_equal(got, np.broadcast_to(want, got.shape))


@pytest.mark.gpu
@pytest.mark.parametrize("base,unit", [(4096.0, 0.75), (16384.0, 1.0)])
@pytest.mark.parametrize("group,q_len", [(8, 1), (16, 1), (8, 4), (16, 4)])
def test_top_scores_that_rise_page_by_page_past_24_bits(group, q_len, base, unit):
    """The first key of page j scores base * 768 * 112 + 128 unit j, every other key
    0.  The scores are whole steps of fp32 (32 near 2^28, 128 near 2^30), and a
    page's top is 96 or 128 above the one before: more than the 83.7 that the
    probabilities' range allows, and no more than the next float past 83.7.  It is
    so for every row (one row's move of the reference moves all).  2048 (page,
    head) units, so that every team's range holds several pages of a request."""
    hkv, pages, batch = 4, 8, 64
    c = Case(group * hkv, hkv, [128 * pages] * batch, q_len=q_len, seed=51)
    c.block_table[:] = c.block_table[:1].clone()
    ids = to_np(c.block_table[0]).astype(int)
    c.pool[:, 0::2] = 0
    c.q[:, :, :112] = base
    c.q[:, :, 112:] = unit
    for j, page in enumerate(ids):
        codes = np.full(128, 7)                        # 6 * 128
        codes[112:] = 2 * (np.arange(16) < j)          # 1 * 128
        row = np.concatenate([codes[0::2] + 16 * codes[1::2], np.full(8, 0x70)])
        c.pool[page, 0::2, 0] = torch.from_numpy(row.astype(np.uint8)).cuda()
    d = c.run()
    assert msa.check_device_error(d.ws) == 0
    pool = c.pool[torch.from_numpy(ids).cuda()].cpu().numpy()
    step = 128 * unit * np.arange(pages) * c.cfg.k_scale * c.cfg.softmax_scale
    w = np.exp(step - step[-1])
    v = oracle.nvfp4_dequant(pool, 128)[:, 1::2, 0] * c.cfg.v_scale        # [pages, hkv, 128]
    v = np.repeat(v, group, axis=1)
    out = np.einsum("j,jhd->hd", w / w.sum(), v)
    mag = np.einsum("j,jhd->hd", w / w.sum(), np.abs(v))
    # differences of scores are exact; their scale is off by a few 2^-24, times an
    # exponent of 13 or less wherever the weight counts; weights below 2^-24 may go
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -17) * mag + 2.0 ** -22 * np.abs(v).max()
    got = to_np(d.out)
    assert np.all(np.abs(got - out) <= tol), np.abs(got - out).max()
    top = base * 768 * 112 * c.cfg.k_scale * c.cfg.softmax_scale + step[-1] + np.log(w.sum())
    assert np.all(np.abs(to_np(d.lse) - top) <= (128 + 4) * 2.0 ** -24 * top)
