"""msa_dense_decode where a team's range holds many pages.

The cases have more (page, head) units than twice the teams of the machine (two
to four an SM), so that a range holds several pages of a request."""
import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from oracle_io import to_np
from test_dense_decode import Case


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
