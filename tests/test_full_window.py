"""Full attention over bf16 and e4m3 pages: a local window as wide as the
context, through the sparse decode.  Every block is then local, the selection
all of them, and the result the dense attention of the request (the oracle's
selection and attention; for NVFP4 pages also the full-context decode's)."""
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
from block_sparse_paged_msa_gb300 import workloads as wl
from gpu_util import BF16_OUT_REL, LSE_MAX, OUT_MAX, compare, run_gpu
from oracle_io import run_oracle


def _spec(name, **kw):
    kw = {**dict(batch=3, num_q_heads=16, num_kv_heads=2, seq_len_range=None,
                 seq_lens=(20011, 1, 7000), num_pages=220, local_tokens=20480, topk_blocks=0), **kw}
    return wl.small(name, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("name,seq_lens", [("medium_decode", (20011, 1, 7000)),
                                           ("fp8_decode", (20011, 1, 7000)),
                                           ("nvfp4_decode", (20011, 1, 7000)),
                                           ("verify", (20011, 4, 7000))])
def test_a_window_as_wide_as_the_context(name, seq_lens):
    spec = _spec(name, seq_lens=seq_lens)
    w = wl.make_workload(spec, device="cuda")
    sa = run_gpu(w)
    assert msa.check_device_error(sa.ws) == 0
    nb = -(-int(w.seq_lens[0]) // 128)
    assert sa.selected[0, 0, :nb].tolist() == list(range(nb))
    compare(w, sa, run_oracle(w.to("cpu")))
    if spec.kv_dtype == "nvfp4":
        d = msa.DenseAttention(sa.cfg)
        d.run(w.seq_lens, w.block_table, w.q, w.k_pages, w.v_pages)
        out = sa.out.float()
        assert bool(((d.out.float() - out).abs() <= 2 * (OUT_MAX + BF16_OUT_REL * out.abs())).all())
        assert bool(((d.lse - sa.lse).abs() <= 2 * LSE_MAX).all())
