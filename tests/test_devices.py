"""Tensors on a device that is not the current one: every call makes theirs
current for its duration and takes its stream, not the current device's.  The
library, the tensors and the device switch are stand-ins: no GPU is needed."""
import contextlib

import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
from block_sparse_paged_msa_gb300 import ops


class Tensor:
    """A tensor on device 1 that passes every check."""
    shape = (2, 4096, 64, 64)
    is_cuda = True

    def numel(self):
        return 1 << 30

    def get_device(self):
        return 1

    def data_ptr(self):
        return 256


@pytest.fixture
def calls(monkeypatch):
    """[(call, current device, stream)] of the library; device 0 is current."""
    made, current = [], [0]

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                made.append((name, current[0], args[-1]))
                return 0
            return fn

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    lib = Lib()
    monkeypatch.setattr(ops, "lib", lambda: lib)
    monkeypatch.setattr(ops, "_device", lambda: current[0])
    monkeypatch.setattr(ops, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    for name in ("_need", "_need_ws", "_need_tokens", "_need_pools", "_need_block_table"):
        monkeypatch.setattr(ops, name, lambda *a, **k: None)
    monkeypatch.setattr(ops, "_need_batch", lambda *a, **k: 2)
    monkeypatch.setattr(ops, "_sizes", lambda cfg: (0, 0, 0, 0))
    monkeypatch.setattr(ops, "index_attention_scratch_bytes", lambda cfg: 1)
    return made


def _cfg(**kw):
    kw = {**dict(kv_dtype="nvfp4", q_len=1, max_batch=2), **kw}
    return msa.make_config(num_q_heads=8, num_kv_heads=1, init_blocks=1, local_blocks=2,
                           topk_blocks=4, index_dim=64, max_blocks_per_req=8, num_pages=16, **kw)


def _all(t, cfg):
    ops.plan(cfg, t, t, t)
    ops.plan_from_req_to_token(cfg, t, t, t, t)
    ops.cache_write(cfg, t, t, t, t, t, t, t)
    ops.index_attention(cfg, t, t, t, t, t, t)
    ops.index_score(cfg, t, t, t, t)
    ops.decode_step(cfg, t, t, t, t, t, t, t, t, t, t, t, t)
    ops.index_score_topk(cfg, t, t, t, t, t)
    ops.topk_select(cfg, t, t, t)
    ops.sparse_decode(cfg, t, t, t, t, t)
    ops.compact_selected(cfg, t, t, t, t)
    ops.paged_decode(cfg, t, t, t, t, t, t)
    ops.combine(cfg, t, t, t)
    ops.build_k2q_csr(cfg, t, t, t, t)
    ops.sparse_prefill(cfg, t, t, t, t, t, t, t)
    ops.sparse_decode_noalloc(cfg, t, t, t, t, t, t, t, t)
    ops.selftest_wait_timeout(cfg, t)
    ops.check_device_error(t)


def test_every_call_runs_on_its_tensors_device(calls):
    _all(Tensor(), _cfg())
    assert len(calls) == 17 and len({n for n, *_ in calls}) == 17
    for name, device, stream in calls:
        assert (device, getattr(stream, "value", stream)) == (1, 1001), name


def test_a_stream_of_another_device_is_refused(calls):
    stream = type("S", (), dict(device_index=0, cuda_stream=5))()
    with pytest.raises(ValueError, match="device 0"):
        ops.plan(_cfg(), Tensor(), Tensor(), Tensor(), stream=stream)
    stream.device_index = 1
    ops.plan(_cfg(), Tensor(), Tensor(), Tensor(), stream=stream)
    assert calls == [("msa_plan", 1, 5)]
    # a handle that does not say where it lives is taken as it is
    ops.plan(_cfg(), Tensor(), Tensor(), Tensor(), stream=type("S", (), dict(cuda_stream=6))())
    assert calls[1] == ("msa_plan", 1, 6)


def test_a_layers_run_stays_on_its_device(calls, monkeypatch):
    """DenseAttention.run: plan, cache write and decode, without and with new rows."""
    monkeypatch.setattr(ops, "_expect", lambda t, *a: t.data_ptr())
    y = type("Y", (), dict(ws=0, q=0, kv_dtypes=0, pool=0, dense_scratch=(1,), lse=0))()
    monkeypatch.setattr(ops, "_layout", lambda cfg: y)
    monkeypatch.setattr(ops, "_device_of", lambda t, name: t.get_device())
    t = Tensor()
    layer = object.__new__(msa.DenseAttention)
    layer.cfg, layer.rope = _cfg(), None
    layer.ws = layer.scratch = layer.out = layer.lse = t
    layer.run(t, t, t, t, t, new_kv=(t, t))
    assert [c[0] for c in calls] == ["msa_plan", "msa_cache_write", "msa_dense_decode"]
    assert all(c[1:] == (1, 1001) for c in calls)
