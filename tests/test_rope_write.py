"""msa_rope_cache_write: the rotary embedding applied on the way into the pools.

The rotation is byte work too: its products, differences and sums are single
IEEE fp32 operations, so the rotated queries (rounded to bf16 once) and the
pools after the write -- bf16 rows, e4m3 codes, NVFP4 rows -- must equal the
oracle's byte for byte, for both pair layouts, partial rotations, an index
table of its own, strided rows of a fused projection, explicit positions and
slots.  Refused arguments are checked without a GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from block_sparse_paged_msa_gb300 import ops
from block_sparse_paged_msa_gb300 import workloads as wl
from oracle_io import to_np

INVALID, UNSUPPORTED = 1, 2


# ------------------------------------------------------------ oracle pins (CPU)
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_the_complex_product(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 3, 128)).astype(np.float32)
    ang = rng.uniform(0, 6, (5, 32))
    y = oracle.rotate_rows(x, np.cos(ang), np.sin(ang), interleaved).astype(np.float64)
    a, b = (x[..., 0:64:2], x[..., 1:64:2]) if interleaved else (x[..., :32], x[..., 32:64])
    z = (a + 1j * b) * np.exp(1j * ang)[:, None, :]
    ya, yb = (y[..., 0:64:2], y[..., 1:64:2]) if interleaved else (y[..., :32], y[..., 32:64])
    # three roundings of a value of magnitude <= |z|, and the table's
    assert np.all(np.abs(ya - z.real) <= 4 * 2.0 ** -24 * 2 * np.abs(z))
    assert np.all(np.abs(yb - z.imag) <= 4 * 2.0 ** -24 * 2 * np.abs(z))
    assert np.array_equal(y[..., 64:], x[..., 64:])


def test_oracle_bf16_rounding():
    x = np.concatenate([np.random.default_rng(4).standard_normal(4096) * 3,
                        [0.0, 1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -1.0 - 2.0 ** -8]])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(oracle.bf16_round(x.astype(np.float32)), want)


# ------------------------------------------------------------ refusals (CPU)
def _args(**kw):
    """Arguments that pass every host check, as a dict of plain numbers."""
    a = dict(q=16, k=16, v=16, iq=16, ik=16, iv=None, pos=None, loc=None, qo=16, iqo=16, kp=16,
             vp=16, ikp=16, ivp=None, cs=16, ics=None, rot=64, irot=64, n=100, qs=1024, ks=128,
             vs=128, iqs=64, iks=64, ivs=64, ws=256)
    a.update(kw)
    return a


def _call(cfg, a):
    P = ctypes.c_void_p
    r = ops.MsaRope()
    r.cos_sin, r.idx_cos_sin = a["cs"], a["ics"]
    r.rotary_dim, r.idx_rotary_dim, r.num_positions = a["rot"], a["irot"], a["n"]
    for f, n in (("q_stride", "qs"), ("k_stride", "ks"), ("v_stride", "vs"),
                 ("idx_q_stride", "iqs"), ("idx_k_stride", "iks"), ("idx_v_stride", "ivs")):
        setattr(r, f, a[n])
    return ops.lib().msa_rope_cache_write(
        ctypes.byref(cfg), P(a["ws"]), ctypes.byref(r),
        *[P(a[n]) for n in ("q", "k", "v", "iq", "ik", "iv", "pos", "loc", "qo", "iqo", "kp",
                            "vp", "ikp", "ivp")], None)


@pytest.mark.parametrize("bad,status", [
    (dict(ws=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(cs=None), INVALID), (dict(qo=None), INVALID),
    (dict(kp=None), INVALID), (dict(vp=None), INVALID),
    (dict(iqo=None), INVALID), (dict(ikp=None), INVALID), (dict(iv=16), INVALID),
    (dict(rot=0), INVALID), (dict(rot=160), INVALID), (dict(irot=-32), INVALID),
    (dict(irot=96), INVALID),                        # > index_dim
    (dict(rot=48), UNSUPPORTED), (dict(irot=16, ics=16), UNSUPPORTED),
    (dict(irot=32), INVALID),                        # not the heads' table's width
    (dict(n=0), INVALID),
    (dict(qs=1023), INVALID), (dict(qs=1016), INVALID), (dict(ks=120), INVALID),
    (dict(vs=132), INVALID), (dict(iqs=60), INVALID), (dict(iks=68), INVALID),
    (dict(q=24), INVALID), (dict(k=8), INVALID), (dict(v=8), INVALID), (dict(cs=8), INVALID),
    (dict(ics=8), INVALID), (dict(qo=8), INVALID), (dict(iqo=8), INVALID), (dict(kp=8), INVALID),
    (dict(vp=8), INVALID), (dict(ikp=8), INVALID), (dict(iq=8), INVALID), (dict(ik=8), INVALID),
])
def test_refused_on_the_host(bad, status):
    cfg = msa.config_for(wl.WORKLOADS["tiny_decode"])        # 8 query heads, 1 KV head, d = 64
    assert _call(cfg, _args(**bad)) == status
    cfg.head_dim = 64
    assert _call(cfg, _args(**bad)) == UNSUPPORTED           # the config is checked first


def test_limits_refused_on_the_host():
    """Head rows of the largest step are counted in 31 bits."""
    kw = dict(init_blocks=1, local_blocks=1, topk_blocks=1, index_dim=64, max_batch=1,
              max_blocks_per_req=8192, num_pages=8192)
    cfg = msa.make_config(num_q_heads=1024, num_kv_heads=1024, max_q_tokens=1 << 20, **kw)
    wide = 1024 * 128
    assert _call(cfg, _args(qs=wide, ks=wide, vs=wide, iqs=wide, iks=wide)) == UNSUPPORTED
    cfg.max_batch = 0                          # a config of no tokens has nothing to do
    cfg.max_q_tokens = 0
    assert _call(cfg, _args(qs=wide, ks=wide, vs=wide, iqs=wide, iks=wide)) == 0


def test_a_misaligned_workspace_is_refused():
    """The kernels read the plan in words of 16 bytes: a workspace that msa_plan
    would refuse (256-byte alignment) is refused here too."""
    P, lib = ctypes.c_void_p, ops.lib()
    cfg = msa.make_config(num_q_heads=8, num_kv_heads=1, init_blocks=1, local_blocks=2,
                          topk_blocks=4, index_dim=64, max_batch=2, max_blocks_per_req=8,
                          num_pages=16, kv_dtype="nvfp4")
    for ws in (257, 260, 272, 384):
        assert lib.msa_plan(ctypes.byref(cfg), 1, P(256), None, P(256), 8, P(ws), None) == INVALID
        assert lib.msa_dense_decode(ctypes.byref(cfg), P(ws), *[P(256)] * 6, None) == INVALID
        assert _call(cfg, _args(ws=ws)) == INVALID


def test_rows_layouts_refused_by_the_binding():
    with pytest.raises(ValueError, match="CUDA"):
        ops._expect_rows(torch.zeros(2, 1, 128, dtype=torch.bfloat16), "q", (2, 1, 128), 0)


# ------------------------------------------------------------ parity (GPU)
def _table(n, rot, device="cuda"):
    inv = 1.0e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().to(device)


def _fused(spec, T, seed, extra=8):
    """q | k | v | idx_q | idx_k | idx_v as slices of one projection row."""
    hq, hkv, d, D = spec.num_q_heads, spec.num_kv_heads, spec.index_dim, spec.head_dim
    widths = [hq * D, hkv * D, hkv * D, hkv * d, hkv * d, hkv * d]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    row = torch.randn((T, sum(widths) + extra), generator=gen, device="cuda").to(torch.bfloat16)
    parts = torch.split(row[:, :sum(widths)], widths, dim=1)
    return [p.reshape(T, -1, w) if T == 0 else p.view(T, p.shape[1] // w, w)
            for p, w in zip(parts, (D, D, D, d, d, d))]


def _expected(w, rows, pos, slots, cos_sin, idx_cos_sin, interleaved):
    s = w.spec
    q, k, v, iq, ik, iv = (to_np(x) for x in rows)
    cs, ics = cos_sin.cpu().numpy(), idx_cos_sin.cpu().numpy()
    n, m = cs.shape[1] // 2, ics.shape[1] // 2

    def rot(x, tab, half):
        return oracle.rotate_rows(x, tab[pos, :half], tab[pos, half:], interleaved)

    qr, kr = rot(q, cs, n), rot(k, cs, n)
    iqr, ikr = rot(iq, ics, m), rot(ik, ics, m)
    if s.kv_dtype == "nvfp4":
        kp = oracle.cache_write_nvfp4(to_np(w.k_pages), slots, kr, s.kv_scale, 0)
        kp = vp = oracle.cache_write_nvfp4(kp, slots, v, s.kv_scale, 1)
    elif s.kv_dtype == "fp8_e4m3":
        kp = oracle.cache_write(to_np(w.k_pages), slots, kr, e4m3_scale=s.kv_scale)
        vp = oracle.cache_write(to_np(w.v_pages), slots, v, e4m3_scale=s.kv_scale)
    else:
        kp = oracle.cache_write(to_np(w.k_pages), slots, oracle.bf16_round(kr))
        vp = oracle.cache_write(to_np(w.v_pages), slots, v)
    return (oracle.bf16_round(qr), oracle.bf16_round(iqr), kp, vp,
            oracle.cache_write(to_np(w.idx_k_pages), slots, oracle.bf16_round(ikr)))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["medium_decode", "fp8_decode", "nvfp4_decode", "tiny_decode",
                                  "verify", "prefill", "nvfp4_prefill"])
@pytest.mark.parametrize("rot,interleaved", [(32, False), (64, True), (96, False), (128, False)])
def test_rotated_rows_and_pools_match_oracle(name, rot, interleaved):
    spec = wl.small(name, batch=3) if name.endswith("_decode") and name != "tiny_decode" \
        else wl.small(name)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    sa = msa.SparseAttention(cfg)
    T = w.num_tokens
    rows = _fused(spec, T, 11 + rot)
    pos = np.array([p for _, p in oracle.query_positions(to_np(w.seq_lens), to_np(w.q_lens))])
    slots = oracle.cache_slots(to_np(w.seq_lens), to_np(w.q_lens), to_np(w.block_table), 128)
    tab = _table(int(w.seq_lens.max()), rot)
    own = _table(int(w.seq_lens.max()), 32) if rot > spec.index_dim or rot == 96 else None
    want = _expected(w, rows, pos, slots, tab, tab if own is None else own, interleaved)
    q_out = torch.empty_like(sa.out)
    iq_out = torch.empty((T, spec.num_kv_heads, spec.index_dim), dtype=torch.bfloat16,
                         device="cuda")
    iv_pages = torch.zeros_like(w.idx_k_pages)
    msa.plan(cfg, w.seq_lens, w.block_table, sa.ws, w.cu_seqlens_q if sa.prefill else None)
    msa.rope_cache_write(cfg, sa.ws, *rows[:5], tab, q_out, iq_out, w.k_pages, w.v_pages,
                         w.idx_k_pages, interleaved=interleaved, idx_cos_sin=own, idx_v=rows[5],
                         idx_v_pages=iv_pages)
    torch.cuda.synchronize()
    assert msa.check_device_error(sa.ws) == 0
    for what, got, exp in zip(("q", "idx_q", "k_pages", "v_pages", "idx_k_pages"),
                              (q_out, iq_out, w.k_pages, w.v_pages, w.idx_k_pages), want):
        assert np.array_equal(to_np(got), exp), what
    exp = oracle.cache_write(np.zeros(iv_pages.shape), slots, to_np(rows[5]))
    assert np.array_equal(to_np(iv_pages), exp)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tiny_decode", "nvfp4_decode"])
def test_positions_slots_in_place_and_no_index_rows(name):
    """Explicit positions and slots; queries rotated in place; no index rows;
    rows past the step's tokens stay as they are."""
    spec = wl.small(name) if name == "tiny_decode" else wl.small(name, batch=3)
    w = wl.make_workload(spec, device="cuda")
    B = spec.batch
    cfg = msa.config_for(spec, max_batch=B + 2)
    sa = msa.SparseAttention(cfg)
    T = w.num_tokens
    q, k, v, *_ = (x.contiguous() for x in _fused(spec, T + 2, 5))
    pos = torch.tensor([7, 0, 4095][:T] + [0, 0], device="cuda")
    slots = torch.randperm(spec.num_pages * 128, device="cuda")[:T + 2]
    tab = _table(4096, 64)
    rows = [x[:T] for x in (q, k, v)] + [x[:T] for x in _fused(spec, T, 6)[3:]]
    want = _expected(w, rows, pos[:T].cpu().numpy(), slots[:T].tolist(), tab, tab, False)
    tail, idx_before = q[T:].clone(), w.idx_k_pages.clone()
    msa.plan(cfg, w.seq_lens, w.block_table, sa.ws)
    msa.rope_cache_write(cfg, sa.ws, q, k, v, None, None, tab, q, None, w.k_pages, w.v_pages,
                         None, positions=pos, out_cache_loc=slots)
    assert msa.check_device_error(sa.ws) == 0
    assert np.array_equal(to_np(q[:T]), want[0]) and torch.equal(q[T:], tail)
    assert np.array_equal(to_np(w.k_pages), want[2])
    assert np.array_equal(to_np(w.v_pages), want[3])
    assert torch.equal(w.idx_k_pages, idx_before)


@pytest.mark.gpu
def test_bad_positions_and_slots_are_flagged_and_skipped():
    spec = wl.small("fp8_decode", batch=3)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    sa = msa.SparseAttention(cfg)
    rows = _fused(spec, 3, 8)
    tab = _table(64, 64)
    q_out = torch.zeros_like(sa.out)
    iq_out = torch.zeros((3, spec.num_kv_heads, spec.index_dim), dtype=torch.bfloat16,
                         device="cuda")
    for pos, loc, bits, kept, rotated in (
            ([5, 64, -1], [130, 400, 401], 32, [130, -1, -1], [0]),
            ([5, 6, 7], [130, spec.num_pages * 128, -3], 1, [130, -1, -1], [0, 1, 2])):
        q_out.zero_()
        want = _expected(w, rows, np.clip(pos, 0, 63), kept, tab, tab, False)
        msa.plan(cfg, w.seq_lens, w.block_table, sa.ws)
        msa.rope_cache_write(cfg, sa.ws, *rows[:5], tab, q_out, iq_out, w.k_pages, w.v_pages,
                             w.idx_k_pages, positions=torch.tensor(pos, device="cuda"),
                             out_cache_loc=torch.tensor(loc, device="cuda"))
        assert msa.check_device_error(sa.ws) == bits
        got = to_np(q_out)
        for t in range(3):
            assert np.array_equal(got[t], want[0][t] if t in rotated else 0 * got[t])
        for a, b in zip((w.k_pages, w.v_pages, w.idx_k_pages), want[2:]):
            assert np.array_equal(to_np(a), b)


@pytest.mark.gpu
def test_idle_requests_are_skipped():
    spec = wl.small("medium_decode", seq_lens=(900, 0, 300), seq_len_range=None, batch=3,
                    num_pages=40)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    sa = msa.SparseAttention(cfg)
    rows = _fused(spec, 3, 9)
    tab = _table(900, 128)
    slots = oracle.cache_slots(to_np(w.seq_lens), to_np(w.q_lens), to_np(w.block_table), 128)
    want = _expected(w, rows, np.array([899, 0, 299]), slots, tab, tab, False)
    q_out = torch.full_like(sa.out, 3.0)
    iq_out = torch.full((3, spec.num_kv_heads, spec.index_dim), 3.0, dtype=torch.bfloat16,
                        device="cuda")
    msa.plan(cfg, w.seq_lens, w.block_table, sa.ws)
    msa.rope_cache_write(cfg, sa.ws, *rows[:5], tab, q_out, iq_out, w.k_pages, w.v_pages,
                         w.idx_k_pages)
    assert msa.check_device_error(sa.ws) == 0
    assert np.array_equal(to_np(q_out)[[0, 2]], want[0][[0, 2]])
    assert bool((q_out[1] == 3.0).all()) and bool((iq_out[1] == 3.0).all())
    for a, b in zip((w.k_pages, w.v_pages, w.idx_k_pages), want[2:]):
        assert np.array_equal(to_np(a), b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["medium_decode", "nvfp4_decode", "verify", "prefill"])
def test_sparse_step_with_a_rope_equals_rotation_then_write(name):
    """SparseAttention(rope=...): the step equals, bit for bit, the one fed with
    rows rotated beforehand (by the oracle) through cache_write."""
    spec = wl.small(name, batch=3) if name.endswith("_decode") else wl.small(name)
    w1, w2 = (wl.make_workload(spec, device="cuda") for _ in range(2))
    cfg = msa.config_for(spec)
    T = w1.num_tokens
    q, k, v, iq, ik, _ = _fused(spec, T, 21)
    tab = _table(int(w1.seq_lens.max()), 64)
    pos = [p for _, p in oracle.query_positions(to_np(w1.seq_lens), to_np(w1.q_lens))]

    def turned(x):
        c = tab[pos].cpu().numpy()
        y = oracle.bf16_round(oracle.rotate_rows(to_np(x), c[:, :32], c[:, 32:], False))
        return torch.from_numpy(y).to(torch.bfloat16).cuda()

    cu = w1.cu_seqlens_q if cfg.mode == ops.MSA_MODE_PREFILL else None
    a = msa.SparseAttention(cfg, rope=msa.Rope(tab))
    a.run(w1.seq_lens, w1.block_table, iq, w1.idx_k_pages, q, w1.k_pages, w1.v_pages,
          cu_seqlens_q=cu, new_kv=(k, v, ik))
    b = msa.SparseAttention(cfg)
    if spec.kv_dtype == "nvfp4":
        # its codes come from the unrounded rotated key: take the pools from the first run
        kp, ikp, kv_new = w1.k_pages, w1.idx_k_pages, None
    else:
        kp, ikp, kv_new = w2.k_pages, w2.idx_k_pages, (turned(k), v.contiguous(), turned(ik))
    b.run(w2.seq_lens, w2.block_table, turned(iq), ikp, turned(q), kp,
          w1.v_pages if kv_new is None else w2.v_pages, cu_seqlens_q=cu, new_kv=kv_new)
    torch.cuda.synchronize()
    assert msa.check_device_error(a.ws) == 0
    assert torch.equal(a.selected[:T], b.selected[:T])
    assert torch.equal(a.out[:T], b.out[:T]) and torch.equal(a.lse[:T], b.lse[:T])
    with pytest.raises(ValueError, match="new_kv"):
        a.run(w1.seq_lens, w1.block_table, iq, w1.idx_k_pages, q, w1.k_pages, w1.v_pages)


@pytest.mark.gpu
def test_dense_sparse_step_with_a_rope():
    """The compacted form of the step takes the rotated queries too."""
    spec = wl.small("medium_decode", batch=3)
    cfg = msa.config_for(spec)
    runs = []
    for dense_sparse in (False, True):
        w = wl.make_workload(spec, device="cuda")
        q, k, v, iq, ik, _ = _fused(spec, w.num_tokens, 25)
        sa = msa.SparseAttention(cfg, dense_sparse=dense_sparse,
                                 rope=msa.Rope(_table(int(w.seq_lens.max()), 128)))
        sa.run(w.seq_lens, w.block_table, iq, w.idx_k_pages, q, w.k_pages, w.v_pages,
               new_kv=(k, v, ik))
        torch.cuda.synchronize()
        assert msa.check_device_error(sa.ws) == 0
        runs.append(sa)
    a, b = runs
    T = w.num_tokens
    assert torch.equal(a.selected[:T], b.selected[:T])
    # the same keys, in splits of their own: the bound of the dense-sparse form
    assert (a.out[:T].float() - b.out[:T].float()).abs().max() <= 1e-2
    assert (a.lse[:T] - b.lse[:T]).abs().max() <= 1e-3


@pytest.mark.gpu
def test_token_strides_and_pools_past_32_bits():
    """Rows 2^31 elements apart, and pages whose byte offset passes 2^32."""
    pages = 140000                                 # of 32 KiB
    far = [139999, 131072]
    cfg = msa.make_config(num_q_heads=2, num_kv_heads=1, init_blocks=0, local_blocks=1,
                          topk_blocks=1, index_dim=64, max_batch=2, max_blocks_per_req=1,
                          num_pages=pages)
    g = torch.Generator(device="cuda").manual_seed(31)
    wide = torch.empty((1 << 31) + 1024, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((2, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    fused = wide.as_strided((2, 4, 128), (1 << 31, 128, 1))
    fused.copy_(rows)
    q, k, v = fused[:, :2], fused[:, 2:3], fused[:, 3:]
    tab = _table(128, 128)
    kp, vp = (torch.zeros((pages, 1, 128, 128), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    ws = torch.empty(msa.workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    q_out = torch.empty((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([5, 128], dtype=torch.int32, device="cuda")
    table = torch.tensor(far, dtype=torch.int32, device="cuda")[:, None].contiguous()
    msa.plan(cfg, lens, table, ws)
    msa.rope_cache_write(cfg, ws, q, k, v, None, None, tab, q_out, None, kp, vp, None)
    assert msa.check_device_error(ws) == 0
    cs = tab[[4, 127]].cpu().numpy()

    def turned(x):
        return oracle.bf16_round(oracle.rotate_rows(to_np(x), cs[:, :64], cs[:, 64:], False))

    assert np.array_equal(to_np(q_out), turned(rows[:, :2]))
    for t, (page, row) in enumerate(zip(far, (4, 127))):
        assert np.array_equal(to_np(kp[page, 0, row]), turned(rows[:, 2:3])[t, 0])
        assert np.array_equal(to_np(vp[page, 0, row]), to_np(rows[t, 3]))
        for x in (kp, vp):
            assert int((x[page] != 0).any(-1).sum()) == 1
    assert int((kp != 0).any(-1).sum()) == 2 and int((vp != 0).any(-1).sum()) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["medium_decode", "tiny_decode"])
def test_index_rows_without_rotation(name):
    """An index table of width 0: the index rows are stored as they are."""
    spec = wl.small(name)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    sa = msa.SparseAttention(cfg)
    T = w.num_tokens
    q, k, v, iq, ik, _ = _fused(spec, T, 33)
    n = int(w.seq_lens.max())
    iq_out = torch.zeros_like(iq, memory_format=torch.contiguous_format)
    rope = msa.Rope(_table(n, 64), idx_cos_sin=torch.zeros((n, 0), device="cuda"))
    msa.plan(cfg, w.seq_lens, w.block_table, sa.ws)
    rope.write(cfg, sa.ws, q, k, v, iq, ik, sa.out, iq_out, w.k_pages, w.v_pages, w.idx_k_pages)
    assert msa.check_device_error(sa.ws) == 0
    assert torch.equal(iq_out, iq)
    slots = oracle.cache_slots(to_np(w.seq_lens), to_np(w.q_lens), to_np(w.block_table), 128)
    for t, s in enumerate(slots):
        assert torch.equal(w.idx_k_pages[s // 128, :, s % 128], ik[t])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["medium_decode", "nvfp4_decode"])
def test_inputs_of_exactly_the_steps_tokens(name):
    """By the C call the inputs, positions and slots hold the step's tokens and no
    more, whatever the config's maxima are."""
    spec = wl.small(name, batch=3)
    w1, w2 = (wl.make_workload(spec, device="cuda") for _ in range(2))
    cfg = msa.config_for(spec, max_batch=3 + 200)
    T, most = w1.num_tokens, ops.max_tokens(cfg)
    rows = [x.contiguous() for x in _fused(spec, T, 41)[:5]]
    tab = _table(int(w1.seq_lens.max()), 64)
    pos = torch.tensor([p for _, p in oracle.query_positions(to_np(w1.seq_lens),
                                                             to_np(w1.q_lens))], device="cuda")
    slots = torch.tensor(oracle.cache_slots(to_np(w1.seq_lens), to_np(w1.q_lens),
                                            to_np(w1.block_table), 128), device="cuda")
    a = msa.SparseAttention(cfg)
    msa.plan(cfg, w1.seq_lens, w1.block_table, a.ws)

    def pad(x, n=most):
        y = torch.zeros((n, *x.shape[1:]), dtype=x.dtype, device="cuda")
        y[:len(x)] = x
        return y

    full = [pad(x) for x in rows]
    outs = torch.empty_like(full[0]), torch.empty_like(full[3])
    msa.rope_cache_write(cfg, a.ws, *full, tab, *outs, w1.k_pages, w1.v_pages, w1.idx_k_pages,
                         positions=pad(pos), out_cache_loc=pad(slots))
    rope = ops.MsaRope(tab.data_ptr(), None, 64, 64, 0, tab.shape[0],
                       *[x.stride(0) for x in rows], 0)
    exact = torch.empty_like(rows[0]), torch.empty_like(rows[3])
    P = ctypes.c_void_p
    assert ops.lib().msa_rope_cache_write(
        ctypes.byref(cfg), P(a.ws.data_ptr()), ctypes.byref(rope),
        *[P(x.data_ptr()) for x in rows], None, P(pos.data_ptr()), P(slots.data_ptr()),
        P(exact[0].data_ptr()), P(exact[1].data_ptr()), P(w2.k_pages.data_ptr()),
        P(w2.v_pages.data_ptr()), P(w2.idx_k_pages.data_ptr()), None,
        P(torch.cuda.current_stream().cuda_stream)) == 0
    assert msa.check_device_error(a.ws) == 0
    assert torch.equal(exact[0], outs[0][:T]) and torch.equal(exact[1], outs[1][:T])
    for x, y in ((w1.k_pages, w2.k_pages), (w1.v_pages, w2.v_pages),
                 (w1.idx_k_pages, w2.idx_k_pages)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("length", [0, 1, 7])
def test_an_index_table_that_is_not_read_limits_no_position(length):
    """Of width 0, whatever its length; and any table when the call has no index
    rows (the full-attention layers of the same model)."""
    spec = wl.small("nvfp4_decode", batch=3)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    T = w.num_tokens
    q, k, v, iq, ik, _ = _fused(spec, T, 45)
    tab = _table(int(w.seq_lens.max()), 64)
    ws = torch.empty(msa.workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    msa.plan(cfg, w.seq_lens, w.block_table, ws)

    def write(idx_cos_sin, with_index):
        kp, ikp = w.k_pages.clone(), w.idx_k_pages.clone()
        q_out = torch.zeros((T, spec.num_q_heads, 128), dtype=torch.bfloat16, device="cuda")
        iq_out = torch.zeros((T, spec.num_kv_heads, spec.index_dim), dtype=torch.bfloat16,
                             device="cuda")
        msa.Rope(tab, idx_cos_sin=idx_cos_sin).write(
            cfg, ws, q, k, v, iq if with_index else None, ik if with_index else None, q_out,
            iq_out if with_index else None, kp, kp, ikp if with_index else None)
        assert msa.check_device_error(ws) == 0
        return q_out, iq_out, kp, ikp

    full = torch.zeros((tab.shape[0], 0), device="cuda")
    for a, b in zip(write(torch.zeros((length, 0), device="cuda"), True), write(full, True)):
        assert torch.equal(a, b)
    for a, b in zip(write(torch.zeros((length, 32), device="cuda"), False), write(None, False)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_position_outside_the_index_table_is_flagged():
    """A table of the index heads that is read does limit the positions."""
    spec = wl.small("medium_decode", batch=3)
    w = wl.make_workload(spec, device="cuda")
    cfg = msa.config_for(spec)
    q, k, v, iq, ik, _ = _fused(spec, 3, 46)
    sa = msa.SparseAttention(cfg)
    iq_out = torch.empty((3, spec.num_kv_heads, spec.index_dim), dtype=torch.bfloat16,
                         device="cuda")
    msa.plan(cfg, w.seq_lens, w.block_table, sa.ws)
    before = w.k_pages.clone()
    msa.rope_cache_write(cfg, sa.ws, q, k, v, iq, ik, _table(int(w.seq_lens.max()), 64), sa.out,
                         iq_out, w.k_pages, w.v_pages, w.idx_k_pages,
                         idx_cos_sin=_table(1, 32))
    assert msa.check_device_error(sa.ws) == 32
    assert torch.equal(w.k_pages, before)
