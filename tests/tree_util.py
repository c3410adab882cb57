"""Steps that verify draft trees, drawn for the tests."""
import numpy as np
import torch

import block_sparse_paged_msa_gb300 as msa
import oracle
from oracle_io import to_np

SCALES = {"bf16": (1.0, 1.0), "fp8_e4m3": (2.0 ** -5, 2.0 ** -4), "nvfp4": (0.75, 0.5)}


def config(hq, hkv, batch, blocks, pages, tokens, kv="bf16", **kw):
    ks, vs = SCALES[kv]
    kw = {**dict(kv_dtype=kv, k_scale=ks, v_scale=vs, max_q_tokens=tokens, index_dim=64), **kw}
    return msa.make_config(num_q_heads=hq, num_kv_heads=hkv, init_blocks=1, local_blocks=1,
                           topk_blocks=0, max_batch=batch, max_blocks_per_req=blocks,
                           num_pages=pages, **kw)


def random_tree(n, width, rng):
    """Parents of n nodes, each one of the `width` nodes before it."""
    return [-1] + [max(0, i - 1 - int(rng.integers(width))) for i in range(1, n)]


class Step:
    """Ragged trees over a paged cache of `kv` rows.  Pages of no request and
    rows past each end hold NaN."""

    def __init__(self, hq, hkv, lens, nodes, kv="bf16", width=3, seed=1, q_std=1.0,
                 max_batch=None, max_blocks=None, extra_tokens=0, extra_pages=3, masks=None, **kw):
        assert all(n <= L or L == 0 for L, n in zip(lens, nodes))
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.kv, self.lens, self.nodes = hq, hkv, kv, lens, nodes
        B, self.T = len(lens), sum(nodes)
        nb = [-(-L // 128) for L in lens]
        pages, blocks = sum(nb) + extra_pages, max_blocks or max(max(nb), 1)
        rows = self.T + extra_tokens
        self.cfg = config(hq, hkv, max_batch or B, blocks, pages, rows, kv, **kw)
        self.parents_of = [random_tree(n, width, rng) if n else [] for n in nodes]
        self.masks = masks or [m for p in self.parents_of for m in oracle.tree_masks(p)]
        perm = rng.permutation(pages).tolist()
        table = np.full((B, blocks), -1, dtype=np.int32)
        used = 0
        for r, n in enumerate(nb):
            table[r, :n] = perm[used:used + n]
            used += n
        bad = [(p, 0) for p in perm[used:]] + [
            (table[r, nb[r] - 1], lens[r] % 128) for r in range(B) if lens[r] % 128]
        if kv == "nvfp4":
            pool = torch.randint(0, 256, (pages, 2 * hkv, 128, 72), generator=g, device="cuda",
                                 dtype=torch.uint8)
            pool[..., 64:] = torch.randint(0x20, 0x39, (pages, 2 * hkv, 128, 8), generator=g,
                                           device="cuda", dtype=torch.uint8)
            for p, u in bad:
                pool[p, :, u:, 64:] = 0x7f
            self.k = self.v = pool
        else:
            dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
            self.k, self.v = ((torch.randn((pages, hkv, 128, 128), generator=g, device="cuda")
                               / s).to(dt) for s in SCALES[kv])
            for x in (self.k, self.v):
                for p, u in bad:
                    x.view(torch.uint8)[p, :, u:] = 0xff if u % 2 else 0x7f
        dev = dict(device="cuda")
        self.block_table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, **dev)
        self.cu = torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32, **dev)
        pad = [7] * extra_tokens
        self.parents = torch.tensor([p for x in self.parents_of for p in x] + pad,
                                    dtype=torch.int32, **dev)
        self.mask = torch.tensor([(m + (1 << 63)) % (1 << 64) - (1 << 63) for m in self.masks] + pad,
                                 dtype=torch.int64, **dev)
        self.q = (q_std * torch.randn((rows, hq, 128), generator=g, **dev)).to(torch.bfloat16)

    def layer(self):
        d = msa.TreeAttention(self.cfg)
        d.out.fill_(7.0)
        d.lse.fill_(7.0)
        return d

    def attend(self, d=None, mask=True, stream=None):
        """plan, then the attention under self.mask (None: as chains)."""
        d = d or self.layer()
        msa.plan(self.cfg, self.seq_lens, self.block_table, d.ws, self.cu, stream)
        msa.tree_attention(self.cfg, d.ws, self.q, self.k, self.v, self.mask if mask else None,
                           d.scratch, d.out, d.lse, stream)
        return d

    def pools(self, h):
        """Dequantised K and V of KV head h, fp64 [pages, 1, 128, 128]."""
        both = []
        for x, slot, s in ((self.k, 2 * h, self.cfg.k_scale), (self.v, 2 * h + 1, self.cfg.v_scale)):
            if self.kv == "nvfp4":
                y = oracle.nvfp4_dequant(x[:, slot:slot + 1].cpu().numpy(), 128) * s
            elif self.kv == "fp8_e4m3":
                y = oracle.e4m3_to_float(to_np(x[:, h:h + 1])) * s
            else:
                y = to_np(x[:, h:h + 1])
            both.append(np.nan_to_num(y, nan=0.0))
        return both

    def check(self, d, masks=None, heads=None):
        """Within bounds derived from the roundings (test_tree_attention.py)."""
        c, G, T = self.cfg, self.hq // self.hkv, self.T
        out_all, lse_all = to_np(d.out), to_np(d.lse)
        assert np.all(out_all[T:] == 7.0) and np.all(lse_all[T:] == 7.0)
        for h in range(self.hkv) if heads is None else heads:
            k, v = self.pools(h)
            rows = slice(h * G, (h + 1) * G)
            q = to_np(self.q[:T, rows])
            out, lse, mag = oracle.tree_attention(
                seq_lens=self.lens, q_lens=self.nodes, masks=masks or self.masks,
                block_table=to_np(self.block_table), q=q, k=k, v=v, num_kv_heads=1,
                block_size=128, softmax_scale=c.softmax_scale)
            top = np.sqrt((k ** 2).sum(-1)).max() * np.sqrt((q ** 2).sum(-1)) * c.softmax_scale
            e = 16 * 2.0 ** -22 * top + 2.0 ** -21
            if self.kv == "fp8_e4m3":            # Q as two e4m3 values
                e = e + (2.0 ** -17 * np.abs(q).max(-1) * np.abs(k).sum(-1).max()
                         * c.softmax_scale)
            n = max(max(self.lens), 1)
            tol = (2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2 * e + (n / 4 + 64) * 2.0 ** -24
                                              )[..., None] * mag + 2.0 ** -24)
            err = np.abs(out_all[:T, rows] - out)
            assert np.all(err <= tol), (h, float((err - tol).max()))
            fin = np.isfinite(lse)
            got = lse_all[:T, rows]
            assert np.array_equal(got[~fin], lse[~fin])
            lt = (e + (n / 4 + 64) * 2.0 ** -24)[fin] + 2.0 ** -22 * np.abs(lse[fin])
            assert np.all(np.abs(got[fin] - lse[fin]) <= lt), np.abs(got[fin] - lse[fin]).max()
