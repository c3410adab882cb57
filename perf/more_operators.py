"""Cases of the operators that verify a tree of drafted tokens over a paged
cache, with their plain forms.

Four operators of one step of speculative decoding:

* ``plan``: the nodes' parents become visibility masks and rotary positions;
* ``attention``: every node attends to its request's cached tokens and to its
  ancestors among the step's nodes (bf16, e4m3 or NVFP4 pools);
* ``verify``: the drafted tokens are accepted or refused against the target's
  probabilities, from given random numbers, and the next token is drawn;
* ``commit``: the accepted nodes' rows of every layer's pools move to
  consecutive positions.

Node i of a request with n nodes and length L (nodes included) is stored at
position L - n + i.  ``run`` computes them from elementary torch operations,
or, where ``own`` is true, by the library's calls.
"""
import math

import torch

own = False          # False: plain torch; True: the library's operators

P = 128              # tokens per page
D = 128              # head dim
ROW4 = D // 2 + D // 16
NODES = 64           # nodes a request may have
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
KV_SCALE = {"bf16": 1.0, "fp8_e4m3": 2.0 ** -5, "nvfp4": 0.75}
ROW_BYTES = {"bf16": 2 * D, "fp8_e4m3": D, "nvfp4": ROW4}
# What a drawn case may cost at most: the largest listed ones.
MOST_KEYS = 32 * 20480 * 8          # (key, KV head) pairs of an attention
MOST_PADDED = 32 * 32768 * 8        # the same, requests padded to the longest
MOST_PAIRS = 16 * 20480 * 64 * 32   # (query row, key) pairs
MOST_PAD_PAIRS = 16 * 32768 * 64 * 32
MOST_PROBS = 64 * 16 * 131072       # target probabilities of a verification
MOST_POOL = 32 * (2 * 64 + 3) * 8 * P * 6 * D  # bytes of the pools of a commit


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the nodes of one small tree: the least a step can ask for
        dict(name="plan, 1 x 4 nodes", op="plan", batch=1, min_nodes=4, max_nodes=4, width=3,
             max_len=1500),
        # a serving batch of large ragged trees
        dict(name="plan, 64 x 17-64 nodes", op="plan", batch=64, min_nodes=17, max_nodes=64,
             width=20, max_len=32768),
        # two short chats on one rank of a sharded model: latency counts
        dict(name="attention, 8 nodes x 2 x 1.5k, bf16, 1 KV head", op="attention", batch=2,
             idle=0, min_nodes=8, max_nodes=8, width=4, q_heads=8, kv_heads=1, kv_dtype="bf16",
             min_len=1000, max_len=1500),
        # a serving batch of mixed lengths, trees of 32 nodes
        dict(name="attention, 32 nodes x 16 x 8k-32k, bf16", op="attention", batch=16, idle=0,
             min_nodes=32, max_nodes=32, width=8, q_heads=64, kv_heads=8, kv_dtype="bf16",
             min_len=8192, max_len=32768),
        # one user, a very long document, the largest tree
        dict(name="attention, 64 nodes x 1 x 131071, e4m3", op="attention", batch=1, idle=0,
             min_nodes=64, max_nodes=64, width=20, q_heads=64, kv_heads=8, kv_dtype="fp8_e4m3",
             min_len=131071, max_len=131071),
        # a rank with one KV head of 16 query heads, ragged trees, a batch
        # padded to a captured size by idle requests, first tokens among them
        dict(name="attention, 1-40 nodes x (61 + 3 idle) x 40-6001, e4m3", op="attention",
             batch=61, idle=3, min_nodes=1, max_nodes=40, width=6, q_heads=16, kv_heads=1,
             kv_dtype="fp8_e4m3", min_len=40, max_len=6001),
        # small trees over a 4-bit cache
        dict(name="attention, 6 nodes x 32 x 8k-32k, nvfp4", op="attention", batch=32, idle=0,
             min_nodes=6, max_nodes=6, width=3, q_heads=64, kv_heads=8, kv_dtype="nvfp4",
             min_len=8192, max_len=32768),
        # one request, three drafted tokens in a row, taken as they are
        dict(name="verify, chain of 4, vocab 32000", op="verify", batch=1, min_nodes=4,
             max_nodes=4, width=1, vocab=32000, pad=0, dtype="float32", drawn=False),
        # a serving batch, trees of the draft's best tokens
        dict(name="verify, 64 x 16 nodes, vocab 131072", op="verify", batch=64, min_nodes=16,
             max_nodes=16, width=4, vocab=131072, pad=0, dtype="float32", drawn=False),
        # drafts drawn from the draft model's distribution, ragged trees, an odd
        # vocabulary in padded rows
        dict(name="verify, 24 x 2-12 nodes, vocab 100003, drawn", op="verify", batch=24,
             min_nodes=2, max_nodes=12, width=4, vocab=100003, pad=61, dtype="float32",
             drawn=True),
        # one request, a few layers of a 4-bit cache
        dict(name="commit, 1 x 8 nodes, 4 layers, nvfp4", op="commit", batch=1, min_nodes=8,
             max_nodes=8, width=3, layers=4, kv_heads=8, index_dim=0, kv_dtype="nvfp4",
             max_len=1000),
        # a serving batch, many layers with index keys; the pools hold the
        # trees' own pages (the rest of a context takes no part), nodes on both
        # sides of a page's end
        dict(name="commit, 64 x 16 nodes, 32 layers, bf16", op="commit", batch=64, min_nodes=16,
             max_nodes=16, width=3, layers=32, kv_heads=8, index_dim=128, kv_dtype="bf16",
             max_len=137),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "verify", "verify", "commit", "plan"])
    while True:
        batch = _spread(rng, 1, 64)
        max_nodes = _spread(rng, 1, NODES)
        case = dict(op=op, batch=batch, min_nodes=rng.randint(1, max_nodes), max_nodes=max_nodes,
                    width=rng.choice([1, 2, 3, 4, 6, 20]))
        if op == "plan":
            case.update(max_len=rng.randint(NODES, 131072))
            return case
        if op == "attention":
            kv_heads = rng.choice([1, 2, 4, 8])
            max_len = _spread(rng, NODES, 131072)
            case.update(idle=rng.choice([0, 0, 1, 5]),
                        q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8, 8, 16]), kv_heads=kv_heads,
                        kv_dtype=rng.choice(["bf16", "fp8_e4m3", "nvfp4"]),
                        min_len=rng.randint(max_nodes, max(max_nodes, max_len)), max_len=max_len)
            lens, nodes = _lens(case), _nodes(case)
            most = (batch + case["idle"]) * max_len
            if (max_len >= case["min_len"] and sum(lens) * kv_heads <= MOST_KEYS
                    and most * kv_heads <= MOST_PADDED
                    and sum(a * b for a, b in zip(lens, nodes)) * case["q_heads"] <= MOST_PAIRS
                    and most * max_nodes * case["q_heads"] <= MOST_PAD_PAIRS):
                return case
        if op == "verify":
            case.update(vocab=_spread(rng, 1000, 200000), pad=rng.choice([0, 0, 13, 64]),
                        dtype=rng.choice(["float32", "float32", "bfloat16"]),
                        drawn=rng.random() < 0.5)
            # (padded rows; drawn drafts read a second distribution)
            rows = batch * max_nodes * (4 if case["drawn"] else 1)
            if rows * (case["vocab"] + case["pad"]) <= MOST_PROBS:
                return case
        if op == "commit":
            case.update(layers=rng.choice([1, 2, 4, 8, 16, 32, 61]),
                        kv_heads=rng.choice([1, 2, 4, 8]), index_dim=rng.choice([0, 64, 128]),
                        kv_dtype=rng.choice(["bf16", "fp8_e4m3", "nvfp4"]),
                        max_len=_spread(rng, NODES, 1000))
            pages = sum(-(-L // P) for L in _lens(case)) + 3
            row = 2 * ROW_BYTES[case["kv_dtype"]] + 2 * case["index_dim"]
            if case["layers"] * pages * case["kv_heads"] * P * row <= MOST_POOL:
                return case


def _between(lo, hi, n):
    """n whole numbers of [lo, hi], both ends among them where n is two or more."""
    mid = [lo + int((hi - lo) * ((r * 0.6180339887498949) % 1.0)) for r in range(n)]
    if n > 1:
        mid[0], mid[1] = lo, hi
    return mid


def _nodes(case):
    """The nodes of each request's tree."""
    return _between(case["min_nodes"], case["max_nodes"], case["batch"])


def _lens(case):
    """The requests' lengths, tree nodes included."""
    lo, hi = case.get("min_len", case.get("max_len", NODES)), case.get("max_len", NODES)
    return [max(a, n) for a, n in zip(_between(lo, hi, case["batch"])[::-1], _nodes(case))]


def work(case):
    nodes = _nodes(case)
    tokens = sum(nodes)
    if case["op"] == "plan":
        return {"bytes": tokens * (4 + 8 + 8), "flops": tokens * 2}
    if case["op"] == "attention":
        hq, hkv, lens = case["q_heads"], case["kv_heads"], _lens(case)
        T = tokens + case["idle"]
        seen = sum(n * (L - n) + n * min(n, 4) for n, L in zip(nodes, lens))   # (node, key) pairs
        return {"bytes": sum(lens) * hkv * 2 * ROW_BYTES[case["kv_dtype"]]
                + T * (hq * (4 * D + 4) + 8) + 4 * sum(-(-L // P) for L in lens),
                "flops": seen * hq * 4 * D}
    if case["op"] == "verify":
        size, rows = (4 if case["dtype"] == "float32" else 2), (2 if case["drawn"] else 1)
        # one row of the residual a request, the drafts' own entries
        return {"bytes": case["batch"] * case["vocab"] * rows * size + tokens * (12 + rows * size),
                "flops": case["batch"] * case["vocab"] * 2 * rows}
    # at most the deepest path moves; half of it is what is counted here
    moved = sum(max(1, _depth(n, case["width"]) // 2) for n in nodes)
    row = 2 * ROW_BYTES[case["kv_dtype"]] + 2 * case["index_dim"]
    return {"bytes": 2 * moved * case["layers"] * case["kv_heads"] * row + 8 * tokens, "flops": 0}


def _depth(nodes, width):
    """About the depth of a tree of `nodes` nodes whose parents lie up to `width` back."""
    return int(2 * nodes / (width + 1))


# ------------------------------------------------------------------ inputs
def _normal_codes(shape, gen, dev):
    """Bytes of two E2M1 codes each, as 16-element blocks of normal values
    have them under a scale of a sixth of their largest magnitude."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * (1.8 / 6)
    q = torch.special.erf(edges / math.sqrt(2))
    u = (torch.arange(512, dtype=torch.float64) + 0.5) / 512
    mag = torch.searchsorted(q, u)
    table = torch.cat([mag, mag + 8]).to(torch.uint8).to(dev)      # equally likely codes
    out = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat = out.view(-1)
    step = 1 << 27
    for at in range(0, flat.numel(), step):      # in pieces: the indices are wider than the codes
        n = min(step, flat.numel() - at)
        two = torch.randint(0, 1 << 20, (n,), generator=gen, device=dev, dtype=torch.int32)
        flat[at:at + n] = table[two & 1023] | (table[two >> 10] << 4)
    return out


def _pools(shape, kv_dtype, gen, dev):
    """K and V pools [..., H_kv, P, D]; for NVFP4 one pool of [..., 2 H_kv, P, 72]
    bytes that holds both (slot 2h the keys of head h, 2h + 1 its values)."""
    lead, heads = shape[:-1], shape[-1]
    if kv_dtype == "nvfp4":
        pool = torch.empty((*lead, 2 * heads, P, ROW4), dtype=torch.uint8, device=dev)
        pool[..., :D // 2] = _normal_codes((*lead, 2 * heads, P, D // 2), gen, dev)
        pool[..., D // 2:] = torch.randint(0x28, 0x39, (*lead, 2 * heads, P, D // 16),
                                           generator=gen, device=dev, dtype=torch.uint8)
        return pool, pool
    dt = torch.bfloat16 if kv_dtype == "bf16" else torch.float8_e4m3fn
    both = []
    for _ in range(2):
        x = torch.empty((*lead, heads, P, D), dtype=dt, device=dev)
        flat = x.view(-1)
        step = 1 << 28
        for at in range(0, flat.numel(), step):
            n = min(step, flat.numel() - at)
            flat[at:at + n] = (torch.randn(n, generator=gen, device=dev)
                               / KV_SCALE[kv_dtype]).to(dt)
        both.append(x)
    return both


def _pair_table(dev):
    """[256, 2] fp32: the two values of a byte of E2M1 codes, low nibble first."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    b = torch.arange(256, device=dev)
    return torch.stack([v[b & 15], v[b >> 4]], dim=1)


def _trees(s, gen, dev):
    """Ragged trees, request after request: node 0 the root, the parent of node i
    one of the `width` nodes before it; idle requests have no nodes."""
    c = s["case"]
    nodes = _nodes(c) + [0] * c.get("idle", 0)
    n = torch.tensor(nodes, device=dev)
    B, N = len(nodes), max(nodes)
    i = torch.arange(N, device=dev)
    back = 1 + (torch.rand((B, N), generator=gen, device=dev) * c["width"]).long()
    par = (i - back).clamp(min=0)
    par[:, 0] = -1
    on = i[None, :] < n[:, None]
    cu = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    cu[1:] = n.cumsum(0)
    lens = _lens(c) + [0] * c.get("idle", 0)
    s.update(nodes=n, on=on, cu=cu, parents=par[on].to(torch.int32),
             cu_seqlens_q=cu.to(torch.int32), most=N, tokens=sum(nodes),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             # the (request, node) of every token, and the token of every padded place
             req=torch.repeat_interleave(torch.arange(B, device=dev), n),
             at=(cu[:-1, None] + i[None, :]).clamp(max=max(sum(nodes) - 1, 0)))
    s["node"] = i[None, :].expand(B, N)[on]
    return lens


def _table(s, lens, gen, dev, spare):
    """A block table of scattered pages; returns the pages of the pool."""
    nb = [-(-L // P) for L in lens]
    pages = sum(nb) + spare
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table, at = torch.full((len(lens), max(nb)), -1, dtype=torch.int32, device=dev), 0
    for r, k in enumerate(nb):
        table[r, :k] = perm[at:at + k]
        at += k
    s["block_table"] = table
    return pages


def _ancestors(par, steps):
    """[B, N, N] truth: node j is node i or an ancestor of it, from padded parents."""
    B, N = par.shape
    see = torch.eye(N, dtype=torch.bool, device=par.device).expand(B, N, N)
    step = (par[:, :, None] == torch.arange(N, device=par.device)) | see       # i itself, its parent
    see = step.float()
    for _ in range(steps):                       # twice as far each time
        see = ((see @ see) > 0).float()
    return see > 0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case)
    lens = _trees(s, gen, dev)
    s["steps"] = max(1, math.ceil(math.log2(s["most"] + 1)))
    # parents by (request, node); places past a tree's end have none
    s["par"] = torch.where(s["on"], s["parents"].long()[s["at"]], -1)
    op = case["op"]
    if op == "plan":
        if own:
            _own_plan(s, lens)
        return s
    if op == "attention":
        T, hq, hkv = s["tokens"], case["q_heads"], case["kv_heads"]
        pages = _table(s, lens, gen, dev, 7)
        see = _ancestors(s["par"], s["steps"])
        bits = torch.ones((), dtype=torch.int64, device=dev) << torch.arange(s["most"], device=dev)
        mask = torch.where(see, bits, 0).sum(-1)[s["on"]]
        # every 11th node is an unused place of its tree: it sees the prefix alone
        blank = torch.arange(T, device=dev) % 11 == 10
        s["tree_mask"] = torch.where(blank, 0, mask)
        s["q"] = (2.0 * torch.randn((T, hq, D), generator=gen, device=dev)).to(torch.bfloat16)
        s["k_pages"], s["v_pages"] = _pools((pages, hkv), case["kv_dtype"], gen, dev)
        s.update(pairs=_pair_table(dev), kv_scale=KV_SCALE[case["kv_dtype"]],
                 softmax_scale=D ** -0.5)
        if own:
            _own_attention(s, pages)
        return s
    if op == "verify":
        _probabilities(s, gen, dev)
        if own:
            _own_verify(s)
        return s
    # commit: a path of every request's tree, from the root to a random node
    pages = _table(s, lens, gen, dev, 3)
    see = _ancestors(s["par"], s["steps"])
    tip = (torch.rand(len(lens), generator=gen, device=dev) * s["nodes"]).long()
    path = see[torch.arange(len(lens), device=dev), tip]                       # [B, N] truth
    s["num_accepted"] = path.sum(1).to(torch.int32)
    s["accepted"] = torch.full((len(lens), NODES), -1, dtype=torch.int32, device=dev)
    order = torch.argsort(~path, dim=1, stable=True).to(torch.int32)           # the path's nodes first
    j = torch.arange(s["most"], device=dev)
    s["accepted"][:, :s["most"]] = torch.where(j < s["num_accepted"][:, None], order, -1)
    lead, hkv = (case["layers"], pages), case["kv_heads"]
    s["k_pages"], s["v_pages"] = _pools((*lead, hkv), case["kv_dtype"], gen, dev)
    if case["index_dim"]:
        s["idx_k_pages"] = torch.empty((*lead, hkv, P, case["index_dim"]), device=dev,
                                       dtype=torch.bfloat16).normal_(generator=gen)
    if own:
        _own_commit(s, pages)
    return s


def _probabilities(s, gen, dev):
    """Target (and draft) distributions of a language model's shape, and drafted
    tokens that the target often takes."""
    c = s["case"]
    T, V = s["tokens"], c["vocab"]
    dt = getattr(torch, c["dtype"])
    x = torch.randn((T, V), generator=gen, device=dev).mul_(3.0)
    s["target"] = torch.zeros((T, V + c["pad"]), dtype=dt, device=dev)[:, :V]  # padded rows
    s["target"].copy_(torch.softmax(x, dim=1))
    x += torch.randn((T, V), generator=gen, device=dev).mul_(0.7)              # the draft's idea
    up = s["cu"][s["req"]] + s["parents"].long().clamp(min=0)                  # token of the parent
    # how many children of its parent come before a node
    same = (s["req"][:, None] == s["req"]) & (s["parents"][:, None] == s["parents"])
    rank = (same & (s["node"][:, None] > s["node"])).sum(1)
    s["children"] = int(rank.max()) + 1
    s["rank"] = rank
    if c["drawn"]:
        s["draft"] = torch.zeros((T, V + c["pad"]), dtype=dt, device=dev)[:, :V]
        s["draft"].copy_(torch.softmax(x, dim=1))
        ids = torch.multinomial(s["draft"].float(), s["children"], replacement=True, generator=gen)
    else:
        ids = torch.topk(x, s["children"], dim=1).indices
    s["tokens_"] = ids[up, rank].to(torch.int32)
    s["uniform"] = torch.rand(T, generator=gen, device=dev)
    s["uniform_final"] = torch.rand(len(s["nodes"]), generator=gen, device=dev)


def _config(s, msa, pages, **kw):
    kw = {**dict(num_q_heads=8, num_kv_heads=8, kv_dtype="bf16"), **kw}
    return msa.make_config(init_blocks=1, local_blocks=1, topk_blocks=0, max_batch=len(s["nodes"]),
                           max_q_tokens=s["tokens"], num_pages=pages,
                           max_blocks_per_req=s["block_table"].shape[1],
                           **{**dict(index_dim=128), **kw})


def _own_plan(s, lens):
    """The step's plan, in the workspace that a serving program keeps."""
    import block_sparse_paged_msa_gb300 as msa
    dev = s["parents"].device
    s["block_table"] = torch.zeros((len(lens), -(-max(lens) // P)), dtype=torch.int32, device=dev)
    s["cfg"] = _config(s, msa, 1)
    _plan(s, msa)
    s["mask_out"] = torch.empty(s["tokens"], dtype=torch.int64, device=dev)
    s["pos_out"] = torch.empty(s["tokens"], dtype=torch.int64, device=dev)


def _plan(s, msa):
    s["ws"] = torch.empty(msa.workspace_bytes(s["cfg"]), dtype=torch.uint8,
                          device=s["parents"].device)
    msa.plan(s["cfg"], s["seq_lens"], s["block_table"], s["ws"], s["cu_seqlens_q"])


def _own_attention(s, pages):
    import block_sparse_paged_msa_gb300 as msa
    c = s["case"]
    cfg = _config(s, msa, pages, num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"],
                  kv_dtype=c["kv_dtype"], softmax_scale=s["softmax_scale"],
                  k_scale=s["kv_scale"], v_scale=s["kv_scale"])
    s["layer"] = msa.TreeAttention(cfg)
    msa.plan(cfg, s["seq_lens"], s["block_table"], s["layer"].ws, s["cu_seqlens_q"])


def _own_verify(s):
    import block_sparse_paged_msa_gb300 as msa
    dev, B = s["parents"].device, len(s["nodes"])
    s["block_table"] = torch.zeros((B, 1), dtype=torch.int32, device=dev)
    s["cfg"] = _config(s, msa, 1)
    _plan(s, msa)
    s["accepted"] = torch.empty((B, NODES), dtype=torch.int32, device=dev)
    s["num_accepted"] = torch.empty(B, dtype=torch.int32, device=dev)
    s["out_tokens"] = torch.empty((B, NODES), dtype=torch.int32, device=dev)


def _own_commit(s, pages):
    import block_sparse_paged_msa_gb300 as msa
    c = s["case"]
    kw = dict(index_dim=c["index_dim"]) if c["index_dim"] else {}
    s["cfg"] = _config(s, msa, pages, num_q_heads=c["kv_heads"], num_kv_heads=c["kv_heads"],
                       kv_dtype=c["kv_dtype"], **kw)
    _plan(s, msa)
    for name in ("k_pages", "v_pages", "idx_k_pages"):
        s["layers_" + name] = list(s[name].unbind(0)) if name in s else None


# ------------------------------------------------------------------ the operators
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _run_plan(s):
    import block_sparse_paged_msa_gb300 as msa
    msa.tree_plan(s["cfg"], s["ws"], s["parents"], s["mask_out"], s["pos_out"])
    return s["mask_out"], s["pos_out"]


def _run_attention(s):
    import block_sparse_paged_msa_gb300 as msa
    y = s["layer"]
    msa.tree_attention(y.cfg, y.ws, s["q"], s["k_pages"], s["v_pages"], s["tree_mask"], y.scratch,
                       y.out, y.lse)
    return y.out, y.lse


def _run_verify(s):
    import block_sparse_paged_msa_gb300 as msa
    msa.tree_verify(s["cfg"], s["ws"], s["parents"], s["tokens_"], s["target"], s["uniform"],
                    s["uniform_final"], s["accepted"], s["num_accepted"], s["out_tokens"],
                    draft_probs=s.get("draft"))
    return s["accepted"], s["num_accepted"], s["out_tokens"]


def _run_commit(s):
    import block_sparse_paged_msa_gb300 as msa
    msa.tree_commit(s["cfg"], s["ws"], s["accepted"], s["num_accepted"], s["layers_k_pages"],
                    s["layers_v_pages"], s["layers_idx_k_pages"])
    return _pools_of(s)


def _values(codes, scales, pairs):
    """fp32 values of E2M1 code bytes [..., 64] under E4M3 scale bytes [..., 8]."""
    v = pairs[codes.int()]                                          # [..., 64, 2]
    v = v.view(*codes.shape[:-1], D // 16, 16)
    v = v * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return v.view(*codes.shape[:-1], D)


def _pools_of(s):
    """The pools as they are: a commit moves rows and rounds nothing, so that a
    4-bit pool's bytes have to be equal (and their values with them)."""
    both = (s["k_pages"],) if s["case"]["kv_dtype"] == "nvfp4" else (s["k_pages"], s["v_pages"])
    return both + ((s["idx_k_pages"],) if s["case"]["index_dim"] else ())


def _plan_plain(s):
    see = _ancestors(s["par"], s["steps"])
    j = torch.arange(s["most"], device=see.device)
    mask = torch.where(see, torch.ones_like(j) << j, 0).sum(-1)
    base = s["seq_lens"].long() - s["nodes"]
    pos = base[:, None] + see.sum(-1) - 1
    return mask[s["on"]], pos[s["on"]]


def _attention_plain(s):
    c = s["case"]
    hq, hkv, N = c["q_heads"], c["kv_heads"], s["most"]
    B, width = s["block_table"].shape
    G, keys = hq // hkv, width * P
    pages = s["block_table"].clamp(min=0).long()
    if c["kv_dtype"] == "nvfp4":
        rows = s["k_pages"][pages].view(B, width, hkv, 2, P, ROW4).permute(3, 0, 2, 1, 4, 5)
        kv = _values(rows[..., :D // 2], rows[..., D // 2:], s["pairs"]) * s["kv_scale"]
        k, v = kv.reshape(2, B, hkv, keys, D)
    else:
        k, v = ((s[n].view(torch.uint8)[pages].view(s[n].dtype).permute(0, 2, 1, 3, 4)
                 .reshape(B, hkv, keys, D).float() * s["kv_scale"]) for n in ("k_pages", "v_pages"))
    q = s["q"][s["at"]].float().view(B, N, hkv, G, D).permute(0, 2, 1, 3, 4)
    x = (q.reshape(B, hkv, N * G, D) @ k.transpose(2, 3)) * s["softmax_scale"]
    # key u of request r: a prefix token, or node u - base
    u = torch.arange(keys, device=x.device) - (s["seq_lens"].long() - s["nodes"])[:, None]
    mask = s["tree_mask"][s["at"]]                                  # [B, N]
    bit = (mask[:, :, None] >> u.clamp(0, 63)[:, None, :]) & 1
    seen = (u < 0)[:, None, :] | ((bit == 1) & (u < s["nodes"][:, None])[:, None, :])
    x = x.view(B, hkv, N, G, keys).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp_(x.sub_(base))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, N * G, keys) @ v).view(B, hkv, N, G, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (base + torch.log(total))[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4)[s["on"]], lse.permute(0, 2, 1, 3)[s["on"]]
    return o.reshape(-1, hq, D).to(torch.bfloat16), lse.reshape(-1, hq)


def _verify_plain(s):
    c = s["case"]
    B, N, T = len(s["nodes"]), s["most"], s["tokens"]
    dev = s["parents"].device
    tok, node, req = s["tokens_"].long(), s["node"], s["req"]
    up = s["cu"][req] + s["parents"].long().clamp(min=0)            # the parent's token
    child = node > 0
    p = s["target"][up, tok].double()                               # [T] target's p of each draft
    u = s["uniform"].double()
    # weights of the siblings' residual, as the earlier children are refused
    gone = torch.zeros(T, dtype=torch.float64, device=dev)          # A of the parent's row
    if c["drawn"]:
        q = s["draft"][up, tok].double()
        left = torch.ones(T, dtype=torch.float64, device=dev)       # Z, by parent token
        taken = torch.zeros(T, dtype=torch.float64, device=dev)     # A, by parent token
        yes = torch.zeros(T, dtype=torch.bool, device=dev)
        many = torch.zeros(T, dtype=torch.long, device=dev).index_add_(0, up[child],
                                                                       torch.ones_like(up[child]))
        for k in range(s["children"]):           # the k-th children of all nodes
            it = child & (s["rank"] == k)
            w = (p - taken[up] * q).clamp(min=0)
            yes = torch.where(it, u * q * left[up] < w, yes)
            rows = torch.nonzero(many > k)[:, 0]                    # refused by now
            taken[rows] += left[rows]
            left[rows] = (s["target"][rows].double()
                          - taken[rows, None] * s["draft"][rows].double()).clamp_(min=0).sum(1)
        gone = taken
    else:
        same = (up[:, None] == up) & child & child[:, None] & (node[:, None] > node)
        twin = (same & (tok[:, None] == tok)).any(1)                # its token was refused before
        w = torch.where(twin, 0.0, p)
        left = 1.0 - (same.double() @ w[:, None])[:, 0]
        yes = child & (u * left < w)
    # a node is on the path if it and all its ancestors are the first accepted children
    sib = (up[:, None] == up) & child & child[:, None] & (node[:, None] > node)
    first = yes & ~(sib & yes).any(1)
    first = (first | (node == 0))[s["at"]] & s["on"]
    see = _ancestors(s["par"], s["steps"])
    path = (see <= first[:, None, :]).all(-1) & s["on"]             # [B, N]
    num = path.sum(1)
    j = torch.arange(N, device=dev)
    order = torch.argsort(~path, dim=1, stable=True)
    acc = torch.full((B, NODES), -1, dtype=torch.int64, device=dev)
    acc[:, :N] = torch.where(j < num[:, None], order, -1)
    tip = torch.where(path, j, -1).amax(1)                          # the path's last node
    row = s["cu"][:-1] + tip
    # what is left of the target's distribution there
    w = s["target"][row].double()
    if c["drawn"]:
        w = (w - gone[row, None] * s["draft"][row].double()).clamp_(min=0)
    else:
        kids = (s["parents"].long()[s["at"]] == tip[:, None]) & s["on"]         # [B, N]
        refused = torch.zeros((B, c["vocab"] + 1), dtype=torch.bool, device=dev)
        refused.scatter_(1, torch.where(kids, tok[s["at"]], c["vocab"]), True)
        w = w.masked_fill_(refused[:, :c["vocab"]], 0.0)
    cum = w.cumsum(1)
    last = (cum <= s["uniform_final"].double()[:, None] * cum[:, -1:]).sum(1)
    out = torch.full((B, NODES + 1), -1, dtype=torch.int64, device=dev)
    drafted = tok[(s["cu"][:-1, None] + acc.clamp(min=0)).clamp(max=T - 1)]
    out[:, :NODES] = torch.where(acc >= 0, drafted, -1)
    out = out[:, 1:].scatter(1, num[:, None] - 1, last[:, None])    # the root's token is not new
    return acc.int(), num.int(), out.int()


def _commit_plain(s):
    c = s["case"]
    B, N = len(s["nodes"]), s["most"]
    j = torch.arange(N, device=s["parents"].device)
    on = j < s["num_accepted"][:, None]
    base = (s["seq_lens"].long() - s["nodes"])[:, None]

    def place(node):                             # page and row of the cache position of a node
        pos = (base + node)[on]
        r = torch.arange(B, device=pos.device)[:, None].expand(B, N)[on]
        return s["block_table"].long()[r, pos // P], pos % P

    src, dst = place(s["accepted"][:, :N].long()), place(j.expand(B, N))

    def move(pool):
        pool[:, dst[0], :, dst[1]] = pool[:, src[0], :, src[1]]

    move(s["k_pages"].view(torch.uint8))         # bytes: a copy of rows, not of numbers
    if c["kv_dtype"] != "nvfp4":
        move(s["v_pages"].view(torch.uint8))
    if c["index_dim"]:
        move(s["idx_k_pages"])
    return _pools_of(s)


_OWN = dict(plan=_run_plan, attention=_run_attention, verify=_run_verify, commit=_run_commit)
_PLAIN = dict(plan=_plan_plain, attention=_attention_plain, verify=_verify_plain,
              commit=_commit_plain)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _attention_exact(s)
    if case["op"] == "verify":
        return _verify_exact(s)
    return None          # whole numbers, and rows that are moved as they are


def _attention_exact(s):
    """Textbook softmax attention, a request and a KV head at a time."""
    c = s["case"]
    hq, hkv = c["q_heads"], c["kv_heads"]
    G, dev = hq // hkv, s["q"].device
    mags = torch.tensor(E2M1, dtype=torch.float64, device=dev)
    out = torch.zeros((s["tokens"], hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((s["tokens"], hq), -math.inf, dtype=torch.float64, device=dev)

    def decode(tile):                            # rows of a pool -> [m, 128]
        if c["kv_dtype"] != "nvfp4":
            return tile.to(torch.float64) * s["kv_scale"]
        byte = tile[:, :D // 2].long()
        nib = torch.stack([byte % 16, byte // 16], dim=2).reshape(len(tile), D)
        val = mags[nib % 8] * (1.0 - 2.0 * (nib // 8).double())
        code = tile[:, D // 2:].long()           # E4M3 by its fields (no NaN codes here)
        e, m = (code // 8) % 16, (code % 8).double()
        sc = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, e.double() - 7), m / 8 * 2.0 ** -6)
        return val * sc.repeat_interleave(16, dim=1) * s["kv_scale"]

    masks = s["tree_mask"].tolist()
    for r, (L, n) in enumerate(zip(s["seq_lens"].tolist(), s["nodes"].tolist())):
        if n == 0:
            continue
        t0 = int(s["cu"][r])
        pages = s["block_table"][r, :-(-L // P)].long()
        seen = torch.tensor([[False if m >> j & 1 else True for j in range(n)]
                             for m in masks[t0:t0 + n]], device=dev)
        for h in range(hkv):
            both = []
            for name, slot in (("k_pages", 2 * h), ("v_pages", 2 * h + 1)):
                pool = s[name][:, slot if c["kv_dtype"] == "nvfp4" else h]
                tile = pool.view(torch.uint8)[pages].view(pool.dtype).reshape(L + (-L) % P, -1)[:L]
                both.append(decode(tile))
            q = s["q"][t0:t0 + n, h * G:(h + 1) * G].double()
            z = torch.einsum("igd,ud->igu", q, both[0]) * s["softmax_scale"]
            z[:, :, L - n:] = z[:, :, L - n:].masked_fill(seen[:, None, :], -math.inf)
            e = torch.logsumexp(z, dim=2)
            lse[t0:t0 + n, h * G:(h + 1) * G] = e
            w = torch.exp(z - torch.where(e == -math.inf, 0.0, e)[:, :, None])
            out[t0:t0 + n, h * G:(h + 1) * G] = torch.einsum("igu,ud->igd", w, both[1])
    return out, lse


def _verify_exact(s):
    """The walk itself, request by request."""
    B = len(s["nodes"])
    acc = torch.full((B, NODES), -1, dtype=torch.int32)
    out = torch.full((B, NODES), -1, dtype=torch.int32)
    num = torch.zeros(B, dtype=torch.int32)
    par, tok = s["parents"].tolist(), s["tokens_"].tolist()
    u, uf = s["uniform"].tolist(), s["uniform_final"].tolist()
    for r in range(B):
        t0, n, x, got = int(s["cu"][r]), int(s["nodes"][r]), 0, [0]
        while True:
            p = s["target"][t0 + x].double()
            q = s["draft"][t0 + x].double() if "draft" in s else None
            w, z, a, nxt = p.clone(), 1.0, 0.0, None
            for i in (i for i in range(1, n) if par[t0 + i] == x):
                y = tok[t0 + i]
                if u[t0 + i] * (1.0 if q is None else float(q[y])) * z < float(w[y]):
                    nxt = i
                    break
                if q is None:
                    z -= float(w[y])
                    w[y] = 0.0
                else:
                    a += z
                    w = (p - a * q).clamp(min=0)
                    z = float(w.sum())
            if nxt is None:
                break
            x = nxt
            got.append(x)
        cum = torch.cumsum(w, 0)
        num[r] = len(got)
        acc[r, :len(got)] = torch.tensor(got, dtype=torch.int32)
        new = [tok[t0 + i] for i in got[1:]]
        new.append(int(torch.searchsorted(cum, uf[r] * float(cum[-1]), right=True)))
        out[r, :len(new)] = torch.tensor(new, dtype=torch.int32)
    return acc, num, out
