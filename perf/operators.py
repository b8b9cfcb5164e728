"""The operators of one speculative-decoding step over the two-pool KV cache, as
measured cases: what a step runs before, in and after its verification.

* ``qknorm``: RMSNorm of every query and key head, the position rotation, and
  the store of K and V into the layer's pool, for prompts and for drafted
  tokens (``swa_qk_norm_rope_store``).
* ``tree``: attention of every node of each request's drafted token tree over
  the request's cached keys and the node's own ancestors
  (``swa_tree_plan`` + ``swa_attn_tree``).
* ``commit``: after verification, the accepted nodes' K/V rows of all layers
  moved to the positions that follow the prefix (``swa_commit_tree``).
* ``copy``: K/V rows of all layers copied between slots, as a fork of a request
  needs for its open page (``swa_copy_kv``).

``own`` is set by whoever measures: False runs the plain torch form, True the
library's calls.  Shapes are those of the library's own workloads (MiMo-,
GPT-OSS-, Llama4-shaped and Tiny).
"""
import math
import random

import numpy as np
import torch

own = False

FULL, SLIDING, CHUNKED = 0, 1, 2
E4M3_MAX = 448.0

# Head shapes of the library's workloads: query heads, head size, stored type,
# page size, and (kind, window, KV heads) of a full and of a windowed layer.
SHAPES = {
    "tiny": dict(hq=4, d=64, dtype="f32", ps=1, full=(FULL, 0, 1), win=(SLIDING, 15, 1)),
    "mimo": dict(hq=64, d=128, dtype="bf16", ps=64, full=(FULL, 0, 4), win=(SLIDING, 127, 8)),
    "gptoss": dict(hq=64, d=64, dtype="bf16", ps=16, full=(FULL, 0, 8), win=(SLIDING, 127, 8)),
    "llama4": dict(hq=40, d=128, dtype="e4m3", ps=64, full=(FULL, 0, 8), win=(CHUNKED, 8192, 8)),
}
ESIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # The library's smallest configuration: two requests of 37 and 200
        # tokens, eight drafted nodes each; latency is all that counts.
        dict(name="tree_tiny_f32", op="tree", shape="tiny", layer="full", bs=2, lo=37, hi=200, nodes=8, spread="ends"),
        # One full layer of a serving batch: 64 requests of 4K to 32K tokens,
        # eight nodes each (128 query rows share every key).
        dict(name="tree_mimo_full", op="tree", shape="mimo", layer="full", bs=64, lo=4096, hi=32768, nodes=8, spread="uniform"),
        # A sliding layer of the same batch (39 of the model's 48): 128 keys
        # and the tree, so launch latency counts.
        dict(name="tree_mimo_sliding", op="tree", shape="mimo", layer="win", bs=64, lo=512, hi=4096, nodes=8, spread="uniform"),
        # Ragged trees of up to 13 nodes, head size 64, pages of 16.
        dict(name="tree_gptoss_ragged", op="tree", shape="gptoss", layer="full", bs=128, lo=1024, hi=16384, nodes=13, spread="log"),
        # Long contexts in FP8: 16 nodes x 5 heads share a key.
        dict(name="tree_llama4_e4m3", op="tree", shape="llama4", layer="full", bs=4, lo=131072, hi=131072, nodes=16, spread="uniform"),
        # One user with a long context and a wide tree: few (request, head)
        # pairs, so the keys have to be split, and 1024 query rows for each.
        dict(name="tree_one_long", op="tree", shape="mimo", layer="full", bs=1, lo=131072, hi=131072, nodes=64, spread="uniform"),
        # Drafted tokens of 64 requests (8 each) entering a full layer.
        dict(name="qknorm_decode", op="qknorm", shape="mimo", layer="full", n=512, rot=128, interleaved=False),
        # A prefill chunk round of 4 x 8192 tokens entering a sliding layer.
        dict(name="qknorm_prefill", op="qknorm", shape="mimo", layer="win", n=32768, rot=128, interleaved=False),
        # FP8 pools: encoded as they are stored; rotation of half the head,
        # neighbouring dims paired.
        dict(name="qknorm_e4m3", op="qknorm", shape="llama4", layer="win", n=4099, rot=64, interleaved=True),
        # End of a verification: 64 requests keep up to 7 of 16 nodes, all 48 layers.
        dict(name="commit_mimo", op="commit", shape="mimo", full=9, win=39, bs=64, prefix=100, nodes=16, keep=7),
        # The same for two requests of the smallest configuration.
        dict(name="commit_tiny", op="commit", shape="tiny", full=1, win=1, bs=2, prefix=37, nodes=8, keep=3),
        # 32 forks, each copying its open page's rows in all layers.
        dict(name="copy_fork", op="copy", shape="mimo", full=9, win=39, n=32 * 47, pool=8192),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "qknorm", "qknorm", "commit", "copy"])
    name = rng.choice(["mimo", "mimo", "gptoss", "llama4"] if op in ("tree", "qknorm") else ["mimo", "tiny"])
    if op == "tree":
        layer = rng.choice(["full", "full", "win"])
        bs = _logint(rng, 1, 96)
        # at most 1M cached tokens (sliding layers 256K) in the batch
        top = max(40, min(131072, (1048576 if layer == "full" else 262144) // bs))
        hi = _logint(rng, 33, top)
        return dict(op=op, shape=name, layer=layer, bs=bs, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                    nodes=_logint(rng, 1, 64 if bs <= 16 else 16), spread=rng.choice(["uniform", "log"]))
    if op == "qknorm":
        d = SHAPES[name]["d"]
        return dict(op=op, shape=name, layer=rng.choice(["full", "win"]), n=_logint(rng, 1, 32768),
                    rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5)
    big = name == "mimo"
    if op == "commit":
        nodes = rng.randint(2, 48)
        return dict(op=op, shape=name, full=rng.randint(1, 9) if big else 1, win=rng.randint(1, 39) if big else 1,
                    bs=_logint(rng, 1, 64), prefix=rng.randint(1, 100), nodes=nodes, keep=rng.randint(1, min(nodes, 12)))
    return dict(op=op, shape=name, full=rng.randint(1, 9) if big else 1, win=rng.randint(1, 39) if big else 1,
                n=_logint(rng, 1, 2000), pool=8192)


# ------------------------------------------------------------------ shapes ---
def _lens(case):
    """Cached tokens of each request and nodes of each tree: fixed by the case."""
    r = random.Random(case["bs"] * 1000003 + case["hi"] * 31 + case["nodes"])
    lo, hi = case["lo"], case["hi"]
    if case["spread"] == "ends":
        pre = [lo if b % 2 == 0 else hi for b in range(case["bs"])]
    elif case["spread"] == "log":
        pre = [_logint(r, lo, hi) for _ in range(case["bs"])]
    else:
        pre = [r.randint(lo, hi) for _ in range(case["bs"])]
    pre[-1] = hi
    n = case["nodes"]
    ragged = case["shape"] == "gptoss" and n > 1
    return pre, [r.randint(1, n) if ragged else n for _ in range(case["bs"])]


def _layer(case):
    s = SHAPES[case["shape"]]
    return s, s[case["layer"]]


def _kept(case):
    r = random.Random(case["bs"] * 7919 + case["nodes"])
    return [r.randint(0, case["keep"]) for _ in range(case["bs"])]


def work(case):
    s = SHAPES[case["shape"]]
    e, io = ESIZE[s["dtype"]], 4 if s["dtype"] == "f32" else 2
    d, hq = s["d"], s["hq"]
    if case["op"] == "tree":
        kind, w, hkv = s[case["layer"]]
        pre, nodes = _lens(case)
        keys = [t + (p if kind == FULL else min(p, w) if kind == SLIDING else p % w) for p, t in zip(pre, nodes)]
        n = sum(nodes)
        return {"bytes": 2 * hkv * d * e * sum(keys) + 2 * n * hq * d * io + 4 * n,
                "flops": 4 * hq * d * sum(k * t for k, t in zip(keys, nodes))}
    if case["op"] == "qknorm":
        _, _, hkv = s[case["layer"]]
        n = case["n"]
        # inputs, q out, stored K and V, one row of the angle table and the slots
        return {"bytes": n * ((hq + 2 * hkv) * d * io + hq * d * io + 2 * hkv * d * e + 4 * case["rot"] + 16),
                "flops": n * ((hq + hkv) * d * 8)}
    rows = sum(_kept(case)) if case["op"] == "commit" else case["n"]
    per = 2 * d * e * (case["full"] * s["full"][2] + case["win"] * s["win"][2])
    return {"bytes": 2 * rows * per, "flops": 0}


# ------------------------------------------------------------------ inputs ---
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pool(g, shape, dtype):
    """A filled K or V pool: about N(0, 1) values; FP8 as raw bytes."""
    if dtype == "f32":
        return torch.randn(shape, generator=g, device="cuda")
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if dtype == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)


def _pages(seq, ps, seed, window=0):
    """Page tables of a batch whose requests were allocated one after another from
    seeded, permuted free lists of both pools: req_to_token (row b + 1 is request b)
    and full_to_swa.  The pools hold at least one window."""
    need = [-(-t // ps) for t in seq]
    n_pages = max(sum(need) + 2, window // ps + 3)
    rng = np.random.RandomState(seed % (1 << 31))
    pf, pw = rng.permutation(n_pages) + 1, rng.permutation(n_pages) + 1
    size = n_pages * ps
    at = np.concatenate([[0], np.cumsum(need)])
    width = -(-(max(seq) + 1) // 64) * 64
    rt = np.zeros((len(seq) + 1, width), np.int32)
    for b, t in enumerate(seq):
        j = np.arange(t)
        rt[b + 1, :t] = pf[at[b] + j // ps] * ps + j % ps
    mapping = np.zeros(size + ps, np.int64)
    used = at[-1]
    off = np.arange(ps)
    mapping[(pf[:used, None] * ps + off).reshape(-1)] = (pw[:used, None] * ps + off).reshape(-1)
    dev = lambda a: torch.tensor(a, device="cuda")  # noqa: E731
    return dict(size=size, pf=dev(pf.astype(np.int64)), pw=dev(pw.astype(np.int64)), rt=dev(rt), mapping=dev(mapping))


def _tree_parents(r, n):
    """A drafted tree: node 0 the last sampled token, later nodes below recent ones, some at the root."""
    return [-1] + [max(0, i - 1 - r.randrange(min(i, 5))) if r.random() < 0.9 else 0 for i in range(1, n)]


def _context(case, st, layers, seq):
    """The library's handle of a program with these pools, its requests allocated through the library."""
    from hybrid_sliding_window_gb300 import api
    s = SHAPES[case["shape"]]
    t = st["tables"]
    dt = {"f32": api.DTYPE_F32, "bf16": api.DTYPE_BF16, "e4m3": api.DTYPE_E4M3}[s["dtype"]]
    ctx = api.SwaCtx([dict(kind=k, window=w, num_kv_heads=h, k=kk, v=vv) for (k, w, h), kk, vv in layers], s["ps"],
                     t["size"], t["size"], s["hq"], s["d"], dt, max_batch=max(len(seq), 1), init_free_full=t["pf"], init_free_swa=t["pw"])
    bs = len(seq)
    rt = torch.zeros_like(t["rt"])
    rows = torch.arange(1, bs + 1, device="cuda")
    n = int(sum(seq))
    f, w = (torch.empty(n, dtype=torch.int64, device="cuda") for _ in range(2))
    api.swa_alloc_extend(ctx, torch.zeros(bs, dtype=torch.int64, device="cuda"), torch.tensor(seq, device="cuda"), None,
                         np.zeros(bs, np.int64), np.asarray(seq, np.int64), f, w, req_to_token=rt, req_idx=rows)
    st.update(api=api, ctx=ctx, rt=rt, rows=rows)


def _prepare_tree(case, seed):
    s, (kind, w, hkv) = _layer(case)
    pre, nodes = _lens(case)
    seq = [p + t for p, t in zip(pre, nodes)]
    g = _gen(seed)
    r = random.Random(seed)
    st = dict(tables=_pages(seq, s["ps"], seed, w))
    rows = st["tables"]["size"] + s["ps"]
    io = torch.float32 if s["dtype"] == "f32" else torch.bfloat16
    st["k"], st["v"] = (_pool(g, (rows, hkv, s["d"]), s["dtype"]) for _ in range(2))
    n = sum(nodes)
    st["q"] = torch.randn((n, s["hq"], s["d"]), generator=g, device="cuda").to(io)
    st["sinks"] = torch.randn(s["hq"], generator=g, device="cuda") if case["shape"] != "llama4" else None
    st["parents_h"] = [_tree_parents(r, t) for t in nodes]
    st["parents"] = torch.tensor([p for t in st["parents_h"] for p in t], dtype=torch.int32, device="cuda")
    st["pre"] = torch.tensor(pre, device="cuda")
    st["indptr"] = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), device="cuda")
    st.update(pre_h=pre, nodes_h=nodes, n=n, max_new=max(nodes), max_seq=max(seq), scale=1.0 / math.sqrt(s["d"]),
              ks=0.5 if s["dtype"] == "e4m3" else 1.0, vs=1.5 if s["dtype"] == "e4m3" else 1.0)
    if own:
        # The other pool of the program is not read by this layer.
        _context(case, st, [((kind, w, hkv), st["k"], st["v"])], seq)
        api, ctx, bs = st["api"], st["ctx"], len(pre)
        st["plan"] = None
        if kind != FULL:
            st["plan"] = torch.zeros(api.swa_plan_bytes(ctx, bs, st["max_new"]), dtype=torch.uint8, device="cuda")
            api.swa_plan(ctx, st["rt"], st["rows"], st["pre"], torch.tensor(seq, device="cuda"), st["plan"], st["max_new"])
        st["tree"] = torch.zeros(api.swa_tree_bytes(ctx, n, st["max_new"]), dtype=torch.uint8, device="cuda")
        st["ws"] = torch.zeros(api.swa_attn_tree_ws_bytes(ctx, 0, bs, n, st["max_new"], st["max_seq"]), dtype=torch.uint8, device="cuda")
        st["positions"] = torch.zeros(n, dtype=torch.int64, device="cuda")
        st["out"] = torch.zeros_like(st["q"])
    return st


def _prepare_qknorm(case, seed):
    s, (kind, w, hkv) = _layer(case)
    g = _gen(seed)
    n, d, hq = case["n"], s["d"], s["hq"]
    # the tokens are the ends of requests of at most 512 of them
    seq = [min(512, n - i) for i in range(0, n, 512)]
    st = dict(tables=_pages(seq, s["ps"], seed, w))
    rows = st["tables"]["size"] + s["ps"]
    io = torch.float32 if s["dtype"] == "f32" else torch.bfloat16
    st["k"], st["v"] = (_pool(g, (rows, hkv, d), s["dtype"]) for _ in range(2))
    # one row of the model's fused projection for each token
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda").mul_(2.0).to(io)
    st["q"], st["kn"], st["vn"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    st["wq"], st["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    max_pos = 65536
    rot = case["rot"]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    st["pos"] = torch.randint(0, max_pos, (n,), generator=g, device="cuda")
    t = st["tables"]
    st["full_loc"] = torch.cat([t["rt"][b + 1, :m] for b, m in enumerate(seq)]).to(torch.int64)
    st["swa_loc"] = t["mapping"][st["full_loc"]]
    st.update(eps=1e-6, ks=0.02 if s["dtype"] == "e4m3" else 1.0, vs=0.03 if s["dtype"] == "e4m3" else 1.0)
    if own:
        _context(case, st, [((kind, w, hkv), st["k"], st["v"])], seq)
        st["q_out"] = torch.zeros((n, hq, d), dtype=io, device="cuda")
    return st


def _layers_of(case, st):
    s = SHAPES[case["shape"]]
    return [(s["full"], st["full"][l, 0], st["full"][l, 1]) for l in range(case["full"])] + \
           [(s["win"], st["win"][l, 0], st["win"][l, 1]) for l in range(case["win"])]


def _prepare_rows(case, seed):
    """Pools of a whole model for the operators that move rows of all layers."""
    s = SHAPES[case["shape"]]
    g = _gen(seed)
    r = random.Random(seed)
    if case["op"] == "commit":
        seq = [case["prefix"] + b % 29 + case["nodes"] for b in range(case["bs"])]
    else:
        seq = [case["pool"] // 8] * 8
    st = dict(tables=_pages(seq, s["ps"], seed, s["win"][1]))
    rows = st["tables"]["size"] + s["ps"]
    for name in ("full", "win"):
        st[name] = _pool(g, (case[name], 2, rows, s[name][2], s["d"]), s["dtype"])
    if case["op"] == "commit":
        kept = _kept(case)
        m = max(case["keep"], 1)
        acc = np.zeros((case["bs"], m), np.int32)
        for b, k in enumerate(kept):
            acc[b, :k] = sorted(r.sample(range(case["nodes"]), k))
        st["pre_h"], st["acc_h"], st["kept_h"] = [q - case["nodes"] for q in seq], acc, kept
        st["pre"] = torch.tensor(st["pre_h"], device="cuda")
        st["acc"] = torch.tensor(acc, device="cuda")
        st["kept"] = torch.tensor(kept, dtype=torch.int32, device="cuda")
    else:
        slots = st["tables"]["rt"][1:, :case["pool"] // 8].reshape(-1).to(torch.int64)
        slots = slots[torch.randperm(len(slots), generator=g, device="cuda")[:2 * case["n"]]]
        st["src"], st["dst"] = slots[:case["n"]].contiguous(), slots[case["n"]:].contiguous()
    if own:
        _context(case, st, _layers_of(case, st), seq)
    return st


def prepare(case, seed):
    make = {"tree": _prepare_tree, "qknorm": _prepare_qknorm}.get(case["op"], _prepare_rows)
    st = make(case, seed)
    st["case"] = case
    return st


# ------------------------------------------------------------- plain forms ---
def _values(x, scale):
    """Stored K or V rows as float32 values."""
    return x.view(torch.float8_e4m3fn).float() * scale if x.dtype == torch.uint8 else x.float()


def _as_values(pool):
    """A pool as the values that it holds."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _plain_tree(case, st):
    s, (kind, w, hkv) = _layer(case)
    hq, d = s["hq"], s["d"]
    G = hq // hkv
    bs, T = len(st["pre_h"]), st["max_new"]
    dev = st["q"].device
    pre, indptr = st["pre"], st["indptr"]
    nodes = indptr[1:] - indptr[:-1]
    ti = torch.arange(T, device=dev)
    valid = ti < nodes[:, None]                                     # [bs, T]
    flat = (indptr[:-1, None] + ti).clamp(max=st["n"] - 1)
    parents = torch.where(valid, st["parents"][flat].long(), -1)
    # ancestors (a node is its own): the sum of the powers of the parent matrix
    step = (parents[:, :, None] == ti).float()
    anc = torch.eye(T, device=dev) + step
    reach = 1
    while reach < T:
        step = step @ step
        anc = anc + step @ anc
        reach *= 2
    anc = anc > 0                                                   # [bs, T (node), T (ancestor)]
    depth = anc.sum(-1) - 1
    pos = pre[:, None] + depth                                      # [bs, T]
    first = pos * 0 if kind == FULL else (pos - w).clamp(min=0) if kind == SLIDING else pos // w * w
    lo = first.min(1).values                                        # first column any node reads
    width = int(max(min(p, p if kind == FULL else w) for p in st["pre_h"])) + T
    col = lo[:, None] + torch.arange(width, device=dev)             # [bs, width]: column of req_to_token
    end = pre + nodes
    slots = torch.gather(st["tables"]["rt"][1:].long(), 1, col.clamp(max=st["tables"]["rt"].shape[1] - 1))
    slots = torch.where(col < end[:, None], slots, 0)
    if kind != FULL:
        slots = st["tables"]["mapping"][slots]
    j = (col - pre[:, None]).clamp(0, T - 1)                        # node of a column behind the prefix
    kpos = torch.where(col < pre[:, None], col, torch.gather(pos, 1, j))
    cached = (col < pre[:, None])[:, None, :]
    seen = torch.gather(anc, 2, j[:, None, :].expand(bs, T, width)) & (col >= pre[:, None])[:, None, :] & (col < end[:, None])[:, None, :]
    mask = (cached | seen) & (kpos[:, None, :] >= first[:, :, None]) & valid[:, :, None]
    K = _values(st["k"][slots], st["ks"]).permute(0, 2, 3, 1)       # [bs, hkv, d, width]
    Q = st["q"].float()[flat].view(bs, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(bs, hkv, T * G, d)
    S = torch.matmul(Q, K).mul_(st["scale"]).view(bs, hkv, T, G, width)
    del K
    S.masked_fill_(~mask[:, None, :, None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    if st["sinks"] is not None:
        sink = st["sinks"].view(1, hkv, 1, G, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    p = S.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    if st["sinks"] is not None:
        den = den + (sink - m).exp()
    V = _values(st["v"][slots], st["vs"]).permute(0, 2, 1, 3)       # [bs, hkv, width, d]
    o = torch.matmul(p.view(bs, hkv, T * G, width), V).view(bs, hkv, T, G, d) / den
    o = o.permute(0, 2, 1, 3, 4).reshape(bs, T, hq, d)[valid]
    return {"out": o.to(st["q"].dtype), "positions": pos[valid]}


def _norm_rotate(x, w, st, rot, interleaved):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w
    t = st["table"][st["pos"]]
    cos, sin = t[:, None, :rot // 2], t[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _stored(x, pool, scale):
    if pool.dtype == torch.uint8:
        return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(pool.dtype)


def _plain_qknorm(case, st):
    loc = st["full_loc"] if case["layer"] == "full" else st["swa_loc"]
    q = _norm_rotate(st["q"], st["wq"], st, case["rot"], case["interleaved"]).to(st["q"].dtype)
    k = _norm_rotate(st["kn"], st["wk"], st, case["rot"], case["interleaved"])
    st["k"][loc] = _stored(k, st["k"], st["ks"])
    st["v"][loc] = _stored(st["vn"], st["v"], st["vs"])
    return {"q": q, "k": _as_values(st["k"]), "v": _as_values(st["v"])}


def _move(st, src, dst):
    """Rows of all layers from full slots src to full slots dst."""
    to_swa = st["tables"]["mapping"]
    st["full"][:, :, dst] = st["full"][:, :, src]
    st["win"][:, :, to_swa[dst]] = st["win"][:, :, to_swa[src]]
    return {"full": st["full"], "win": st["win"]}


def _plain_commit(case, st):
    m = st["acc"].shape[1]
    at = torch.arange(m, device="cuda")
    cols = st["pre"][:, None] + torch.stack([st["acc"].long(), at.expand_as(st["acc"])])     # [2, bs, m]
    rt = st["tables"]["rt"][1:].long()
    src, dst = torch.gather(rt, 1, cols[0]), torch.gather(rt, 1, cols[1].clamp(max=rt.shape[1] - 1))
    # a position that keeps nothing is copied onto itself in page 0, which nobody reads
    live = at < st["kept"][:, None]
    return _move(st, torch.where(live, src, 0).flatten(), torch.where(live, dst, 0).flatten())


# --------------------------------------------------------------------- run ---
def _own_tree(st):
    api = st["api"]
    api.swa_tree_plan(st["ctx"], st["parents"], st["pre"], st["indptr"], st["n"], st["max_new"], st["tree"], st["positions"])
    api.swa_attn_tree(st["ctx"], 0, st["rt"], st["rows"], st["pre"], st["indptr"], st["n"], st["max_new"], st["max_seq"], st["plan"], st["tree"],
                      st["q"], st["sinks"], st["scale"], st["out"], st["ws"], st["ks"], st["vs"])
    return {"out": st["out"], "positions": st["positions"]}


def _own_qknorm(case, st):
    st["api"].swa_qk_norm_rope_store(st["ctx"], 0, st["q"], st["kn"], st["vn"], st["pos"], st["full_loc"], st["q_out"], swa_loc=st["swa_loc"],
                                     q_weight=st["wq"], k_weight=st["wk"], eps=st["eps"], cos_sin=st["table"], rot_dim=case["rot"],
                                     interleaved=case["interleaved"], k_scale=st["ks"], v_scale=st["vs"])
    return {"q": st["q_out"], "k": _as_values(st["k"]), "v": _as_values(st["v"])}


def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if own:
        if op == "tree":
            return _own_tree(st)
        if op == "qknorm":
            return _own_qknorm(case, st)
        if op == "commit":
            st["api"].swa_commit_tree(st["ctx"], st["rt"], st["rows"], st["pre"], st["acc"], st["kept"])
        else:
            st["api"].swa_copy_kv(st["ctx"], st["src"], st["dst"])
        return {"full": st["full"], "win": st["win"]}
    if op == "tree":
        return _plain_tree(case, st)
    if op == "qknorm":
        return _plain_qknorm(case, st)
    return _plain_commit(case, st) if op == "commit" else _move(st, st["src"], st["dst"])


# ------------------------------------------------------------------- exact ---
def _exact_tree(case, st):
    s, (kind, w, hkv) = _layer(case)
    hq, d = s["hq"], s["d"]
    out, positions = [], []
    at = 0
    rt = st["tables"]["rt"]
    for b, (p, t) in enumerate(zip(st["pre_h"], st["nodes_h"])):
        par = st["parents_h"][b]
        above = []
        for i in range(t):
            above.append([i] + (above[par[i]] if par[i] >= 0 else []))
        pos = [p + len(a) - 1 for a in above]
        low = [0 if kind == FULL else max(0, x - w) if kind == SLIDING else x - x % w for x in pos]
        c0 = min(min(low), p)
        mask = np.zeros((t, p + t - c0), bool)
        for i in range(t):
            mask[i, max(low[i] - c0, 0):p - c0] = True
            mask[i, [p - c0 + a for a in above[i] if pos[a] >= low[i]]] = True
        slots = rt[b + 1, c0:p + t].long()
        slots = slots if kind == FULL else st["tables"]["mapping"][slots]
        rows = [(x[slots].view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x[slots]).double() * sc
                for x, sc in ((st["k"], st["ks"]), (st["v"], st["vs"]))]
        m = torch.tensor(mask, device="cuda")
        o = torch.empty((t, hq, d), dtype=torch.float64, device="cuda")
        for h in range(hq):
            z = (st["q"][at:at + t, h].double() @ rows[0][:, h * hkv // hq].T) * st["scale"]
            z = torch.where(m, z, -math.inf)
            if st["sinks"] is not None:
                z = torch.cat([z, st["sinks"][h].double().expand(t, 1)], 1)
            o[:, h] = torch.softmax(z, 1)[:, :m.shape[1]] @ rows[1][:, h * hkv // hq]
        out.append(o)
        positions += pos
        at += t
    return {"out": torch.cat(out), "positions": torch.tensor(positions, device="cuda")}


def _exact_qknorm(case, st):
    rot, inter = case["rot"], case["interleaved"]

    def turned(x, w):
        x = x.double()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.double()
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        z = torch.complex(x[..., a], x[..., b])
        t = st["table"].double()[st["pos"]]
        z = z * torch.complex(t[:, i], t[:, rot // 2 + i])[:, None]
        y = x.clone()
        y[..., a], y[..., b] = z.real, z.imag
        return y

    loc = st["swa_loc"] if case["layer"] == "win" else st["full_loc"]
    pools = []
    for pool, new, sc in ((st["k"], turned(st["kn"], st["wk"]), st["ks"]), (st["v"], st["vn"].double(), st["vs"])):
        whole = _as_values(pool).double()
        if pool.dtype == torch.uint8:
            new = torch.clamp(new / sc, -E4M3_MAX, E4M3_MAX)
        whole[loc] = new
        pools.append(whole)
    return {"q": turned(st["q"], st["wq"]), "k": pools[0], "v": pools[1]}


def _exact_rows(case, st):
    """The moves one after another, in order, on the rows' values."""
    if case["op"] == "commit":
        rt = st["tables"]["rt"].cpu().numpy()
        pairs = [(rt[b + 1, p + st["acc_h"][b, i]], rt[b + 1, p + i])
                 for b, p in enumerate(st["pre_h"]) for i in range(st["kept_h"][b])]
    else:
        pairs = list(zip(st["src"].tolist(), st["dst"].tolist()))
    to_swa = st["tables"]["mapping"].cpu().numpy()
    n = st["full"].shape[2]
    got = {}
    for name, maps in (("full", np.arange(n)), ("win", to_swa)):
        origin = np.arange(n)              # whose row each row holds
        for a, b in pairs:
            origin[maps[b]] = origin[maps[a]]
        got[name] = st[name][:, :, torch.tensor(origin, device="cuda")]
    return got


def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "qknorm": _exact_qknorm}.get(case["op"], _exact_rows)(case, st)
