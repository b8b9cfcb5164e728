"""Draft-tree plan and tree attention on the GPU against the oracle: every
layer kind, head shape, type and layout, on the best kernel and on the generic
one; trees of one node, chains, bushes and stars; requests without nodes or
without cached tokens; windows shorter than the tree is deep; rows that belong
to nobody; wide scores; graphs, streams and a shared workspace; refusals and
device checks."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from hybrid_sliding_window_gb300 import api  # noqa: E402
from oracle import attention as OT  # noqa: E402
from oracle import tree as TR  # noqa: E402
from tests.harness import Pair  # noqa: E402
from tests.spec_harness import TreeStep, assert_attention, dev, grow, random_parents  # noqa: E402

MIMO = dict(Hq=64, D=128, dtype="bf16", layers=[(OT.SLIDING, 127, 8), (OT.FULL, 0, 4)])
GPTOSS = dict(Hq=64, D=64, dtype="bf16", layers=[(OT.SLIDING, 127, 8), (OT.FULL, 0, 8)])
LLAMA4 = dict(Hq=40, D=128, dtype="e4m3", layers=[(OT.CHUNKED, 192, 8), (OT.FULL, 0, 8)],
              k_scale=0.41, v_scale=1.7)
TINY = dict(Hq=4, D=64, dtype="f32", layers=[(OT.SLIDING, 15, 1), (OT.FULL, 0, 1)])


def _pair(shape, ps, prompt, nodes, **kw):
    kw = {**shape, **kw}
    need = sum(-(-(p + n) // ps) * ps + ps for p, n in zip(prompt, nodes)) + 4 * ps
    need = max(need, 1024 // ps * ps + 4 * ps)
    layers = kw.pop("layers")
    bs = len(prompt)
    return Pair(layers, ps=ps, size_full=need, size_swa=need, seed=11, perm_free=True,
                max_ctx=-(-(max(p + n for p, n in zip(prompt, nodes)) + 1) // 64) * 64,
                max_reqs=bs, max_batch=max(64, bs), **kw)


def _step(shape, ps, prompt, parents, path=-1, **kw):
    P = _pair(shape, ps, prompt, [len(p) for p in parents], **kw)
    api.swa_set_attn_path(P.ctx, path)
    rows = list(range(1, len(prompt) + 1))
    lens, _ = grow(P, rows, prompt)
    S = TreeStep(P, rows, lens, parents)
    P.check_state()
    return P, S


def _trees(seed, sizes):
    rng = np.random.default_rng(seed)
    return [random_parents(rng, n) for n in sizes]


# ------------------------------------------------------------------- plan ---
@pytest.mark.parametrize("kind,window", [(OT.CHUNKED, 1), (OT.SLIDING, 0)])
def test_request_without_nodes_where_a_token_sees_itself_only(kind, window):
    """Its plan has no position at all: lo = prefix lies past its last token."""
    P, S = _step(GPTOSS, 64, [200, 90, 128], [[-1, 0], [], []], layers=[(kind, window, 8), (OT.FULL, 0, 8)])
    for layer in range(2):
        S.check(layer)
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("sizes", [[1], [8, 0, 3], [32, 33, 31, 64], [200, 1, 77], [1024, 5]])
def test_plan_depths_positions_and_ancestors(sizes):
    P = _pair(TINY, 1, [5] * len(sizes), sizes)
    rows = list(range(1, len(sizes) + 1))
    lens, _ = grow(P, rows, [5 + b for b in range(len(sizes))])
    trees = _trees(1, sizes)
    trees[-1] = list(range(-1, sizes[-1] - 1))      # a chain
    S = TreeStep(P, rows, lens, trees, store=False)
    assert api.swa_device_check(P.ctx) == 0
    n, words = S.n, (S.max_new + 31) // 32
    raw = S.tree.cpu().numpy()
    depth = raw[:4 * n].view(np.int32)
    at = -(-4 * n // 256) * 256
    mask = raw[at:at + 4 * n * words].view(np.uint32).reshape(n, words)
    pos = S.positions.cpu().numpy()
    for b, par in enumerate(trees):
        for i, path in enumerate(TR.paths(par)):
            r = S.indptr[b] + i
            assert depth[r] == len(path) - 1 and pos[r] == S.pre[b] + len(path) - 1
            bits = [j for j in range(32 * words) if mask[r, j >> 5] >> (j & 31) & 1]
            assert bits == path


def test_plan_flags_bad_parents_and_counts():
    P = _pair(TINY, 1, [5, 9], [6, 6])
    lens, _ = grow(P, [1, 2], [5, 9])
    S = TreeStep(P, [1, 2], lens, [[-1, 0, 0, 2, 3, 3], [-1, 0, 1, 2, 3, 4]], store=False)
    assert api.swa_device_check(P.ctx) == 0
    good = S.positions.clone()
    # a parent that is the node itself, or behind it, counts as the root
    S.d["parents"].copy_(dev([-1, 0, 2, 2, 5, 3, -1, 0, -2, 2, 3, 4], torch.int32))
    S.make_plans()
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    assert S.positions.cpu().tolist() == [5, 6, 5, 6, 5, 7, 9, 10, 9, 10, 11, 12]
    # more nodes than max_new: those are left out, the next call is clean
    S.positions.fill_(-7)
    api.swa_tree_plan(P.ctx, S.d["parents"], S.d["pre"], S.d["indptr"], S.n, 4, S.tree, S.positions)
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    assert S.positions.cpu().tolist()[4:6] == [-7, -7]
    # an indptr that ends behind the buffers
    bad = dev([0, 6, 13])
    S.positions.fill_(-7)
    api.swa_tree_plan(P.ctx, S.d["parents"], S.d["pre"], bad, S.n, 16,
                      torch.zeros(api.swa_tree_bytes(P.ctx, S.n, 16), dtype=torch.uint8, device="cuda"),
                      S.positions)
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    S.d["parents"].copy_(dev([-1, 0, 0, 2, 3, 3, -1, 0, 1, 2, 3, 4], torch.int32))
    S.make_plans()
    assert api.swa_device_check(P.ctx) == 0
    assert torch.equal(S.positions, good)


# -------------------------------------------------------------- attention ---
CASES = [
    pytest.param(MIMO, 64, "per_layer", id="mimo-ps64"),
    pytest.param(MIMO, 16, "per_layer", id="mimo-ps16"),
    pytest.param(MIMO, 1, "per_layer", id="mimo-ps1"),
    pytest.param(MIMO, 48, "per_layer", id="mimo-ps48"),
    pytest.param(MIMO, 128, "per_layer", id="mimo-ps128"),
    pytest.param(GPTOSS, 8, "envelope", id="gptoss-envelope-ps8"),
    pytest.param(LLAMA4, 4, "envelope", id="llama4-envelope-ps4"),
    pytest.param(LLAMA4, 1, "per_layer", id="llama4-ps1"),
    pytest.param(GPTOSS, 16, "per_layer", id="gptoss-ps16"),
    pytest.param(GPTOSS, 32, "envelope", id="gptoss-envelope-ps32"),
    pytest.param(LLAMA4, 64, "envelope", id="llama4-envelope-ps64"),
    pytest.param(LLAMA4, 16, "per_layer", id="llama4-ps16"),
    pytest.param(TINY, 1, "per_layer", id="tiny-f32-ps1"),
]


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("shape,ps,layout", CASES)
def test_tree_attention(shape, ps, layout, path):
    prompt = [700, 333, 0, 65, 1]
    P, S = _step(shape, ps, prompt, _trees(3, [13, 1, 17, 33, 8]), path, layout=layout)
    for l in range(len(P.layers)):
        S.check(l, what=f"path {path}")
        S.check(l, sinks=False, what=f"path {path}, no sinks")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("kind,window", [(OT.SLIDING, 3), (OT.SLIDING, 0), (OT.CHUNKED, 5),
                                         (OT.CHUNKED, 1), (OT.SLIDING, 40)])
def test_windows_shorter_than_the_tree(kind, window, path):
    shape = dict(Hq=32, D=128, dtype="bf16", layers=[(kind, window, 4), (OT.FULL, 0, 4)])
    rng = np.random.default_rng(5)
    P, S = _step(shape, 16, [130, 47, 0, 12],
                 [list(range(-1, 39)), random_parents(rng, 70, 0.02), list(range(-1, 19)), [-1] * 9], path)
    for l in range(2):
        S.check(l, what=f"window {window}")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("Hq,hkv,D", [(8, 8, 128), (24, 8, 128), (40, 8, 64), (16, 1, 128),
                                      (12, 4, 64), (8, 4, 32)])
def test_group_sizes(Hq, hkv, D, path):
    shape = dict(Hq=Hq, D=D, dtype="bf16", layers=[(OT.SLIDING, 63, hkv), (OT.FULL, 0, hkv)])
    P, S = _step(shape, 32, [200, 31, 150], _trees(7, [9, 140, 26]), path)
    for l in range(2):
        S.check(l, what=f"Hq {Hq} hkv {hkv}")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, GPTOSS, LLAMA4], ids=["mimo", "gptoss", "llama4"])
def test_many_requests_some_without_nodes(shape):
    rng = np.random.default_rng(9)
    n = 70
    prompt = rng.integers(0, 300, n)
    sizes = rng.integers(0, 21, n)
    sizes[[0, 17, 33, 69]] = 0
    P, S = _step(shape, 16, prompt.tolist(), _trees(10, sizes))
    for l in range(2):
        S.check(l, requests=[1, 2, 16, 18, 31, 32, 34, 50, 63, 64, 68], what="70 requests")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, GPTOSS, LLAMA4], ids=["mimo", "gptoss", "llama4"])
@pytest.mark.parametrize("nodes", [1, 8, 64, 300])
def test_one_long_request(shape, nodes):
    """Many key tiles of one request: its keys are split over the GPU and merged."""
    P, S = _step(shape, 64, [4500], _trees(11, [nodes]))
    for l in range(2):
        g, q = S.attend(l)
        some = sorted(set([0, nodes // 3, nodes - 1]))
        slots = P.ort[1]
        ref, mag = [], []
        for i in some:
            cols = TR.node_columns(P.layers[l][0], P.layers[l][1], 4500, S.parents[0], i)
            sl = [int(slots[c]) for c in cols]
            sl = sl if P.layers[l][0] == OT.FULL else [P.oa.mapping[s] for s in sl]
            K, V = P.op.read(l, sl, P.k_scale, P.v_scale)
            ref.append(OT.attend_heads(q[i], K, V, P.sinks[l], P.scale))
            mag.append(OT.attend_heads(q[i], K, np.abs(V), P.sinks[l], P.scale))
        assert_attention(g[some], np.stack(ref), np.stack(mag), P.dtype, f"{nodes} nodes layer {l}")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, LLAMA4], ids=["mimo", "llama4"])
@pytest.mark.parametrize("ps", [1, 20])
def test_gathered_pages(shape, ps):
    """Pages that are gathered key by key: many tiles, items in pairs, blocks of
    several Q tiles, rows of nobody and an evicted page."""
    P, S = _step(shape, ps, [1500, 130, 40, 1], _trees(21, [40, 5, 21, 1]))
    for l in range(2):
        S.check(l, what=f"ps {ps}")
    assert api.swa_last_attn_path(P.ctx) == 3
    assert api.swa_device_check(P.ctx) == 0
    page = int(P.ort[1, 1495]) // ps * ps
    keep = P.ctx.mapping()[page:page + ps].clone()
    P.ctx.mapping()[page:page + ps] = 0
    S.make_plans()
    S.attend(0)
    assert api.swa_device_check(P.ctx) & api.SWA_DEVERR_WINDOW_EVICTED
    P.ctx.mapping()[page:page + ps] = keep


@pytest.mark.parametrize("path", [-1, 0])
def test_rings(path):
    P, S = _step(MIMO, 16, [200, 37, 130], _trees(12, [30, 17, 64]), path, ring_size=400)
    for l in range(2):
        S.check(l, what="ring")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("shape", [MIMO, LLAMA4], ids=["mimo", "llama4"])
def test_wide_scores(shape, path):
    """Scores that climb by hundreds along the keys (each key tile beats the one
    before by more than any fixed reference holds) and sinks from -200 to 200.
    The scores themselves then carry rounding: |score| up to ~1000, 128 products
    in f32, so a weight may be off by 128 x 2^-24 x 1000 x 1.5 ~ 2^-6.5."""
    P = _pair(shape, 64, [900, 420], [14, 9])
    api.swa_set_attn_path(P.ctx, path)
    P.q_gain = 16.0
    P.k_gain = lambda t: 1 + (t % 512) / 16
    for l in range(2):
        P.set_sinks(l, np.linspace(-200, 200, P.Hq))
    lens, _ = grow(P, [1, 2], [900, 420])
    S = TreeStep(P, [1, 2], lens, _trees(13, [14, 9]))
    for l in range(2):
        at, ref, mag = S.oracle(l, S.queries(l))
        tol = 2 * (2.0 ** -8 + 2.0 ** -6.5) * mag + 2.0 ** -8 * np.abs(ref) + 1e-6
        for bound in (S.max_seq, 8192):          # whole items; split and merged
            S.max_seq = bound
            g, _ = S.attend(l)
            assert np.isfinite(g).all() and (np.abs(g[at] - ref) <= tol).all(), f"layer {l}"
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, GPTOSS, LLAMA4], ids=["mimo", "gptoss", "llama4"])
def test_long_windows(shape):
    """Windows of more keys than a work item keeps whole: split and merged like
    full layers, with a first column inside a page, and nodes on both sides of a
    chunk's border."""
    hkv = shape["layers"][1][2]
    layers = [(OT.SLIDING, 2500, hkv), (OT.CHUNKED, 3000, hkv), (OT.SLIDING, 600, hkv)]
    rng = np.random.default_rng(18)
    parents = [random_parents(rng, 7), list(range(-1, 14)), random_parents(rng, 5)]
    P, S = _step(shape, 16, [4483, 2990, 20], parents, layers=layers)
    for l in range(3):
        S.check(l, what="long window")
    assert api.swa_device_check(P.ctx) == 0


def test_output_alignment():
    """An output that is 16-byte but not 32-byte aligned gets the same bits."""
    for shape, prompt in ((MIMO, [700, 65]), (GPTOSS, [700, 65]), (LLAMA4, [100, 20])):
        P, S = _step(shape, 64, prompt, _trees(19, [9, 12]))
        for l in range(2):
            q = P.to_dev(S.queries(l))
            out = torch.empty_like(q)
            S.run(l, q, out, S.workspace(l))
            buf = torch.full((q.numel() + 16,), 3.0, dtype=q.dtype, device="cuda")
            off = buf[8:8 + q.numel()].view(q.shape)
            assert off.data_ptr() % 32 == 16
            S.run(l, q, off, S.workspace(l))
            assert torch.equal(off, out) and (buf[:8] == 3).all() and (buf[8 + q.numel():] == 3).all()


def test_chain_equals_extend():
    """A chain is the causal chunk that swa_attn_extend attends."""
    P, S = _step(MIMO, 64, [700, 333], [list(range(-1, 39)), list(range(-1, 6))])
    for l in range(2):
        g, q = S.attend(l)
        qd = P.to_dev(q)
        out = torch.empty_like(qd)
        ws = torch.zeros(api.swa_attn_extend_ws_bytes(P.ctx, l, S.n, S.max_seq), dtype=torch.uint8,
                         device="cuda")
        api.swa_attn_extend(P.ctx, l, P.rt, S.d["rows"], S.d["pre"], S.d["seq"], S.d["indptr"], S.n,
                            S.max_new, S.max_seq, S.plan, qd, P.sinks_d[l], P.scale, out, ws)
        at, _, mag = S.oracle(l, q)
        # each within its own bound of the same sum
        assert_attention(g, out.float().cpu().numpy(), 2 * mag, "bf16", f"layer {l}")


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("shape", [MIMO, LLAMA4, TINY], ids=["mimo", "llama4", "tiny"])
def test_rows_of_nobody(shape, path):
    """Query rows behind the last request's nodes stay as they were (positions
    too), whatever they and their parents hold."""
    ps = 1 if shape is TINY else 16
    P = _pair(shape, ps, [90, 40], [9, 20])
    api.swa_set_attn_path(P.ctx, path)
    lens, _ = grow(P, [1, 2], [90, 40])
    S = TreeStep(P, [1, 2], lens, _trees(14, [9, 20]), max_new=24)
    for l in range(2):
        want, q = S.attend(l)
        n, pad = S.n, 5
        qd = torch.cat([P.to_dev(q), torch.full((pad, P.Hq, P.D), float("nan"), dtype=P.to_dev(q).dtype,
                                                device="cuda")])
        out = torch.full_like(qd, 7.0)
        tree = torch.full((api.swa_tree_bytes(P.ctx, n + pad, 24),), 0xA5, dtype=torch.uint8, device="cuda")
        parents = torch.cat([S.d["parents"], dev([99] * pad, torch.int32)])
        pos = torch.full((n + pad,), -3, dtype=torch.int64, device="cuda")
        api.swa_tree_plan(P.ctx, parents, S.d["pre"], S.d["indptr"], n + pad, 24, tree, pos)
        ws = torch.zeros(api.swa_attn_tree_ws_bytes(P.ctx, l, 2, n + pad, 24, S.max_seq),
                         dtype=torch.uint8, device="cuda")
        api.swa_attn_tree(P.ctx, l, P.rt, S.d["rows"], S.d["pre"], S.d["indptr"], n + pad, 24, S.max_seq,
                          S.plan, tree, qd, P.sinks_d[l], P.scale, out, ws, P.k_scale, P.v_scale)
        assert (out[n:] == 7).all() and (pos[n:] == -3).all()
        np.testing.assert_array_equal(out[:n].float().cpu().numpy(), want)
    assert api.swa_device_check(P.ctx) == 0


def test_repeats_streams_and_graphs():
    """One workspace for layers of other shapes, repeated calls, another stream
    and replays of a captured step: bit for bit the same."""
    P, S = _step(MIMO, 64, [2500, 333, 0, 65], _trees(15, [13, 1, 17, 33]))
    n_ws = max(S.workspace(l).numel() for l in range(2))
    ws = torch.zeros(n_ws, dtype=torch.uint8, device="cuda")
    qs = [P.to_dev(S.queries(l)) for l in range(2)]
    want = [torch.empty_like(q) for q in qs]
    for l in range(2):
        S.run(l, qs[l], want[l], S.workspace(l))
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for q in qs]
    for _ in range(3):
        for l in (1, 0):
            S.run(l, qs[l], outs[l], ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    S.make_plans(stream=side)
    for l in range(2):
        S.run(l, qs[l], outs[l], ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.make_plans()
        for l in range(2):
            S.run(l, qs[l], outs[l], ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # the replay reads the tree and lengths that are there then
    S.d["parents"].copy_(dev([-1] * S.n, torch.int32))
    g.replay()
    torch.cuda.synchronize()
    S.parents = [[-1] * k for k in S.nodes]
    for l in range(2):
        q = S.queries(l)
        at, ref, mag = S.oracle(l, q)
        assert_attention(outs[l].float().cpu().numpy()[at], ref, mag, "bf16", "stars")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, TINY], ids=["mimo", "tiny"])
def test_workspace_shared_with_decode_and_across_kernels(shape):
    """One workspace, zeroed once, under tree attention on either kernel and
    decode attention in turn: bits as with fresh ones."""
    ps = 1 if shape is TINY else 64
    P, S = _step(shape, ps, [2500, 333], _trees(20, [13, 7]))
    d_seq, rows = S.d["seq"], S.d["rows"]
    dplan = torch.zeros(api.swa_plan_bytes(P.ctx, 2, 1), dtype=torch.uint8, device="cuda")
    api.swa_plan(P.ctx, P.rt, rows, None, d_seq, dplan, 1)
    qs = [P.to_dev(S.queries(l)) for l in range(2)]
    size = 0
    for path in (-1, 0):
        api.swa_set_attn_path(P.ctx, path)
        size = max([size] + [S.workspace(l).numel() for l in range(2)]
                   + [api.swa_attn_decode_ws_bytes(P.ctx, l, 2, S.max_seq) for l in range(2)])

    def run(ws):
        got = []
        for path in (-1, 0, -1):
            api.swa_set_attn_path(P.ctx, path)
            for l in range(2):
                out, dec = torch.empty_like(qs[l]), torch.empty_like(qs[l][:2])
                S.run(l, qs[l], out, ws())
                api.swa_attn_decode(P.ctx, l, P.rt, rows, d_seq, S.max_seq, dplan, qs[l][:2].contiguous(),
                                    P.sinks_d[l], P.scale, dec, ws())
                got += [out, dec]
        return got

    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = run(lambda: torch.zeros(size, dtype=torch.uint8, device="cuda"))
    for a, b in zip(run(lambda: shared), want):
        assert torch.equal(a, b)
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [TINY, MIMO, dict(LLAMA4, D=64)], ids=["tiny", "mimo", "e4m3-d64"])
@pytest.mark.parametrize("big,small", [(260, 130), (1000, 500)])
def test_workspace_reused_by_calls_of_other_sizes(shape, big, small):
    """One workspace, zeroed once, under generic-kernel tree and extend calls
    whose rows - more than max_batch of them, or more than the tickets that every
    call keeps clear - rise and fall, with decode calls between: outputs as with
    fresh ones."""
    ps = 1 if shape is TINY else 64
    P, S = _step(shape, ps, [900, 333], _trees(23, [big, small]), 0)
    rows, pre, seq = S.d["rows"], S.d["pre"], S.d["seq"]
    assert P.ctx.cfg.max_batch == 64
    dplan = torch.zeros(api.swa_plan_bytes(P.ctx, 2, 1), dtype=torch.uint8, device="cuda")
    api.swa_plan(P.ctx, P.rt, rows, None, seq, dplan, 1)
    qs = [P.to_dev(S.queries(l)) for l in range(2)]
    size = max([api.swa_attn_extend_ws_bytes(P.ctx, l, S.n, S.max_seq) for l in range(2)]
               + [S.workspace(l).numel() for l in range(2)])

    def tree_call(l, sizes, ws, chain):
        """The first nodes of each tree (with the parents' smaller indices, trees again)."""
        at = np.concatenate([np.arange(a, a + k) for a, k in zip(S.indptr, sizes)])
        n, indptr = int(sum(sizes)), dev(np.concatenate([[0], np.cumsum(sizes)]))
        q = qs[l][dev(at)].contiguous()
        out = torch.full_like(q, 7.0)
        end = pre + dev(sizes)
        plan = torch.zeros(api.swa_plan_bytes(P.ctx, 2, big), dtype=torch.uint8, device="cuda")
        api.swa_plan(P.ctx, P.rt, rows, pre, end, plan, big)
        if chain:
            api.swa_attn_extend(P.ctx, l, P.rt, rows, pre, end, indptr, n, big, S.max_seq, plan, q, P.sinks_d[l],
                                P.scale, out, ws, P.k_scale, P.v_scale)
            return out
        tree = torch.zeros(api.swa_tree_bytes(P.ctx, n, big), dtype=torch.uint8, device="cuda")
        api.swa_tree_plan(P.ctx, S.d["parents"][dev(at)].contiguous(), pre, indptr, n, big, tree)
        api.swa_attn_tree(P.ctx, l, P.rt, rows, pre, indptr, n, big, S.max_seq, plan, tree, q, P.sinks_d[l],
                          P.scale, out, ws, P.k_scale, P.v_scale)
        return out

    def decode_call(l, ws):
        out = torch.full_like(qs[l][:2], 7.0)
        api.swa_attn_decode(P.ctx, l, P.rt, rows, seq, S.max_seq, dplan, qs[l][:2].contiguous(), P.sinks_d[l],
                            P.scale, out, ws, P.k_scale, P.v_scale)
        return out

    def run(ws):
        got = []
        for sizes in ([big // 4, 9], [big, small], [30, 40], [big - 60, small], [3, 2], [big, 1]):
            for l in (1, 0):
                for chain in (False, True):
                    got.append(tree_call(l, sizes, ws(), chain))
                    got.append(decode_call(l, ws()))
        return got

    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = run(lambda: torch.zeros(size, dtype=torch.uint8, device="cuda"))
    for i, (a, b) in enumerate(zip(run(lambda: shared), want)):
        assert torch.equal(a, b), f"call {i}"
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape", [MIMO, LLAMA4], ids=["mimo", "llama4"])
def test_one_tile_items_behind_pairs_and_wide_items(shape):
    """CTAs whose last item has one key tile, behind a pair of items (whole items)
    or an item of two Q tiles (stretches): many launches, always the same bits."""
    n = 57                                  # three items for each of 19 CTAs of a KV head
    sizes = [12 if b % 3 == 0 else 3 for b in range(n)]
    P, S = _step(shape, 64, [20 + b for b in range(n)], _trees(25, sizes))
    for l in range(2):
        S.check(l, requests=[0, 1, 2, 27, 55, 56], what="one tile")
        q = P.to_dev(S.queries(l))
        for bound in (S.max_seq, 8192):
            S.max_seq = bound
            ws, want = S.workspace(l), torch.empty_like(q)
            S.run(l, q, want, ws)
            out = torch.empty_like(q)
            for _ in range(300):
                S.run(l, q, out, ws)
            assert torch.equal(out, want)
        S.max_seq = int(S.seq.max())
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape,nodes", [(MIMO, 65), (MIMO, 300), (LLAMA4, 130)], ids=["mimo-65", "mimo-300", "llama4-130"])
def test_captured_step_of_wide_trees_with_changing_parents(shape, nodes):
    """Plan and attention captured back to back, trees of more nodes than a
    register holds: every replay attends the parents that are there then."""
    rng = np.random.default_rng(26)
    P, S = _step(shape, 64, [150, 60], [random_parents(rng, nodes), random_parents(rng, 20)])
    qs = [P.to_dev(S.queries(l)) for l in range(2)]
    outs, wss = [torch.empty_like(q) for q in qs], [S.workspace(l) for l in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for l in range(2):
            S.make_plans()
            S.run(l, qs[l], outs[l], wss[l])
    for roots in (0.1, 1.0, 0.5):
        S.parents = [random_parents(rng, nodes, roots), random_parents(rng, 20, roots)]
        S.d["parents"].copy_(dev([p for t in S.parents for p in t], torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for l in range(2):
            at, ref, mag = S.oracle(l, S.queries(l))
            assert_attention(outs[l].float().cpu().numpy()[at], ref, mag, P.dtype, f"roots {roots} layer {l}")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("path", [-1, 0])
@pytest.mark.parametrize("shape", [MIMO, GPTOSS, LLAMA4], ids=["mimo", "gptoss", "llama4"])
def test_not_a_number_stays_in_its_row(shape, path):
    """A query that is not a number gives an output that is not a number, on
    items whose keys one group of rows takes, that two share, and that are split
    over the GPU; every other row keeps its bits."""
    P, S = _step(shape, 64, [300, 700, 20], _trees(24, [9, 20, 1]), path)
    for l in range(2):
        q = P.to_dev(S.queries(l))
        hurt = q.clone()
        at = [0, 4, 9 + 17, 9 + 20]
        for i, r in enumerate(at):
            hurt[r, 3 * i, 5] = float("nan")
        for bound in (S.max_seq, 8192):
            S.max_seq = bound
            out, bad = torch.empty_like(q), torch.empty_like(q)
            S.run(l, q, out, S.workspace(l))
            S.run(l, hurt, bad, S.workspace(l))
            is_bad = torch.isnan(bad)
            for i, r in enumerate(at):
                assert is_bad[r, 3 * i].all(), f"layer {l} row {r}"
                is_bad[r, 3 * i] = False
                out[r, 3 * i] = bad[r, 3 * i] = 0
            assert not is_bad.any() and torch.equal(out, bad)
        S.max_seq = int(S.seq.max())
    assert api.swa_device_check(P.ctx) == 0


# ---------------------------------------------------------------- refusals ---
def test_refusals_leave_the_context_usable():
    P, S = _step(MIMO, 64, [100, 30], _trees(16, [5, 9]))
    q = P.to_dev(S.queries(1))
    out = torch.empty_like(q)
    ws = S.workspace(1)
    L, h = api.lib(), P.ctx.handle

    def plan(**kw):
        a = dict(bs=2, parents=S.d["parents"].data_ptr(), pre=S.d["pre"].data_ptr(),
                 indptr=S.d["indptr"].data_ptr(), n=S.n, max_new=9, pos=None, tree=S.tree.data_ptr(),
                 nb=S.tree.numel())
        a.update(kw)
        return L.swa_tree_plan(h, *a.values(), None)

    def attn(**kw):
        a = dict(layer=1, bs=2, rt=P.rt.data_ptr(), stride=P.rt.shape[1], rows=S.d["rows"].data_ptr(),
                 pre=S.d["pre"].data_ptr(), indptr=S.d["indptr"].data_ptr(), n=S.n, max_new=9,
                 msl=S.max_seq, plan=S.plan.data_ptr(), tree=S.tree.data_ptr(), q=q.data_ptr(),
                 sinks=None, scale=0.1, ks=1.0, vs=1.0, out=out.data_ptr(), ws=ws.data_ptr(),
                 nb=ws.numel())
        a.update(kw)
        return L.swa_attn_tree(h, *a.values(), None)

    bad = api.SWA_ERR_INVALID
    for kw in (dict(bs=-1), dict(bs=65), dict(n=-1), dict(max_new=0), dict(max_new=1025),
               dict(parents=None), dict(pre=None), dict(indptr=None), dict(tree=None), dict(nb=8),
               dict(tree=S.tree.data_ptr() + 4)):
        assert plan(**kw) == bad, kw
    for kw in (dict(layer=2), dict(layer=-1), dict(bs=-1), dict(bs=65), dict(n=-1), dict(max_new=0),
               dict(max_new=1025), dict(msl=0), dict(rt=None), dict(rows=None), dict(pre=None),
               dict(indptr=None), dict(tree=None), dict(q=None), dict(out=None), dict(ws=None),
               dict(nb=16), dict(q=q.data_ptr() + 2), dict(out=out.data_ptr() + 8),
               dict(layer=0, plan=None), dict(tree=S.tree.data_ptr() + 8), dict(layer=0, plan=S.plan.data_ptr() + 4),
               dict(ws=ws.data_ptr() + 8)):
        assert attn(**kw) == bad, kw
    assert api.swa_tree_bytes(P.ctx, 4, 1025) == 0 and api.swa_tree_bytes(P.ctx, -1, 4) == 0
    assert api.swa_attn_tree_ws_bytes(P.ctx, 5, 2, 4, 4, 100) == 0
    assert plan(bs=0) == 0 and plan(n=0) == 0 and attn(bs=0) == 0 and attn(n=0) == 0
    assert plan() == 0 and attn() == 0
    torch.cuda.synchronize()
    assert api.swa_device_check(P.ctx) == 0
    S.check(1, what="after refusals")


@pytest.mark.parametrize("shape", [MIMO, LLAMA4], ids=["mimo", "llama4"])
def test_scales_that_a_masked_score_does_not_survive(shape):
    """-inf times a scale that is not positive is no -inf: refused where the
    kernel scales after masking, served by the generic kernel."""
    P, S = _step(shape, 64, [100, 30], _trees(27, [5, 9]))
    q = P.to_dev(S.queries(1))
    out = torch.full_like(q, 7.0)
    ws = S.workspace(1)
    good = P.scale
    for bad in (0.0, -good, float("nan"), float("inf")):
        P.scale = bad
        with pytest.raises(api.SwaError) as e:
            S.run(1, q, out, ws)
        assert e.value.status == api.SWA_ERR_INVALID
    assert (out == 7).all()
    api.swa_set_attn_path(P.ctx, 0)
    for P.scale in (0.0, -good):
        S.check(1, what=f"scale {P.scale}")
    P.scale = good
    api.swa_set_attn_path(P.ctx, -1)
    S.check(1)
    assert api.swa_device_check(P.ctx) == 0


def test_device_checks():
    """Columns past the req_to_token row, and an evicted key in the window."""
    P, S = _step(MIMO, 64, [700, 30], _trees(17, [5, 9]))
    q = P.to_dev(S.queries(1))
    out = torch.empty_like(q)
    ws = S.workspace(1)
    S.run(1, q, out, ws)
    assert api.swa_device_check(P.ctx) == 0
    # a prefix that puts the nodes past the row
    good = S.d["pre"].clone()
    S.d["pre"][1] = P.rt.shape[1] - 3
    S.run(1, q, out, ws)
    assert api.swa_device_check(P.ctx) & api.SWA_DEVERR_RANGE
    S.d["pre"].copy_(good)
    S.run(1, q, out, ws)
    assert api.swa_device_check(P.ctx) == 0
    # the SWA slot of a page inside the window released behind the plan's back
    slot = int(P.ort[1, 690])
    page = slot // 64 * 64
    keep = P.ctx.mapping()[page:page + 64].clone()
    P.ctx.mapping()[page:page + 64] = 0
    S.make_plans()
    assert api.swa_device_check(P.ctx) & api.SWA_DEVERR_WINDOW_EVICTED
    P.ctx.mapping()[page:page + 64] = keep
    S.make_plans()
    for l in range(2):
        S.check(l, what="after device checks")
    assert api.swa_device_check(P.ctx) == 0


@pytest.mark.parametrize("shape,ps,kernel", [(MIMO, 64, 3), (MIMO, 16, 3), (MIMO, 1, 3), (GPTOSS, 32, 3),
                                             (LLAMA4, 64, 3), (TINY, 1, 0)],
                         ids=["mimo-ps64", "mimo-ps16", "mimo-ps1", "gptoss", "llama4", "tiny"])
def test_kernel_taken(shape, ps, kernel):
    """The tensor-core kernel serves bf16 and E4M3 pools; -1 and 0 select."""
    P, S = _step(shape, ps, [40], [[-1, 0, 0]])
    S.attend(1)
    assert api.swa_last_attn_path(P.ctx) == kernel
    api.swa_set_attn_path(P.ctx, 0)
    S.attend(1)
    assert api.swa_last_attn_path(P.ctx) == 0
