"""Row moves of all layers: the commit of a verified tree and copies between
slots, bit for bit against the oracle's pools (types, layouts, rings, rows of
odd sizes, windows that released a source); padding, bad entries, refusals,
graphs; and a whole speculative step - allocate, plan, norm + rotate + store,
attend, commit, free, decode - run as a program would."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from hybrid_sliding_window_gb300 import api  # noqa: E402
from oracle import attention as OT  # noqa: E402
from oracle import tree as TR  # noqa: E402
from tests.harness import TOL, Pair, assert_close  # noqa: E402
from tests.spec_harness import TreeStep, assert_attention, dev, grow, random_parents  # noqa: E402

SHAPES = {
    "mimo": dict(Hq=64, D=128, dtype="bf16", layers=[(OT.SLIDING, 127, 8), (OT.FULL, 0, 4)] * 2, ps=64),
    "envelope": dict(Hq=40, D=128, dtype="e4m3", layers=[(OT.CHUNKED, 192, 8), (OT.FULL, 0, 8)], ps=16,
                     layout="envelope"),
    "tiny": dict(Hq=4, D=64, dtype="f32", layers=[(OT.SLIDING, 15, 1), (OT.FULL, 0, 1)], ps=1),
    "thin": dict(Hq=3, D=32, dtype="e4m3", layers=[(OT.FULL, 0, 3), (OT.SLIDING, 40, 1)], ps=4),
    "ring": dict(Hq=16, D=64, dtype="bf16", layers=[(OT.SLIDING, 63, 2), (OT.FULL, 0, 2)], ps=16, ring_size=300),
    "deep": dict(Hq=2, D=32, dtype="bf16", layers=[(OT.SLIDING, 15, 1), (OT.FULL, 0, 2)] * 37, ps=8),
}


def _pair(name, **kw):
    s = dict(SHAPES[name], **kw)
    ps, layers = s.pop("ps"), s.pop("layers")
    if s["D"] == 32 and s["dtype"] == "e4m3":
        s["Hq"] = 3
    return Pair(layers, ps=ps, size_full=ps * (2048 // ps + 8), size_swa=ps * (2048 // ps + 8), seed=21,
                perm_free=True, max_ctx=1024, max_reqs=4, **s)


@pytest.mark.parametrize("name", list(SHAPES))
def test_commit(name):
    P = _pair(name)
    rows, pre = [1, 2, 3, 4], np.array([100, 37, 0, 65])
    grow(P, rows, pre)
    nodes = 70
    P.extend(rows, pre, pre + nodes)
    rng = np.random.default_rng(3)
    acc = np.full((4, 48), -99, np.int32)        # entries behind the count are not read
    lists = [sorted(rng.choice(nodes, 40, replace=False).tolist()), list(range(9)), [], [69]]
    for b, a in enumerate(lists):
        acc[b, :len(a)] = a
        TR.commit(P.op, P.oa.mapping, P.ort[rows[b]], int(pre[b]), a)
    api.swa_commit_tree(P.ctx, P.rt, dev(rows), dev(pre), dev(acc, torch.int32),
                        dev([len(a) for a in lists], torch.int32))
    P.check_state()


@pytest.mark.parametrize("name", list(SHAPES))
def test_copy(name):
    P = _pair(name)
    rows, lens = [1, 2, 3], np.array([400, 150, 33])
    grow(P, rows, lens, step=200)                # what lies behind the window is released
    rng = np.random.default_rng(4)
    src = np.concatenate([P.ort[1, 200:400], P.ort[2, 100:150]])
    live = np.array([P.oa.mapping[s] > 0 for s in src])
    assert name == "envelope" or not live.all()
    # destinations whose SWA slots live
    dst_all = [s for s in np.concatenate([P.ort[3, :33], P.ort[2, 149:150], P.ort[1, 399:400]])
               if P.oa.mapping[s] > 0 and s not in src]
    m = len(dst_all)
    src = rng.permutation(src)[:m]
    dst = np.array(dst_all)
    TR.move_rows(P.op, P.oa.mapping, zip(src, dst))
    s, d = (np.concatenate([x, [-1, 5, -1]]) for x in (src, dst))
    d[-2] = -1
    api.swa_copy_kv(P.ctx, dev(s), dev(d))
    P.check_state()


def test_long_copy_list():
    """More entries than one launch takes, mostly padding; rows move at both ends."""
    P = _pair("tiny")
    grow(P, [1, 2], np.array([20, 20]))
    n, src, dst = (1 << 24) + 9, P.ort[1, 15:20], P.ort[2, 15:20]
    TR.move_rows(P.op, P.oa.mapping, zip(src, dst))
    lists = torch.full((2, n), -1, dtype=torch.int64, device="cuda")
    at = torch.tensor([0, 9, (1 << 24) - 1, 1 << 24, n - 1], device="cuda")
    lists[0, at], lists[1, at] = dev(src), dev(dst)
    api.swa_copy_kv(P.ctx, lists[0], lists[1])
    P.check_state()


def test_long_commit_in_batches():
    """A commit of more rows than a warp looks up at once, every one moving."""
    P = _pair("mimo", layers=[(OT.FULL, 0, 4), (OT.SLIDING, 300, 8)])
    pre, nodes = 50, 400
    grow(P, [1], [pre])
    P.extend([1], [pre], [pre + nodes])
    acc = list(range(3, 400, 3))
    TR.commit(P.op, P.oa.mapping, P.ort[1], pre, acc)
    api.swa_commit_tree(P.ctx, P.rt, dev([1]), dev([pre]), dev([acc], torch.int32), dev([len(acc)], torch.int32))
    P.check_state()


def test_device_checks():
    P = _pair("mimo")
    pre = np.array([40, 30])
    grow(P, [1, 2], pre)
    P.extend([1, 2], pre, pre + 20)
    lists = [[0, 5, 5, 9], [2, 4, 7, 3]]         # not ascending from entry 2 (3) on
    for b, k in ((0, 2), (1, 3)):
        TR.commit(P.op, P.oa.mapping, P.ort[b + 1], int(pre[b]), lists[b][:k])
    args = (P.ctx, P.rt, dev([1, 2]), dev(pre))
    api.swa_commit_tree(*args, dev(lists, torch.int32), dev([4, 4], torch.int32))
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    P.check_state()
    for acc, n in (([[1, 2], [1, 2]], [3, -1]), ([[-2, 1], [1024, 1]], [1, 1]), ([[1000, 1], [2000, 1]], [1, 1])):
        api.swa_commit_tree(*args, dev(acc, torch.int32), dev(n, torch.int32))
        assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
        P.check_state()
    n = P.ctx.cfg.size_full + P.ps
    a, b = int(P.ort[1, 45]), int(P.ort[2, 31])
    api.swa_copy_kv(P.ctx, dev([a, n, -2]), dev([n, b, b]))
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    P.check_state()
    # a destination without an SWA slot
    P.ctx.mapping()[b] = 0
    api.swa_copy_kv(P.ctx, dev([a]), dev([b]))
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_WINDOW_EVICTED


@pytest.mark.parametrize("name", ["mimo", "envelope", "ring"])
def test_commit_of_a_node_without_its_swa_slot(name):
    """An accepted node whose SWA slot is missing (a table that is broken: the
    nodes of a step have both slots) is flagged; its row moves on full layers
    only, and the other nodes' on every layer."""
    P = _pair(name)
    pre = np.array([40, 30])
    grow(P, [1, 2], pre)
    P.extend([1, 2], pre, pre + 20)
    lost = int(P.ort[1, 40 + 6])
    P.oa.mapping[lost] = 0
    P.ctx.mapping()[lost] = 0
    acc = [[2, 6, 9], [5, 7, 8]]
    for b in range(2):
        TR.commit(P.op, P.oa.mapping, P.ort[b + 1], int(pre[b]), acc[b])
    api.swa_commit_tree(P.ctx, P.rt, dev([1, 2]), dev(pre), dev(acc, torch.int32), dev([3, 3], torch.int32))
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_WINDOW_EVICTED
    P.check_state()
    # a copy takes such a source on full layers without a flag
    src, dst = [lost], [int(P.ort[2, 31])]
    TR.move_rows(P.op, P.oa.mapping, zip(src, dst))
    api.swa_copy_kv(P.ctx, dev(src), dev(dst))
    assert api.swa_device_check(P.ctx) == 0
    P.check_state()


def test_refusals():
    P = _pair("mimo")
    L, h = api.lib(), P.ctx.handle
    x, i32 = dev([1, 2]), dev([[1], [2]], torch.int32)
    bad = api.SWA_ERR_INVALID

    def commit(**kw):
        a = dict(bs=2, rt=P.rt.data_ptr(), stride=P.rt.shape[1], rows=x.data_ptr(), pre=x.data_ptr(),
                 acc=i32.data_ptr(), m=1, n=i32.data_ptr())
        a.update(kw)
        return L.swa_commit_tree(h, *a.values(), None)

    for kw in (dict(bs=-1), dict(bs=65), dict(rt=None), dict(stride=0), dict(rows=None), dict(pre=None), dict(acc=None),
               dict(n=None), dict(m=-1), dict(m=1025)):
        assert commit(**kw) == bad, kw
    assert commit(bs=0) == 0 and commit(m=0) == 0
    p = x.data_ptr()
    assert L.swa_copy_kv(h, None, p, 2, None) == bad and L.swa_copy_kv(h, p, None, 2, None) == bad
    assert L.swa_copy_kv(h, p, p, -1, None) == bad and L.swa_copy_kv(h, None, None, 0, None) == 0
    assert api.swa_device_check(P.ctx) == 0


def test_captured_commit_reads_what_is_there_at_replay():
    P = _pair("mimo")
    pre = np.array([40, 30])
    grow(P, [1, 2], pre)
    P.extend([1, 2], pre, pre + 20)
    acc, n = dev([[0, 1, 2], [0, 1, 2]], torch.int32), dev([3, 3], torch.int32)
    rows, pd = dev([1, 2]), dev(pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        api.swa_commit_tree(P.ctx, P.rt, rows, pd, acc, n, stream=side)
    for lists in ([[1, 4, 6], [2]], [[0, 2], [5, 6, 7]]):
        a = np.zeros((2, 3), np.int32)
        for b, x in enumerate(lists):
            a[b, :len(x)] = x
            TR.commit(P.op, P.oa.mapping, P.ort[b + 1], int(pre[b]), x)
        acc.copy_(dev(a, torch.int32))
        n.copy_(dev([len(x) for x in lists], torch.int32))
        g.replay()
        P.check_state()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_speculative_steps_end_to_end(dtype):
    """Three steps: draft slots allocated, the tree planned, projections
    normalised, rotated at the tree's positions and stored, tree attention,
    the accepted path committed, the rest freed; then a decode step reads the
    committed rows."""
    ps = 16
    P = Pair([(OT.SLIDING, 60, 2), (OT.FULL, 0, 2)], Hq=16, D=64, dtype=dtype, ps=ps, size_full=ps * 96,
             size_swa=ps * 96, seed=31, max_reqs=3, max_ctx=512, k_scale=0.05 if dtype == "e4m3" else 1.0,
             v_scale=0.06 if dtype == "e4m3" else 1.0)
    rows = [1, 2, 3]
    lens, evicted = grow(P, rows, [200, 37, 0])
    rng = np.random.default_rng(8)
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    ang = np.arange(512)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    w = torch.tensor((1 + 0.2 * rng.standard_normal((2, 64))).astype(np.float32), device="cuda")
    for step in range(3):
        P.evict(rows, lens, evicted, 0)
        parents = [random_parents(rng, int(k)) for k in rng.integers(3, 15, 3)]
        S = TreeStep(P, rows, lens, parents, store=False)
        want_pos = [int(p) + d for p, t in zip(lens, parents) for d in TR.depths(t)]
        assert S.positions.cpu().tolist() == want_pos
        for l in range(2):
            qkv = torch.tensor(rng.standard_normal((S.n, 20, 64)), device="cuda").to(io)
            q = torch.empty((S.n, 16, 64), dtype=io, device="cuda")
            api.swa_qk_norm_rope_store(P.ctx, l, qkv[:, :16], qkv[:, 16:18], qkv[:, 18:], S.positions, S.slots[0], q,
                                       swa_loc=S.slots[1], q_weight=w[0], k_weight=w[1], eps=1e-6,
                                       cos_sin=torch.tensor(table, device="cuda"), rot_dim=64,
                                       k_scale=P.k_scale, v_scale=P.v_scale)
            x = qkv.float().cpu().numpy()
            k = TR.norm_rope(x[:, 16:18], w[1].cpu().numpy(), 1e-6, table, np.array(want_pos), 64, False)
            of, osw = P.last_alloc
            slots = of if P.layers[l][0] == OT.FULL else osw
            at = dev(slots)
            raw = P.kv[l][0][at]
            got = (raw.view(torch.float8_e4m3fn) if dtype == "e4m3" else raw).float().cpu().numpy()
            half = {"f32": 2.0 ** -18, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}[dtype]   # f32: D + 8 steps of 2^-24
            assert (np.abs(got * P.k_scale - k) <= 1.01 * half * np.abs(k) + 2.0 ** -18 * 4 + P.k_scale * 2.0 ** -10 * (dtype == "e4m3")).all()
            # from here on the oracle holds the stored bytes
            for is_v in range(2):
                host = P.kv[l][is_v][at].cpu()
                host = host.view(torch.int16).numpy().view(np.uint16) if dtype == "bf16" else host.numpy()
                for i, s in enumerate(slots):
                    P.op._rows(l, bool(is_v), [s])[0][...] = host[i]
            out = torch.empty_like(q)
            S.run(l, q, out, S.workspace(l))
            a, ref, mag = S.oracle(l, q.float().cpu().numpy())
            assert_attention(out.float().cpu().numpy()[a], ref, mag, dtype, f"step {step} layer {l}")
        P.check_state()
        # verification accepts a random path from a root
        kept = []
        for t in parents:
            path = TR.paths(t)[int(rng.integers(0, len(t)))]
            kept.append(path[:max(1, len(path) - 1)])
        acc = np.zeros((3, max(map(len, kept))), np.int32)
        for b, a in enumerate(kept):
            acc[b, :len(a)] = a
            TR.commit(P.op, P.oa.mapping, P.ort[rows[b]], int(lens[b]), a)
        api.swa_commit_tree(P.ctx, P.rt, S.d["rows"], S.d["pre"], dev(acc, torch.int32),
                            dev([len(a) for a in kept], torch.int32))
        P.check_state()
        new = lens + np.array([len(a) for a in kept])
        for b, r in enumerate(rows):
            keep_to = -(-int(new[b]) // ps) * ps
            idx = [int(i) for i in P.ort[r, keep_to:int(S.seq[b])]]
            if idx:
                api.swa_free(P.ctx, dev(idx), len(set(i // ps for i in idx)),
                             len(set(P.oa.mapping[i] // ps for i in idx if P.oa.mapping[i] > 0)))
                P.oa.free(idx)
            P.rt[r, int(new[b]):].zero_()
            P.ort[r, int(new[b]):] = 0
        P.check_state()
        lens = new
    P.extend(rows, lens, lens + 1)
    for l, (g, o) in P.decode_attention(rows, lens + 1).items():
        assert_close(g, o, TOL[dtype], f"decode layer {l}")
    assert api.swa_device_check(P.ctx) == 0
