"""Per-head q/k norm, rotation and KV store in one pass, against the float64
oracle: head sizes, types, rotations of a part of the head, both pairings,
strided inputs, absent parts, in-place queries, both layouts and pools; padding
and bad positions or slots; refusals."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from hybrid_sliding_window_gb300 import api  # noqa: E402
from oracle import attention as OT  # noqa: E402
from oracle import codecs as OC  # noqa: E402
from oracle import tree as TR  # noqa: E402
from tests.harness import Pair  # noqa: E402
from tests.spec_harness import dev  # noqa: E402

EPS = 1e-6


def _table(max_pos, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    ang = np.arange(max_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Run:
    """n tokens of two requests on a windowed and a full layer."""

    def __init__(self, Hq, hkv, D, dtype, ps=16, layout="per_layer", n=(37, 12), ks=1.0, vs=1.0, ring=0):
        self.P = P = Pair([(OT.SLIDING, 127, hkv), (OT.FULL, 0, hkv)], Hq=Hq, D=D, dtype=dtype, ps=ps,
                          size_full=ps * (256 // ps + 8), size_swa=ps * (256 // ps + 8), seed=5,
                          layout=layout, perm_free=True, k_scale=ks, v_scale=vs, ring_size=ring)
        self.slots = P.extend([1, 2], [0, 0], list(n), store=False)
        self.n = sum(n)
        rng = np.random.default_rng(6)
        self.io = torch.float32 if dtype == "f32" else torch.bfloat16
        self.qkv = torch.tensor(rng.standard_normal((self.n, Hq + 2 * hkv, D)) * 2, device="cuda").to(self.io)
        self.q, self.k, self.v = self.qkv.split([Hq, hkv, hkv], 1)
        self.wq, self.wk = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
        self.pos = rng.integers(0, 2048, self.n)
        self.Hq, self.hkv, self.D, self.dtype = Hq, hkv, D, dtype

    def rows(self, layer, is_v):
        """The stored rows of the tokens as values, and what the scale leaves of a unit."""
        P = self.P
        slots = P.last_alloc[0] if P.layers[layer][0] == OT.FULL else P.last_alloc[1]
        if P.op.layout == "per_layer":
            raw = P.kv[layer][int(is_v)][dev(slots)]
            raw = raw.view(torch.float8_e4m3fn) if raw.dtype == torch.uint8 else raw
            return raw.float().cpu().numpy().astype(np.float64)
        full = P.layers[layer][0] == OT.FULL
        P.op.raw[full][...] = (P.ctx.full_envelope if full else P.ctx.swa_envelope).cpu().numpy()
        return np.stack([P.op.decode(r, 1.0) for r in P.op._rows(layer, is_v, slots)])


def _norm_tol(x, w, want, rot, dtype):
    """The row is summed, scaled and rotated in f32: every step is off by at most
    a few half steps of 2^-24 relative (D + 8 for the sum's D additions, the
    reciprocal root's 2 ulp, the products), relative to the pair's magnitude; the
    result is then rounded once (half of 2^-8 for bf16; E4M3: 2^-4, or half its
    least step of 2^-9, after the division by the scale)."""
    amp = np.abs(TR.norm_rope(x, w, EPS if w is not None else 0.0, None, None, 0, False))
    big = np.max(amp, -1, keepdims=True) if rot else amp
    calc = (x.shape[-1] + 8) * 2.0 ** -24 * 2 * big
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]
    return calc + half * (np.abs(want) + calc) + 1e-30


def _close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3])


def _check(R, layer, rot, inter, weights, q_out, table, tokens=slice(None)):
    io = "f32" if R.dtype == "f32" else "bf16"
    w = (R.wq, R.wk) if weights else (None, None)
    pos = R.pos if rot else None
    q, k, v = (t.float().cpu().numpy().astype(np.float64) for t in (R.q, R.k, R.v))
    if q_out is not None:
        want = TR.norm_rope(q, w[0], EPS, table, pos, rot, inter)
        _close(q_out.float().cpu().numpy()[tokens], want[tokens], _norm_tol(q, w[0], want, rot, io)[tokens], "q")
    want = TR.norm_rope(k, w[1], EPS, table, pos, rot, inter)
    tol = _norm_tol(k, w[1], want, rot, "f32")
    got_k, got_v = R.rows(layer, False), R.rows(layer, True)
    if R.dtype == "e4m3":
        want, tol = np.clip(want / R.P.k_scale, -448, 448), tol / R.P.k_scale
        tol = tol + np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10)
        code = OC.e4m3_encode(v.astype(np.float32), R.P.v_scale)
        _close(got_k[tokens], want[tokens], tol[tokens], "k")
        np.testing.assert_array_equal(got_v[tokens], OC.e4m3_decode(code)[tokens])
    else:
        _close(got_k[tokens], want[tokens], _norm_tol(k, w[1], want, rot, io)[tokens], "k")
        np.testing.assert_array_equal(got_v[tokens], v[tokens])


def _call(R, layer, rot=0, inter=False, weights=True, table=None, q=None, q_out=None, **kw):
    P = R.P
    args = dict(q=R.q if q is None else q, k=R.k, v=R.v, positions=dev(R.pos) if rot else None,
                full_loc=R.slots[0], swa_loc=R.slots[1],
                q_weight=torch.tensor(R.wq, device="cuda") if weights else None,
                k_weight=torch.tensor(R.wk, device="cuda") if weights else None, eps=EPS,
                cos_sin=torch.tensor(table, device="cuda") if rot else None, rot_dim=rot,
                interleaved=inter, k_scale=P.k_scale, v_scale=P.v_scale)
    args.update(kw)
    q, k, v, pos, loc = (args.pop(n) for n in ("q", "k", "v", "positions", "full_loc"))
    if q is not None and q_out is None:
        q_out = torch.full((R.n, R.Hq, R.D), 9.0, dtype=R.io, device="cuda")
    api.swa_qk_norm_rope_store(P.ctx, layer, q, k, v, pos, loc, q_out, **args)
    return q_out


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("Hq,hkv,D,dtype,rot", [
    (64, 4, 128, "bf16", 128), (64, 8, 128, "bf16", 96), (64, 8, 64, "bf16", 64), (5, 1, 64, "bf16", 16),
    (8, 8, 32, "bf16", 32), (40, 8, 128, "e4m3", 64), (8, 2, 64, "e4m3", 64), (8, 4, 32, "e4m3", 0),
    (4, 1, 64, "f32", 64), (3, 3, 128, "f32", 112), (2, 1, 32, "f32", 16), (64, 4, 128, "bf16", 0)])
def test_norm_rotate_store(Hq, hkv, D, dtype, rot, inter):
    R = Run(Hq, hkv, D, dtype, ks=0.03 if dtype == "e4m3" else 1.0, vs=0.05 if dtype == "e4m3" else 1.0)
    table = _table(2048, rot) if rot else None
    for layer in range(2):
        for weights in (True, False):
            out = _call(R, layer, rot, inter, weights, table)
            _check(R, layer, rot, inter, weights, out, table)
    assert api.swa_device_check(R.P.ctx) == 0


@pytest.mark.parametrize("dtype,ring", [("bf16", 0), ("e4m3", 0), ("bf16", 300)])
def test_envelope_rings_and_own_translation(dtype, ring):
    """Envelope rows and rings; without swa_loc the mapping is read."""
    R = Run(16, 4, 128, dtype, layout="per_layer" if ring else "envelope", ks=0.03 if dtype == "e4m3" else 1.0, ring=ring)
    table = _table(2048, 128)
    for layer in range(2):
        out = _call(R, layer, 128, table=table, swa_loc=None)
        _check(R, layer, 128, False, True, out, table)
    assert api.swa_device_check(R.P.ctx) == 0


def test_absent_parts_strides_and_in_place():
    R = Run(16, 4, 128, "bf16")
    table = _table(2048, 128)
    want = _call(R, 1, 128, table=table)
    _check(R, 1, 128, False, True, want, table)
    # queries only: the pool keeps what it has
    before = R.rows(1, False)
    R.P.kv[1][1].zero_()
    out = _call(R, 1, 128, table=table, k=None, v=None, full_loc=None, swa_loc=None)
    assert torch.equal(out, want) and not R.P.kv[1][1].any()
    # keys only
    R.P.kv[1][0].zero_()
    P = R.P
    api.swa_qk_norm_rope_store(P.ctx, 1, None, R.k, R.v, dev(R.pos), R.slots[0], None,
                               k_weight=torch.tensor(R.wk, device="cuda"), eps=EPS,
                               cos_sin=torch.tensor(table, device="cuda"), rot_dim=128)
    np.testing.assert_array_equal(R.rows(1, False), before)
    # contiguous inputs, then the queries in place
    q = R.q.contiguous()
    assert torch.equal(_call(R, 1, 128, table=table, q=q, k=R.k.contiguous(), v=R.v.contiguous()), want)
    _call(R, 1, 128, table=table, q=q, q_out=q)
    assert torch.equal(q, want)
    # one token, and none
    one = torch.empty((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    api.swa_qk_norm_rope_store(P.ctx, 1, R.q[5:6], R.k[5:6], R.v[5:6], dev(R.pos[5:6]), R.slots[0][5:6], one,
                               q_weight=torch.tensor(R.wq, device="cuda"),
                               k_weight=torch.tensor(R.wk, device="cuda"), eps=EPS,
                               cos_sin=torch.tensor(table, device="cuda"), rot_dim=128)
    assert torch.equal(one[0], want[5])
    api.swa_qk_norm_rope_store(P.ctx, 1, R.q[:0], R.k[:0], R.v[:0], dev([]), R.slots[0][:0], one[:0])
    assert api.swa_device_check(P.ctx) == 0


def test_same_bytes_as_store_kv():
    """Without weights and rotation the pool holds what swa_store_kv stores."""
    for dtype in ("bf16", "e4m3", "f32"):
        R = Run(16, 4, 128, dtype, ks=0.03 if dtype == "e4m3" else 1.0, vs=0.02 if dtype == "e4m3" else 1.0)
        for layer in range(2):
            api.swa_store_kv(R.P.ctx, layer, R.k.contiguous(), R.v.contiguous(), R.slots[0], R.slots[1],
                             R.P.k_scale, R.P.v_scale)
            want = [t.clone() for t in R.P.kv[layer]]
            for t in R.P.kv[layer]:
                t.zero_()
            _call(R, layer, 0, weights=False)
            for a, b in zip(R.P.kv[layer], want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 1 / 448, 0.03, 1 / 3, 5.0, 1 + 2.0 ** -23, 2 - 2.0 ** -23,
                                   0.3 * 2.0 ** -100, 1e30, 3e38, 1.2e-38, 1e-38, 1e-40, 2.0 ** -149])
def test_e4m3_bytes_of_every_bf16_value(scale):
    """Every bf16 pattern as K and as V: the bytes that swa_store_kv stores, and
    the encoding of the float32 quotient."""
    R = Run(4, 4, 128, "e4m3", n=(96, 32))
    bits = np.random.default_rng(8).permutation(65536).astype(np.uint16).view(np.int16)
    R.k = torch.tensor(bits, device="cuda").view(torch.bfloat16).reshape(R.n, 4, 128)
    R.v = R.k.flip(0).contiguous()
    R.P.k_scale, R.P.v_scale = scale, scale
    api.swa_store_kv(R.P.ctx, 1, R.k, R.v, R.slots[0], R.slots[1], scale, scale)
    want = [t.clone() for t in R.P.kv[1]]
    for t in R.P.kv[1]:
        t.zero_()
    _call(R, 1, 0, weights=False)
    rows = dev(R.P.last_alloc[0])
    for x, t, w in zip((R.k, R.v), R.P.kv[1], want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
        x, got = x.float().cpu().numpy(), t[rows].view(torch.uint8).cpu().numpy().reshape(R.n, 4, 128)
        ok = np.isfinite(x)
        with np.errstate(all="ignore"):
            codes = OC.e4m3_encode(np.clip(x[ok] / np.float32(scale), -1e30, 1e30).astype(np.float32), 1.0)
        np.testing.assert_array_equal(got[ok], codes)


def test_not_a_number_stays_in_its_row():
    R = Run(16, 4, 128, "bf16")
    table = _table(2048, 64)
    clean = _call(R, 1, 64, table=table)
    R.qkv[7, 3, 5] = float("nan")
    R.qkv[9, 2, 100] = float("inf")         # not rotated, no norm below
    out = _call(R, 1, 64, table=table)
    bad = torch.isnan(out).any(-1)
    assert bad[7, 3] and bad[9, 2] and int(bad.sum()) == 2
    keep = torch.ones_like(bad)
    keep[7, 3] = keep[9, 2] = False
    assert torch.equal(out[keep], clean[keep])
    plain = _call(R, 1, 64, weights=False, table=table)
    assert plain[9, 2, 100] == float("inf") and not torch.isnan(plain[9, 2]).any()


def test_bad_positions_and_slots():
    R = Run(16, 4, 128, "bf16")
    table = _table(2048, 128)
    P = R.P
    for t in P.kv[1]:
        t.zero_()
    pos = R.pos.copy()
    pos[4], pos[11] = 2048, -1
    out = _call(R, 1, 128, table=table, positions=dev(pos))
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    assert (out[4] == 9).all() and (out[11] == 9).all()
    assert not R.rows(1, False)[[4, 11]].any()
    keep = [i for i in range(R.n) if i not in (4, 11)]
    _check(R, 1, 128, False, True, out, table, keep)
    loc = R.slots[0].clone()
    loc[2], loc[3] = -1, P.ctx.cfg.size_full + P.ps
    for t in P.kv[1]:
        t.zero_()
    out = _call(R, 1, 128, table=table, full_loc=loc)
    assert api.swa_device_check(P.ctx) == api.SWA_DEVERR_RANGE
    assert not R.rows(1, False)[[2, 3]].any()
    _check(R, 1, 128, False, True, out, table, [i for i in range(R.n) if i not in (2, 3)])
    assert not R.rows(1, True)[[2, 3]].any()


@pytest.mark.parametrize("dtype,D,Hq,hkv,n,rot,inter", [
    ("bf16", 64, 5, 1, 25001, 64, False),        # a token is a unit, 41 units of every CTA
    ("bf16", 128, 80, 80, 6900, 96, False),      # three chunks of 80 rows, 608 CTAs: 34 units, carries
    ("f32", 32, 160, 160, 6907, 32, True),
    ("e4m3", 64, 160, 160, 6901, 64, True),
    ("e4m3", 128, 40, 8, 21000, 64, False)])
def test_many_units_of_every_cta(dtype, D, Hq, hkv, n, rot, inter):
    """Calls long enough that a CTA turns its ring over many times and looks up
    positions and slots more than once: bit for bit the calls on 200 tokens at a
    time, in which a CTA has one unit; some tokens against the oracle; bad
    positions and slots anywhere leave their tokens alone."""
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    store = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}[dtype]
    ks, vs = (0.03, 0.05) if dtype == "e4m3" else (1.0, 1.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rows = -(-n // 16) * 16 + 16
    pool = [torch.zeros((rows, hkv, D), dtype=store, device="cuda") for _ in range(2)]
    ctx = api.SwaCtx([dict(kind=api.LAYER_SLIDING, window=127, num_kv_heads=hkv, k=pool[0], v=pool[1])], 16, rows - 16,
                     rows - 16, Hq, D, {"f32": api.DTYPE_F32, "bf16": api.DTYPE_BF16, "e4m3": api.DTYPE_E4M3}[dtype])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert n * -(-(Hq + 2 * hkv) * D * io.itemsize // 24576) > 32 * 4 * sms
    qkv = (torch.randn((n, Hq + 2 * hkv, D), generator=g, device="cuda") * 2).to(io)
    q, k, v = qkv.split([Hq, hkv, hkv], 1)
    w = 1 + 0.3 * torch.randn((2, D), generator=g, device="cuda")
    pos = torch.randint(0, 2048, (n,), generator=g, device="cuda")
    loc = torch.randperm(rows - 16, generator=g, device="cuda")[:n] + 16
    table = _table(2048, rot)
    td = torch.tensor(table, device="cuda")
    out = torch.empty((n, Hq, D), dtype=io, device="cuda")

    def call(a, b, pos=pos, loc=loc):
        api.swa_qk_norm_rope_store(ctx, 0, q[a:b], k[a:b], v[a:b], pos[a:b], loc[a:b], out[a:b], swa_loc=loc[a:b], q_weight=w[0],
                                   k_weight=w[1], eps=EPS, cos_sin=td, rot_dim=rot, interleaved=inter, k_scale=ks, v_scale=vs)

    def run(step, **kw):
        for t in (*pool, out):
            t.fill_(3)
        for a in range(0, n, step):
            call(a, min(n, a + step), **kw)
        return [t.clone() for t in (out, *pool)]

    want = run(200)
    assert all(torch.equal(a, b) for a, b in zip(run(n), want))
    assert api.swa_device_check(ctx) == 0
    # the oracle, on tokens of the first and later units
    some = np.unique(np.concatenate([[0, n - 1], np.random.default_rng(1).integers(0, n, 30)]))
    at = torch.tensor(some, device="cuda")
    f64 = lambda t: t[at].float().cpu().numpy().astype(np.float64)  # noqa: E731
    wq, wk, p = w[0].cpu().numpy(), w[1].cpu().numpy(), pos[at].cpu().numpy()
    io_name = "f32" if dtype == "f32" else "bf16"
    ref = TR.norm_rope(f64(q), wq, EPS, table, p, rot, inter)
    _close(f64(want[0]), ref, _norm_tol(f64(q), wq, ref, rot, io_name), "q")
    ref = TR.norm_rope(f64(k), wk, EPS, table, p, rot, inter)
    stored = [t[loc[at]] for t in want[1:]]
    if dtype == "e4m3":
        got = [t.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64) for t in stored]
        tol = _norm_tol(f64(k), wk, ref, rot, "f32") / ks
        ref = np.clip(ref / ks, -448, 448)
        _close(got[0], ref, tol + np.maximum(2.0 ** -4 * (np.abs(ref) + tol), 2.0 ** -10), "k")
        np.testing.assert_array_equal(got[1], OC.e4m3_decode(OC.e4m3_encode(f64(v).astype(np.float32), vs)))
    else:
        _close(stored[0].float().cpu().numpy(), ref, _norm_tol(f64(k), wk, ref, rot, io_name), "k")
        assert torch.equal(stored[1], v[at])
    # bad positions and slots, in units behind the first 32 too
    bad_pos, bad_loc = pos.clone(), loc.clone()
    no_pos, no_loc = [5, n // 2, n - 3], [9, n // 2 + 1, n - 1]
    bad_pos[no_pos] = torch.tensor([2048, -1, 1 << 40], device="cuda")
    bad_loc[no_loc] = torch.tensor([-1, rows, 1 << 40], device="cuda")
    got = run(n, pos=bad_pos, loc=bad_loc)
    assert api.swa_device_check(ctx) == api.SWA_DEVERR_RANGE
    want[0][no_pos] = 3
    for t in want[1:]:
        t[loc[no_pos + no_loc]] = 3
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_over_inputs_are_refused():
    """Queries written over a fused projection, shifted over themselves or over
    the keys; a contiguous q itself, one token's slice and the place behind the
    inputs are served."""
    R = Run(16, 4, 128, "bf16")
    L, P = api.lib(), R.P
    st, row = R.q.stride(0), 16 * 128
    q = R.q.contiguous()
    spare = torch.zeros(3 * R.n * row, dtype=torch.bfloat16, device="cuda")

    def call(qp, qs, out, n=R.n, k=R.k.data_ptr(), v=R.v.data_ptr(), ks=st):
        return L.swa_qk_norm_rope_store(P.ctx.handle, 1, qp, qs, k, ks, v, ks, n, None, None, None, 0.0, None, 0, 0, 0,
                                        R.slots[0].data_ptr(), None, 1.0, 1.0, out, None)

    base, bad = R.qkv.data_ptr(), api.SWA_ERR_INVALID
    assert call(base, st, base) == bad                                  # packed outputs over strided inputs
    assert call(q.data_ptr(), row, q.data_ptr() + 2 * row) == bad       # a token's shift
    assert call(q.data_ptr(), row, q.data_ptr() - 2 * row) == bad
    assert call(q.data_ptr(), row, R.k.data_ptr()) == bad               # over the keys, or the last value row
    assert call(q.data_ptr(), row, R.v.data_ptr() + 2 * ((R.n - 1) * st + 4 * 128 - 8)) == bad
    assert call(base, st, base, n=1) == 0 and call(q.data_ptr(), row, q.data_ptr()) == 0
    end = spare.data_ptr() + 2 * R.n * row
    assert call(spare.data_ptr(), row, end) == 0 and call(end, row, spare.data_ptr()) == 0
    torch.cuda.synchronize()
    assert api.swa_device_check(P.ctx) == 0


def test_refusals():
    R = Run(16, 4, 128, "bf16")
    table = torch.tensor(_table(64, 128), device="cuda")
    P, L = R.P, api.lib()
    pos = dev(R.pos % 64)
    out = torch.empty((R.n, 16, 128), dtype=torch.bfloat16, device="cuda")
    st = R.q.stride(0)

    def call(**kw):
        a = dict(layer=1, q=R.q.data_ptr(), qs=st, k=R.k.data_ptr(), ks=st, v=R.v.data_ptr(), vs=st, n=R.n,
                 pos=pos.data_ptr(), wq=None, wk=None, eps=1e-6, table=table.data_ptr(), max_pos=64, rot=128,
                 inter=0, full=R.slots[0].data_ptr(), swa=None, kscale=1.0, vscale=1.0, out=out.data_ptr())
        a.update(kw)
        return L.swa_qk_norm_rope_store(P.ctx.handle, *a.values(), None)

    for kw in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(q=None), dict(out=None), dict(k=None), dict(v=None),
               dict(full=None), dict(q=None, out=None, k=None, v=None), dict(rot=-16), dict(rot=8), dict(rot=144),
               dict(pos=None), dict(table=None), dict(max_pos=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(q=R.q.data_ptr() + 2), dict(k=R.k.data_ptr() + 8), dict(out=out.data_ptr() + 4), dict(table=table.data_ptr() + 4),
               dict(qs=st + 4), dict(vs=4 * 128 - 8), dict(ks=0)):
        assert call(**kw) == api.SWA_ERR_INVALID, kw
    assert call(n=0) == 0 and call() == 0 and call(rot=0, pos=None, table=None) == 0
    torch.cuda.synchronize()
    assert api.swa_device_check(P.ctx) == 0
    F = Run(8, 2, 64, "e4m3")
    with pytest.raises(api.SwaError):
        _call(F, 1, 0, k_scale=0.0)
