"""Drives the speculative-step calls and their oracle on a ``Pair`` (tests only)."""
from __future__ import annotations

import numpy as np
import torch

from hybrid_sliding_window_gb300 import api
from oracle import attention as OT
from oracle import tree as TR

# Half a rounding step relative to the value, by stored / output type.
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -8}


def dev(x, dtype=torch.int64):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def random_parents(rng, n, roots=0.1):
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(max(0, i - 6), i))
            for i in range(n)]


def grow(P, rows, prompt, step=256):
    """Requests grown to their prompts by chunks, evicting before each one."""
    n = len(rows)
    prompt = np.asarray(prompt, np.int64)
    lens, ev = np.zeros(n, np.int64), np.zeros(n, np.int64)
    while (lens < prompt).any():
        sel = [i for i in range(n) if lens[i] < prompt[i]]
        e = ev[sel].copy()
        P.evict([rows[i] for i in sel], lens[sel], e, 0)
        ev[sel] = e
        new = np.minimum(lens[sel] + step, prompt[sel])
        P.extend([rows[i] for i in sel], lens[sel], new)
        lens[sel] = new
    P.evict(rows, lens, ev, 0)
    return lens, ev


class TreeStep:
    """The drafted nodes of a batch: allocated, stored (unless store=False),
    planned on the device; ``attend`` runs a layer both ways."""

    def __init__(self, P, rows, lens, parents, store=True, max_new=None):
        self.P, self.rows, self.parents = P, list(rows), [list(p) for p in parents]
        self.pre = np.asarray(lens, np.int64)
        self.nodes = np.array([len(p) for p in parents], np.int64)
        self.seq = self.pre + self.nodes
        self.indptr = np.concatenate([[0], np.cumsum(self.nodes)])
        self.n = int(self.indptr[-1])
        self.max_new = int(max_new or max(1, self.nodes.max()))
        self.max_seq = int(max(1, self.seq.max()))
        self.slots = P.extend(self.rows, self.pre, self.seq, store=store)
        self.d = dict(rows=dev(self.rows), pre=dev(self.pre), seq=dev(self.seq), indptr=dev(self.indptr),
                      parents=dev([p for t in parents for p in t], torch.int32))
        self.positions = torch.full((self.n,), -7, dtype=torch.int64, device="cuda")
        bs = len(self.rows)
        self.plan = torch.zeros(api.swa_plan_bytes(P.ctx, bs, self.max_new), dtype=torch.uint8,
                                device="cuda")
        # any contents: what the plan does not write must not be read
        self.tree = torch.full((api.swa_tree_bytes(P.ctx, self.n, self.max_new),), 0xA5,
                               dtype=torch.uint8, device="cuda")
        self.make_plans()

    def make_plans(self, stream=None):
        api.swa_plan(self.P.ctx, self.P.rt, self.d["rows"], self.d["pre"], self.d["seq"], self.plan,
                     self.max_new, stream=stream)
        api.swa_tree_plan(self.P.ctx, self.d["parents"], self.d["pre"], self.d["indptr"], self.n,
                          self.max_new, self.tree, self.positions, stream=stream)

    def queries(self, layer):
        reqs = np.repeat(self.rows, self.nodes)
        cols = np.concatenate([np.arange(a, b) for a, b in zip(self.pre, self.seq)])
        return self.P.q_in(layer, reqs, cols)

    def workspace(self, layer):
        return torch.zeros(api.swa_attn_tree_ws_bytes(self.P.ctx, layer, len(self.rows), self.n,
                                                      self.max_new, self.max_seq),
                           dtype=torch.uint8, device="cuda")

    def run(self, layer, q, out, ws, stream=None, sinks=True):
        P = self.P
        api.swa_attn_tree(P.ctx, layer, P.rt, self.d["rows"], self.d["pre"], self.d["indptr"], self.n,
                          self.max_new, self.max_seq, self.plan, self.tree, q,
                          P.sinks_d[layer] if sinks else None, P.scale, out, ws, P.k_scale, P.v_scale,
                          stream=stream)

    def attend(self, layer, sinks=True):
        q = self.queries(layer)
        qd = self.P.to_dev(q)
        out = torch.empty_like(qd)
        ws = self.workspace(layer)
        self.run(layer, qd, out, ws, sinks=sinks)
        return out.float().cpu().numpy(), q

    def oracle(self, layer, q, sinks=True, requests=None):
        """(rows, outputs, magnitudes) of the given requests (default all)."""
        P = self.P
        at, ref, mag = [], [], []
        for b in range(len(self.rows)) if requests is None else requests:
            if not self.parents[b]:
                continue
            sl = slice(int(self.indptr[b]), int(self.indptr[b + 1]))
            o, m = TR.attend(P.op, P.oa.mapping, layer, P.ort[self.rows[b]], int(self.pre[b]),
                             self.parents[b], q[sl], P.sinks[layer] if sinks else None, P.scale,
                             P.k_scale, P.v_scale)
            at += list(range(sl.start, sl.stop))
            ref.append(o)
            mag.append(m)
        return np.array(at), np.concatenate(ref), np.concatenate(mag)

    def check(self, layer, sinks=True, requests=None, what="", bounds=(None, 8192)):
        """Against the oracle, with each bound on the lengths (the caller's
        max_seq_len; None: the longest sequence) - a large one makes the
        tensor-core kernel split and merge the keys of short requests too."""
        q = self.queries(layer)
        at, ref, mag = self.oracle(layer, q, sinks, requests)
        exact = self.max_seq
        for bound in bounds:
            self.max_seq = bound or exact
            g, _ = self.attend(layer, sinks)
            assert_attention(g[at], ref, mag, self.P.dtype, f"{what} layer {layer} bound {bound}")
        self.max_seq = exact


def assert_attention(got, ref, mag, dtype, what=""):
    """|got - ref| within what the roundings allow: every softmax weight may be
    off by half a step of the type it is held in (bf16; nothing for f32), and
    by 2^-12 of itself from its score (D = 128 products of up to ~7 in total
    magnitude, summed in f32: 128 x 2^-24 x 7 x log2 e < 2^-13, and the
    exponential's 2 ulp), so the weighted sum and the sum of weights are each
    off by that share of `mag` = sum w |v|; then the output is rounded once."""
    share = 2 * ((HALF["bf16"] if dtype != "f32" else 0.0) + 2.0 ** -12)
    tol = share * mag + HALF[dtype] * (np.abs(ref) + share * mag) + 2.0 ** -24
    bad = np.abs(got - ref) > tol
    if bad.any() or not np.isfinite(got).all():
        i = tuple(np.argwhere(bad | ~np.isfinite(got))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {i}: got "
                             f"{got[i]} want {ref[i]} tol {tol[i]}")
