"""Oracle: draft trees over a paged cache, per-head q/k norm with rotation, and
row moves.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A request with ``prefix`` cached tokens carries drafted nodes 0, 1, ... at
columns ``prefix + i`` of its req_to_token row.  Node i is a child of node
``parents[i] < i``, or of the last cached token when ``parents[i] = -1``; its
position is ``prefix`` plus the number of its ancestors among the nodes.  It
attends every cached position its layer kind allows from its own position
(``attention.key_positions``) and those of its ancestors, itself included,
whose positions are allowed.  All arithmetic is float64.
"""
from __future__ import annotations

import numpy as np

from . import attention as A


def paths(parents) -> list:
    """For each node, its ancestors from the root down to itself."""
    out = []
    for i, p in enumerate(parents):
        assert -1 <= p < i
        out.append((out[p] if p >= 0 else []) + [i])
    return out


def depths(parents) -> list:
    return [len(p) - 1 for p in paths(parents)]


def node_columns(kind: int, window: int, prefix: int, parents, i: int) -> list:
    """Columns node i reads, ascending."""
    path = paths(parents)[i]
    allowed = A.key_positions(kind, window, prefix + len(path) - 1)
    return ([t for t in range(allowed.start, min(allowed.stop, prefix))]
            + [prefix + a for d, a in enumerate(path) if prefix + d in allowed])


def attend(pools, mapping, layer: int, row, prefix: int, parents, q, sinks, scale: float,
           k_scale=1.0, v_scale=1.0):
    """Outputs [n, Hq, D] of a request's nodes, and the weighted sums of the
    values' magnitudes (the scale that rounding errors are relative to)."""
    kind, window, _ = pools.layers[layer]
    out, mag = [], []
    for i in range(len(parents)):
        slots = [int(row[c]) for c in node_columns(kind, window, prefix, parents, i)]
        if kind != A.FULL:
            slots = [int(mapping[s]) for s in slots]
            assert all(s > 0 for s in slots), "in-window key has no SWA slot"
        K, V = pools.read(layer, slots, k_scale, v_scale)
        qi = np.asarray(q[i], np.float64)
        out.append(A.attend_heads(qi, K, V, sinks, scale))
        mag.append(A.attend_heads(qi, K, np.abs(V), sinks, scale))
    return np.stack(out), np.stack(mag)


def norm_rope(x, weight, eps: float, cos_sin, positions, rot: int, interleaved: bool):
    """Rows ``x[n, H, D]`` normalised over D (no weight: as they are), then their
    first ``rot`` values rotated in pairs."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y = x.copy()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c = np.asarray(cos_sin, np.float64)[positions, j][:, None]
        s = np.asarray(cos_sin, np.float64)[positions, rot // 2 + j][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def move_rows(pools, mapping, pairs) -> None:
    """Rows of all layers from full slots to full slots, one pair after another;
    a source without an SWA slot moves on full layers only."""
    for src, dst in pairs:
        for layer, (kind, _, _) in enumerate(pools.layers):
            a, b = int(src), int(dst)
            if kind != A.FULL:
                a, b = int(mapping[a]), int(mapping[b])
                if a <= 0:
                    continue
                assert b > 0
            for is_v in (False, True):
                pools._rows(layer, is_v, [b])[0][...] = pools._rows(layer, is_v, [a])[0].copy()


def commit(pools, mapping, row, prefix: int, accepted) -> None:
    """Accepted nodes' rows to the columns that follow the prefix."""
    move_rows(pools, mapping, [(row[prefix + a], row[prefix + j])
                               for j, a in enumerate(accepted) if a != j])
