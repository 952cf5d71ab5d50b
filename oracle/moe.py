"""Routing to experts and the experts' products, fp64 (test infrastructure only).

The definitions are spelled out token by token and slot by slot: no sorting of
scores, no batching.  Matrices are those of ``oracle.fp8``; the experts' weights
are lists with one matrix each.
"""
from __future__ import annotations

import numpy as np
from scipy import special

from . import fp8


def scores(logits, kind: str) -> np.ndarray:
    x = np.asarray(logits, dtype=np.float64)
    if kind == "softmax":
        with np.errstate(invalid="ignore"):
            e = np.exp(x - x.max(1, keepdims=True))
            return e / e.sum(1, keepdims=True)
    return special.expit(x)


def route(logits, k, kind="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True,
          scale=1.0, mask=None):
    """(ids [T, k], weights [T, k] in fp64): slots without an expert are -1, 0."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    p = scores(x, kind)
    ids, w = np.full((T, k), -1, dtype=np.int64), np.zeros((T, k))
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    size = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        here = x[t] > -np.inf
        bad = np.isnan(x[t]).any() or (kind == "softmax" and np.isposinf(x[t]).any())
        bad = bad or np.isnan((p[t] + b)[here]).any()
        if bad:
            ids[t], w[t] = np.arange(k), np.nan
            continue
        c = np.where(here, x[t] if bias is None else p[t] + b, -np.inf)
        of_group = np.where(here, p[t], -np.inf) if bias is None and group_top == 2 else c
        score = []
        for g in range(groups):
            best = sorted((v for v in of_group[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:group_top]
            score.append(sum(best) if best else -np.inf)
        kept = [g for g in sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups] if score[g] > -np.inf]
        free = [e for e in range(E) if c[e] > -np.inf and e // size in kept]
        taken = sorted(free, key=lambda e: (-c[e], e))[:k]
        v = p[t][taken]
        if renormalize and len(taken):
            v = v / v.sum() if v.sum() > 0 else np.full(len(taken), 1.0 / len(taken))
        ids[t, :len(taken)], w[t, :len(taken)] = taken, v * scale
    return ids, w


def plan(ids, E):
    """(offsets [E + 1], order [T·k]): the slots of each expert, ascending."""
    flat = np.asarray(ids).reshape(-1)
    slots = [[i for i in range(flat.size) if flat[i] == e] for e in range(E)]
    order = [i for s in slots for i in s]
    offsets = np.cumsum([0] + [len(s) for s in slots])
    return offsets, np.array(order + [-1] * (flat.size - len(order)), dtype=np.int64)


def linear(a, b, bias, kind, residual):
    """(act(A·Bᵀ + bias) + residual, function of `grouped`: bound of its fp32
    error).  The activations' evaluation is bounded as in ``fp8.gated``; bias
    and residual add one rounding each."""
    c, mag = fp8.matmul(a, b)
    K = a[0].shape[1]
    v = c if bias is None else c + np.asarray(bias, dtype=np.float64)
    f = v if kind is None else fp8.activation(v, kind)
    y = f if residual is None else f + np.asarray(residual, dtype=np.float64)

    def bound(grouped):
        e = fp8.accumulation_bound(mag, K, grouped) + np.abs(v) * 2.0 ** -24
        if kind is not None:
            z = np.minimum(np.abs(v) + np.abs(v) ** 3 / 8, 100.0)
            e = 1.13 * e + np.abs(f) * 2.0 ** -24 * (8 + 4 * z) + 1e-37
        return e + np.abs(y) * 2.0 ** -24

    return y, bound


def gated(a, ids, gate, up, kind, grouped=False):
    """(h, bound) by sorted position, the positions without an expert left out."""
    k = ids.shape[1]
    offsets, order = plan(ids, len(gate))
    n = gate[0][0].shape[0]
    h, bound = np.zeros((offsets[-1], n)), np.zeros((offsets[-1], n))
    for e in range(len(gate)):
        s = order[offsets[e]:offsets[e + 1]]
        if len(s):
            rows = (a[0][s // k], a[1][s // k])
            h[offsets[e]:offsets[e + 1]], bound[offsets[e]:offsets[e + 1]] = fp8.gated(rows, gate[e], up[e], kind, grouped)
    return h, bound


def combined(h, ids, weights, down, residual, grouped=False, half_terms=False):
    """(y, bound): the sum over j in fp32 loses a rounding for each term, of the
    terms' magnitudes; so does the residual's.  half_terms: the terms are
    rounded to fp16 on their way, times a power of two for each row of a group
    of neighbouring columns that divides a block of 128 and that brings the
    group's largest term to 2^14 .. 2^15: half a step is 2^-11 of the term, or
    2^-25 of 2^-14 of the largest among fp16's subnormal numbers."""
    T, k = ids.shape
    offsets, order = plan(ids, len(down))
    n = down[0][0].shape[0]
    y, bound, size = np.zeros((T, n)), np.zeros((T, n)), np.zeros((T, n))
    w = np.asarray(weights, dtype=np.float64).reshape(-1)
    for e in range(len(down)):
        s = order[offsets[e]:offsets[e + 1]]
        if len(s) == 0:
            continue
        rows = slice(offsets[e], offsets[e + 1])
        c, mag = fp8.matmul((h[0][rows], h[1][rows]), down[e])
        b = fp8.accumulation_bound(mag, h[0].shape[1], grouped)
        np.add.at(y, s // k, c * w[s][:, None])
        np.add.at(bound, s // k, b * np.abs(w[s])[:, None])
        np.add.at(size, s // k, (np.abs(c) + b) * np.abs(w[s])[:, None])
        if half_terms:
            top = np.maximum.reduceat(np.abs(c) + b, np.arange(0, n, fp8.BLOCK), axis=1)[:, np.arange(n) // fp8.BLOCK]
            np.add.at(bound, s // k, ((np.abs(c) + b) * 2.0 ** -11 + top * 2.0 ** -39) * np.abs(w[s])[:, None])
    r = np.zeros((T, n)) if residual is None else np.asarray(residual, dtype=np.float64)
    return y + r, bound + size * 2.0 ** -24 * k + np.abs(y + r) * 2.0 ** -24
