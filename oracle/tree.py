"""Oracle of the drafted-tree calls: tree attention, append positions,
verification of drafted tokens, commit of the accepted rows.

Plain definitions, node by node.  The verification runs in exact rational
arithmetic (``fractions``): a decision compares sums over the vocabulary with
a random threshold, so its reference carries no rounding at all.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .mla import attend_absorbed, rms_norm, rope_interleave


def ancestors(parent, s: int):
    """Node s and its ancestors, s first; None for an absent node (parent -2);
    ValueError for a chain that leaves the tree."""
    if parent[s] == -2:
        return None
    up = [s]
    while parent[up[-1]] != -1:
        p = int(parent[up[-1]])
        if not 0 <= p < up[-1] or parent[p] == -2:
            raise ValueError(f"node {up[-1]} has parent {p}")
        up.append(p)
    return up


def decode_tree(q, Lc, Rc, T, parent, kv_b, qk_nope, scale, rope_base=10000.0, rows=None):
    """Attention of node s over the prefix rows t < T[b] - S and the rows of its
    ancestors and itself, rotated to T[b] - S + depth(s); absent nodes give 0."""
    q = np.asarray(q)
    B, S, H = q.shape[:3]
    out = np.zeros((B, S, H, np.asarray(kv_b).shape[1] - qk_nope))
    for b in range(B):
        base = int(T[b]) - S
        for s in range(S):
            up = ancestors(parent[b], s)
            if up is None or (rows is not None and (b, s) not in rows):
                continue
            at = list(range(base)) + [base + j for j in sorted(up)]
            out[b, s] = attend_absorbed(q[b, s], Lc[b, at], Rc[b, at], kv_b, qk_nope, base + len(up) - 1, scale,
                                        rope_base)
    return out


def cache_append_tree(comp, kv_a_ln, rms_eps, T, parent, kv_lora, rope_base=10000.0):
    """New rows (latent [B,S,kv_lora], key [B,S,qk_rope], positions [B,S]); absent
    nodes have position -1 and zero rows."""
    comp = np.asarray(comp, dtype=np.float64)
    B, S = comp.shape[:2]
    lat, key = np.zeros((B, S, kv_lora)), np.zeros((B, S, comp.shape[2] - kv_lora))
    pos = np.full((B, S), -1)
    for b in range(B):
        for s in range(S):
            up = ancestors(parent[b], s)
            if up is None:
                continue
            pos[b, s] = int(T[b]) - S + len(up) - 1
            lat[b, s] = rms_norm(comp[b, s, :kv_lora], kv_a_ln, rms_eps)
            if key.shape[2]:
                key[b, s] = rope_interleave(comp[b, s, kv_lora:], float(pos[b, s]), rope_base)
    return lat, key, pos


def tree_verify(p, q, tokens, parent, u):
    """One sequence: p [S+1][V] (row 0 the committed context, row s+1 node s), q the
    same or None, tokens, parent [S], u [S+1] -> (path, token), exact."""
    S = len(tokens)
    at, path = 0, []
    while True:
        w = [max(Fraction(0), Fraction(float(x))) for x in p[at]]
        mass, taken = Fraction(1), None
        for s in range(S):
            if parent[s] != at - 1:
                continue
            x, us = int(tokens[s]), Fraction(float(u[s]))
            qx = Fraction(1) if q is None else Fraction(float(q[at][x]))
            if us * qx * mass < w[x]:
                taken = s
                break
            if q is None:
                mass, w[x] = max(Fraction(0), mass - w[x]), Fraction(0)
            else:
                w = [max(Fraction(0), wv - mass * Fraction(float(qv))) for wv, qv in zip(w, q[at])]
                mass = sum(w)
        if taken is None:
            break
        path.append(taken)
        at = taken + 1
    if sum(w) == 0:
        w = [Fraction(float(x)) for x in p[at]]
    left, token = Fraction(float(u[S])) * sum(w), None
    for x, wv in enumerate(w):
        left -= wv
        if left < 0:
            token = x
            break
    return path, token


def tree_commit(cache, T, path, n_acc):
    """The cache [B, T_cap, row] after the accepted rows moved, and the new lengths."""
    cache, S = np.array(cache), np.asarray(path).shape[1]
    T_out = []
    for b in range(len(T)):
        base, n = int(T[b]) - S, int(n_acc[b])
        cache[b, base:base + n] = cache[b, [base + int(i) for i in path[b][:n]]]
        T_out.append(base + n)
    return cache, T_out
