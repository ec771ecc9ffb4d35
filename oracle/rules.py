"""Oracle: score rules (tanh cap, distance bias, causal, prefix and document
masks) on dense attention and on block scores, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

With z = scale q . k:  z <- cap tanh(z / cap);  z <- z - slope * distance;
hidden pairs get probability 0. A row that sees nothing has o = 0, lse = -inf
and takes part in no gradient.

Parity: the forward is pinned against `attention.dense_masked` with the rules
off and against a triple loop with them on; the backward (q, k, v and slope)
by central differences (tests/test_oracle_rules.py).
"""

from __future__ import annotations

import numpy as np

LOWEST = float(np.finfo(np.float32).min)


def distance(xyz_q, xyz_k, weights):
    """sum_a weights[a] |xyz_q[a] - xyz_k[a]| for every pair of rows."""
    d = np.abs(xyz_q[:, None].astype(np.float64) - xyz_k[None])
    return d @ np.asarray(weights, dtype=np.float64)


def visible(xyz_q, xyz_k, causal=False, prefix=0, doc_q=None, doc_k=None):
    ok = np.ones((len(xyz_q), len(xyz_k)), dtype=bool)
    if causal:
        tq, tk = xyz_q[:, None, 0], xyz_k[None, :, 0]
        ok &= (tk <= tq) | (tk < prefix)
    if doc_q is not None:
        ok &= (doc_q[:, None] == doc_k[None]) & (doc_k[None] >= 0)
    return ok


def attend(q, k, v, seen, scale, cap=0.0, slope=0.0, far=None, do=None):
    """q [Lq, D], k/v [Lk, D], seen bool [Lq, Lk] -> dict: o, lse, p; with do
    also dq, dk, dv, dslope and the magnitudes that bound their rounding."""
    q, k, v = (np.where(np.isfinite(x), x, 0.0).astype(np.float64) for x in (q, k, v))
    z = scale * (q @ k.T)
    gain = np.ones_like(z)
    if cap:
        th = np.tanh(z / cap)
        z, gain = cap * th, 1.0 - th * th
    if far is not None:
        z = z - slope * far
    z = np.where(seen, z, -np.inf)
    top = z.max(axis=1, keepdims=True) if z.shape[1] else np.full((len(q), 1), -np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(z - safe)
    tot = e.sum(axis=1, keepdims=True)
    p = e / np.where(tot > 0, tot, 1.0)
    with np.errstate(divide="ignore"):
        lse = (safe + np.log(tot))[:, 0]
    out = {"o": p @ v, "lse": lse, "p": p, "o_mag": p @ np.abs(v)}
    if do is None:
        return out
    do = np.where(np.isfinite(do), do, 0.0).astype(np.float64)
    live = tot[:, 0] > 0
    do = do * live[:, None]
    dp = do @ v.T
    dz = p * (dp - (do * out["o"]).sum(axis=1, keepdims=True))
    ds = dz * gain * scale
    out.update(dq=ds @ k, dk=ds.T @ q, dv=p.T @ do, dslope=0.0 if far is None else -float((dz * far).sum()))
    # |error| of dS when it, P and O are rounded with relative step 1, and the sums it enters.
    dmag = scale * gain * (np.abs(dz) + p * (np.abs(do) * out["o_mag"]).sum(axis=1, keepdims=True))
    out.update(dq_mag=dmag @ np.abs(k), dk_mag=dmag.T @ np.abs(q), dv_mag=p.T @ np.abs(do),
               dslope_mag=0.0 if far is None else float((p * np.abs(dp) * far).sum() + (p * far).sum(1) @ (p * np.abs(dp)).sum(1)))
    return out


def scores(S, tile_xyz, slopes=None, weights=(1.0, 1.0, 1.0), cap=0.0, causal=False, prefix=None, docs=None):
    """S [B, heads, N, N] under the rules; tile_xyz: per tile the [n, 3]
    coordinates of its real tokens; prefix [B]; docs: per batch and tile the
    ids of its real tokens."""
    out = S.astype(np.float64)
    if cap:
        out = cap * np.tanh(out / cap)
    if slopes is not None:
        mid = np.stack([x.mean(0) for x in tile_xyz])
        out = out - np.asarray(slopes, dtype=np.float64)[None, :, None, None] * distance(mid, mid, weights)
    N = len(tile_xyz)
    for b in range(S.shape[0]):
        for i in range(N):
            for j in range(N):
                hide = False
                if causal:
                    first = tile_xyz[j][:, 0].min()
                    hide = first > tile_xyz[i][:, 0].max() and first >= (0 if prefix is None else prefix[b])
                if docs is not None:
                    x, y = (d[d >= 0] for d in (docs[b][i], docs[b][j]))
                    hide = hide or x.size == 0 or y.size == 0 or x.min() > y.max() or y.min() > x.max()
                if hide:
                    out[b, :, i, j] = LOWEST
    return out
