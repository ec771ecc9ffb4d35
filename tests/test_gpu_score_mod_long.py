"""Attention under score rules and its backward over long lists, where no CTAs
share a block's steps, against the definition in fp64 (torch, a few thousand
query rows at a time). Tolerances as in test_gpu_score_mod.py."""
import numpy as np
import pytest
import torch

from oracle import rope, tiling
from tests.test_gpu_score_mod import _nan, _tiled, bs  # noqa: F401  (bs: fixture)

pytestmark = pytest.mark.gpu

DIST = (1.0, 0.5, 0.25)
CASES = {  # heads, D, grid, tile, kept tiles of a query tile (None: all), rules
    # 100 steps a block, 150 blocks of a pass: four ring stages.
    "sequence": (3, 128, (6400, 1, 1), (64, 1, 1), None, dict(cap=6.0, bias=2.0 ** -6, causal=True)),
    "sequence_d64": (3, 64, (6400, 1, 1), (64, 1, 1), None, dict(bias=2.0 ** -6)),
    # 4,000 tiles, so that lists of up to 4,000 steps leave room for three stages (D = 128).
    "tiles": (1, 128, (20, 40, 40), (2, 2, 2), 40, dict(cap=6.0, bias=2.0 ** -6, causal=True)),
    "tiles_no_rule": (1, 128, (20, 40, 40), (2, 2, 2), 40, dict()),
}


def _definition(q, k, v, do, see, far, scale, cap, slope):
    """Natural fp64 [L, D] tensors of one head; see(rows), far(rows): masks and distances of some query rows.
    Results and the magnitudes that bound their rounding (as oracle/rules.py's attend)."""
    L, D = q.shape
    r = {n: torch.zeros((L, D), dtype=torch.float64, device="cuda") for n in ("o", "dq", "dk", "dv")}
    r |= {n + "_mag": torch.zeros_like(r["o"]) for n in ("o", "dq", "dk", "dv")}
    r |= {"lse": torch.zeros(L, dtype=torch.float64, device="cuda"), "dslope": 0.0, "dslope_mag": 0.0, "score": 0.0}
    for rows in torch.arange(L, device="cuda").split(2000):
        z = scale * q[rows] @ k.T
        r["score"] = max(r["score"], float((scale * q[rows].abs() @ k.abs().T).max()))
        gain = torch.ones_like(z)
        if cap:
            th = torch.tanh(z / cap)
            z, gain = cap * th, 1 - th * th
        d = far(rows)
        z = (z - slope * d).masked_fill(~see(rows), -float("inf"))
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse.nan_to_num(neginf=0.0)[:, None])
        o, omag, g = p @ v, p @ v.abs(), do[rows]
        g = g * (lse > -float("inf"))[:, None]
        dp = g @ v.T
        dz = p * (dp - (g * o).sum(1, keepdim=True))
        ds, dmag = scale * gain * dz, scale * gain * (dz.abs() + p * (g.abs() * omag).sum(1, keepdim=True))
        r["lse"][rows], r["o"][rows], r["o_mag"][rows] = lse, o, omag
        r["dq"][rows], r["dq_mag"][rows] = ds @ k, dmag @ k.abs()
        r["dk"] += ds.T @ q[rows]
        r["dk_mag"] += dmag.T @ q[rows].abs()
        r["dv"] += p.T @ g
        r["dv_mag"] += p.T @ g.abs()
        r["dslope"] -= float((dz * d).sum())
        r["dslope_mag"] += float((p * dp.abs() * d).sum() + ((p * d).sum(1) * (p * dp.abs()).sum(1)).sum())
    return r


@pytest.mark.parametrize("name", list(CASES))
def test_long_lists(bs, name):  # noqa: F811
    heads, D, (T, H, W), tile, keep, kw = CASES[name]
    cap, slope, causal = kw.get("cap", 0.0), kw.get("bias", 0.0), kw.get("causal", False)
    plan = bs.Plan(1, heads, D, T, H, W, rule="window", win=(T, H, W), tile=tile)
    N, L = plan.N, plan.L
    g = np.random.default_rng(31)
    kept = torch.ones((heads, N, N), dtype=torch.bool, device="cuda")
    if keep is not None:
        kept = torch.from_numpy(g.random((heads, N, N)) < keep / N).cuda()
        kept[0, N // 2] = False  # a query tile that keeps nothing
    idx = torch.zeros((1, heads, N, N), dtype=torch.int32, device="cuda")
    order = torch.argsort((~kept).to(torch.uint8), dim=-1, stable=True).to(torch.int32)
    idx[0] = order
    cnt = kept.sum(-1).to(torch.int32)[None].contiguous()
    draw = lambda a: torch.from_numpy(a * g.standard_normal((1, L, heads, D))).to(torch.bfloat16)  # noqa: E731
    x = [draw(3.0), draw(1.0), draw(1.0), draw(1.0)]
    slopes = torch.full((heads,), slope, device="cuda") if slope else None
    mod = bs.ScoreMod(softcap=cap, slopes=slopes, dist=DIST, causal=causal)
    q, k, v, do = _tiled(bs, plan, *x)
    o, lse = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
    bs.attn_forward_mod(plan, mod, q, k, v, idx, cnt, o, plan.workspace("mod_forward"), lse=lse)
    grads = [_nan(plan.tiled_shape()) for _ in range(3)]
    ds = _nan((heads,), torch.float32) if slope else None
    bs.attn_backward_mod(plan, mod, q, k, v, o, do, lse, idx, cnt, *grads, plan.workspace("mod_backward"), d_slopes=ds)
    assert bs.attn_check_device_status(plan) == 0
    nat = []
    for t in (o, *grads):
        nat.append(torch.empty((1, L, heads, D), dtype=torch.bfloat16, device="cuda"))
        bs.attn_unreorder(plan, t, nat[-1])
    tid, row = (torch.from_numpy(np.asarray(a)).cuda() for a in tiling.token_tile_and_row(T, H, W, tile))
    xyz = torch.from_numpy(rope.grid_positions(T, H, W)).cuda().double()

    def far(rows):
        return sum(w * (xyz[rows, a, None] - xyz[None, :, a]).abs() for a, w in enumerate(DIST))

    for h in range(heads):
        def see(rows):
            ok = kept[h][tid[rows]][:, tid]
            return ok & (xyz[None, :, 0] <= xyz[rows, 0, None]) if causal else ok

        r = _definition(*(y[0, :, h].cuda().double() for y in x), see, far, D ** -0.5, cap, slope)
        e = 2.0 ** -20 * (r["score"] + slope * sum(w * n for w, n in zip(DIST, (T, H, W)))) + 3e-7 * cap
        for n, got, rel in zip(("o", "dq", "dk", "dv"), nat, (2.0 ** -8 + 2 * e, *[2.0 ** -8 * 1.02 + 4 * e] * 3)):
            err = (got[0, :, h].double() - r[n]).abs()
            tol = rel * r[n + "_mag"] + 2.0 ** -8 * r[n].abs() + 1e-30
            assert torch.all(err <= tol), (n, h, float((err / tol).max()))
        got = lse[0, h][tid, row].double()
        dead = r["lse"] == -float("inf")
        assert torch.equal(got == -float("inf"), dead)
        tol = e + 2.0 ** -21 * (8 + r["lse"][~dead].abs())
        assert torch.all((got - r["lse"])[~dead].abs() <= tol)
        if slope:
            assert abs(float(ds[h]) - r["dslope"]) <= (2.0 ** -16 + 4 * e) * r["dslope_mag"]
