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
HIDDEN = {  # the same with hidden tokens; share of them
    "sequence": (3, 128, (6400, 1, 1), (64, 1, 1), None, dict(), 0.02),
    "sequence_d64": (3, 64, (6400, 1, 1), (64, 1, 1), None, dict(cap=6.0, causal=True), 0.5),
    "video": (4, 128, (8, 28, 52), (4, 4, 4), 40, dict(), 0.3),
    "video_d64": (4, 64, (8, 28, 52), (4, 4, 4), 40, dict(cap=6.0, bias=2.0 ** -6), 0.3),
    "video688": (4, 64, (12, 24, 40), (6, 8, 8), 6, dict(causal=True), 0.1),
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


class Long:
    def __init__(self, bs, heads, D, grid, tile, keep, kw, hidden=0.0):  # noqa: F811
        self.heads, self.D, self.grid = heads, D, grid
        T, H, W = grid
        self.cap, self.slope, self.causal = kw.get("cap", 0.0), kw.get("bias", 0.0), kw.get("causal", False)
        self.plan = plan = bs.Plan(1, heads, D, T, H, W, rule="window", win=(T, H, W), tile=tile)
        N, L = plan.N, plan.L
        g = np.random.default_rng(31)
        self.kept = torch.ones((heads, N, N), dtype=torch.bool, device="cuda")
        if keep is not None:
            self.kept = torch.from_numpy(g.random((heads, N, N)) < keep / N).cuda()
            self.kept[0, N // 2] = False  # a query tile that keeps nothing
        self.idx = torch.argsort((~self.kept).to(torch.uint8), dim=-1, stable=True).to(torch.int32)[None].contiguous()
        self.cnt = self.kept.sum(-1).to(torch.int32)[None].contiguous()
        draw = lambda a: torch.from_numpy(a * g.standard_normal((1, L, heads, D))).to(torch.bfloat16).cuda()  # noqa: E731
        self.x = [draw(3.0), draw(1.0), draw(1.0), draw(1.0)]
        self.doc = None
        if hidden:
            self.doc = torch.from_numpy(-(g.random((1, L)) < hidden).astype(np.int32)).cuda()
        self.spoilt = [t.clone() for t in self.x]
        for t, y in zip(self.x, self.spoilt):
            if hidden:
                t[self.doc < 0], y[self.doc < 0] = 0.0, float("nan")
        slopes = torch.full((heads,), self.slope, device="cuda") if self.slope else None
        self.mod = bs.ScoreMod(softcap=self.cap, slopes=slopes, dist=DIST, causal=self.causal, doc=self.doc)
        self.tid, self.row = (torch.from_numpy(np.asarray(a)).cuda() for a in tiling.token_tile_and_row(T, H, W, tile))
        self.xyz = torch.from_numpy(rope.grid_positions(T, H, W)).cuda().double()

    def definition(self, h):
        def far(rows):
            return sum(w * (self.xyz[rows, a, None] - self.xyz[None, :, a]).abs() for a, w in enumerate(DIST))

        def see(rows):
            ok = self.kept[h][self.tid[rows]][:, self.tid]
            if self.causal:
                ok = ok & (self.xyz[None, :, 0] <= self.xyz[rows, 0, None])
            return ok if self.doc is None else ok & (self.doc[0] >= 0) & (self.doc[0, rows, None] >= 0)

        r = _definition(*(t[0, :, h].double() for t in self.x), see, far, self.D ** -0.5, self.cap, self.slope)
        span = sum(w * n for w, n in zip(DIST, self.grid))
        return r, 2.0 ** -20 * (r["score"] + self.slope * span) + 3e-7 * self.cap

    def check(self, r, e, h, names, natural, lse):
        """Natural outputs `names`, and the log-sum-exp [heads, L]."""
        for n, got in zip(names, natural):
            err = (got[0, :, h].double() - r[n]).abs()
            rel = 2.0 ** -8 + 2 * e if n == "o" else 2.0 ** -8 * 1.02 + 4 * e
            tol = rel * r[n + "_mag"] + 2.0 ** -8 * r[n].abs() + 1e-30
            assert torch.all(err <= tol), (n, h, float((err / tol).max()))
        dead = r["lse"] == -float("inf")
        assert torch.equal(lse[h] == -float("inf"), dead)
        tol = e + 2.0 ** -21 * (8 + r["lse"][~dead].abs())
        assert torch.all((lse[h].double() - r["lse"])[~dead].abs() <= tol)


def _training_step(bs, c, x):  # noqa: F811
    """Natural o, dq, dk, dv, the log-sum-exp [heads, L], the slopes' gradient."""
    plan = c.plan
    q, k, v, do = _tiled(bs, plan, *x)
    o, lse = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
    bs.attn_forward_mod(plan, c.mod, q, k, v, c.idx, c.cnt, o, plan.workspace("mod_forward"), lse=lse)
    grads = [_nan(plan.tiled_shape()) for _ in range(3)]
    ds = _nan((c.heads,), torch.float32) if c.slope else None
    bs.attn_backward_mod(plan, c.mod, q, k, v, o, do, lse, c.idx, c.cnt, *grads, plan.workspace("mod_backward"),
                         d_slopes=ds)
    assert bs.attn_check_device_status(plan) == 0
    natural = []
    for t in (o, *grads):
        natural.append(torch.empty(plan.natural_shape(), dtype=torch.bfloat16, device="cuda"))
        bs.attn_unreorder(plan, t, natural[-1])
    return natural, lse[0][:, c.tid, c.row], ds


@pytest.mark.parametrize("name", list(CASES))
def test_long_lists(bs, name):  # noqa: F811
    c = Long(bs, *CASES[name])
    natural, lse, ds = _training_step(bs, c, c.x)
    for h in range(c.heads):
        r, e = c.definition(h)
        c.check(r, e, h, ("o", "dq", "dk", "dv"), natural, lse)
        if c.slope:
            assert abs(float(ds[h]) - r["dslope"]) <= (2.0 ** -16 + 4 * e) * r["dslope_mag"]


@pytest.mark.parametrize("name", list(HIDDEN))
def test_hidden_tokens_in_long_lists(bs, name):  # noqa: F811
    """Rows of hidden tokens are taken out of tiles in flight, in step with their loads: many blocks, long lists,
    the same call again and again."""
    c = Long(bs, *HIDDEN[name])
    natural, lse, ds = _training_step(bs, c, c.spoilt)
    for h in range(c.heads):
        r, e = c.definition(h)
        c.check(r, e, h, ("o", "dq", "dk", "dv"), natural, lse)
    for _ in range(10):
        again, lse2, ds2 = _training_step(bs, c, c.spoilt)
        assert all(torch.equal(a, b) for a, b in zip(natural + [lse], again + [lse2]))
        assert ds is None or torch.equal(ds, ds2)
    ws = c.plan.workspace("mod_forward")
    for _ in range(10):
        o, lse2 = _nan(c.plan.natural_shape()), _nan((1, c.heads, c.plan.L), torch.float32)
        bs.attn_forward_natural_mod(c.plan, c.mod, *c.spoilt[:3], c.idx, c.cnt, o, ws, lse_nat=lse2)
        assert torch.equal(o, natural[0]) and torch.equal(lse2[0], lse)
