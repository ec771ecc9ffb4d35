"""Attention, its backward and its routing under score rules, against the
fp64 oracle.

Tolerances. P is rounded to bf16 before P V (half a step: 2^-8 of each term)
and O once more, so |dO| <= 2^-8 (sum p |v| + |o|); scores carry fp32 errors
(2^-20 of sum |q_d k_d|, the cap's 3e-7 cap, fp32 sums of the bias), which
reach O as at most their double times sum p |v| and the log-sum-exp as they
are. In the backward P and dS are rounded to bf16 and so is the O in
rowsum(dO * O): the oracle sums those magnitudes (`*_mag`)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import e4m3, rope, rules, tiling
from tests.helpers import to64

pytestmark = pytest.mark.gpu

GRIDS = {  # B, heads, D, (T, H, W), tile, kept share (None: all tiles)
    "token": (1, 2, 64, (1, 1, 1), (4, 4, 4), None),
    "ragged": (2, 2, 128, (7, 6, 9), (4, 4, 4), 0.6),
    "ragged_d64": (1, 3, 64, (6, 9, 5), (4, 4, 4), 0.5),
    "tile248": (1, 2, 64, (5, 6, 10), (2, 4, 8), 0.7),
    "tile688": (1, 2, 128, (9, 9, 10), (6, 8, 8), None),
    "tile344": (1, 2, 128, (7, 6, 9), (3, 4, 4), 0.7),
    "seq63": (1, 2, 64, (63, 1, 1), (64, 1, 1), None),
    "seq64": (2, 1, 128, (64, 1, 1), (64, 1, 1), None),
    "seq65": (1, 2, 128, (65, 1, 1), (64, 1, 1), None),
    "seq400": (2, 2, 128, (400, 1, 1), (64, 1, 1), None),
    "seq2050": (1, 1, 128, (2050, 1, 1), (64, 1, 1), 0.6),
    "seq300_wide": (1, 2, 64, (300, 1, 1), (128, 1, 1), None),
}
RULES = {
    "off": dict(),
    "cap": dict(cap=4.0),
    "cap_wide": dict(cap=50.0),
    "bias": dict(bias=True),
    "causal": dict(causal=True),
    "prefix": dict(causal=True, prefix=True),
    "docs": dict(docs=3),
    "hidden": dict(docs=2, hidden=True),
    "all": dict(cap=6.0, bias=True, causal=True, prefix=True, docs=3, hidden=True),
}
DIST = (1.0, 0.5, 0.0)
PAIRS = [(g, r) for g in GRIDS for r in RULES if g in ("ragged", "tile688", "seq400") or r in ("cap", "all")]


@pytest.fixture(scope="module")
def bs():
    from block_sparse_attention_reorder_b200 import bsattn
    assert torch.cuda.is_available()
    return bsattn


class Case:
    def __init__(self, bs, grid, rule, seed=0, fp8=False, amp=3.0, random_docs=False):
        self.B, self.heads, self.D, (T, H, W), self.tile, share = GRIDS[grid]
        self.grid = (T, H, W)
        kw = RULES[rule]
        plan = bs.Plan(self.B, self.heads, self.D, T, H, W, rule="window", win=(T, H, W), tile=self.tile, qk_fp8=fp8)
        self.plan, self.L, N = plan, T * H * W, plan.N
        g = np.random.default_rng(seed + 17 * len(grid))
        draw = lambda a: torch.from_numpy(a * g.standard_normal(plan.natural_shape())).to(torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v, self.do = draw(amp), draw(1.0), draw(1.0), draw(1.0)
        self.xyz = rope.grid_positions(T, H, W)
        self.tid = tiling.token_tile_and_row(T, H, W, self.tile)[0]
        self.kept = np.ones((self.B, self.heads, N, N), dtype=bool) if share is None else \
            g.random((self.B, self.heads, N, N)) < share
        if share is not None:
            self.kept[0, 0, N // 2] = False  # a query tile that keeps nothing
        idx = np.zeros((self.B, self.heads, N, N), dtype=np.int32)
        for at in np.ndindex(idx.shape[:3]):
            j = np.nonzero(self.kept[at])[0]
            idx[at][:j.size] = j
        self.idx = torch.from_numpy(idx).cuda()
        self.cnt = torch.from_numpy(self.kept.sum(-1).astype(np.int32)).cuda()
        self.cap = kw.get("cap", 0.0)
        self.slopes = np.array([0.5 ** (h + 1) for h in range(self.heads)], np.float32) if kw.get("bias") else None
        self.causal = kw.get("causal", False)
        self.prefix = g.integers(-1, T + 2, self.B).astype(np.int32) if kw.get("prefix") else None
        self.doc = None
        if kw.get("docs"):
            if random_docs:
                self.doc = g.integers(0, kw["docs"], (self.B, self.L)).astype(np.int32)
            else:
                self.doc = np.sort(g.integers(0, kw["docs"], (self.B, self.L)), axis=1).astype(np.int32)
            if kw.get("hidden"):
                self.doc[g.random((self.B, self.L)) < 0.2] = -1
                self.doc[0, self.L - self.L // 3:] = -7
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        self.mod = bs.ScoreMod(softcap=self.cap, slopes=dev(self.slopes), dist=DIST, causal=self.causal,
                               prefix=dev(self.prefix), doc=dev(self.doc))

    def oracle(self, b, h, q, k, v, do=None):
        seen = self.kept[b, h][self.tid][:, self.tid]
        d = None if self.doc is None else self.doc[b]
        seen = seen & rules.visible(self.xyz, self.xyz, self.causal, 0 if self.prefix is None else self.prefix[b], d, d)
        far = None if self.slopes is None else rules.distance(self.xyz, self.xyz, DIST)
        slope = 0.0 if self.slopes is None else float(self.slopes[h])
        return rules.attend(q, k, v, seen, self.D ** -0.5, self.cap, slope, far, do)

    def score_error(self, q, k):
        """What a fp32 score may be off by: the dot product, the cap, the bias."""
        q, k = (np.where(np.isfinite(x), x, 0.0) for x in (q, k))
        far = 0.0 if self.slopes is None else float(self.slopes.max()) * sum(w * n for w, n in zip(DIST, self.grid))
        mag = self.D ** -0.5 * (np.abs(q) @ np.abs(k).T).max()
        return 2.0 ** -20 * (mag + far) + 3e-7 * self.cap

    def spoil(self):
        """NaN and infinities in every row of a hidden token."""
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.bfloat16)
        hide = torch.from_numpy(self.doc < 0)
        out = []
        for x in (self.q, self.k, self.v, self.do):
            y = x.clone()
            y[hide] = bad[torch.arange(self.D) % 3]
            out.append(y)
        return out

    def check_forward(self, o, lse, q, k, v):
        for b in range(self.B):
            for h in range(self.heads):
                r = self.oracle(b, h, q[b, :, h], k[b, :, h], v[b, :, h])
                e = self.score_error(q[b, :, h], k[b, :, h])
                err = np.abs(o[b, :, h] - r["o"])
                tol = (2.0 ** -8 + 2 * e) * r["o_mag"] + 2.0 ** -8 * np.abs(r["o"]) + 1e-30
                assert np.all(err <= tol), ("o", b, h, (err / tol).max())
                dead = np.isneginf(r["lse"])
                assert np.array_equal(np.isneginf(lse[b, h]), dead)
                tol = e + 2.0 ** -21 * (8 + np.abs(r["lse"][~dead]))
                assert np.all(np.abs(lse[b, h][~dead] - r["lse"][~dead]) <= tol), "lse"


def _tiled(bs, plan, *xs):
    out = []
    for x in xs:
        t = torch.empty(plan.tiled_shape(), dtype=torch.bfloat16, device="cuda")
        bs.attn_reorder(plan, x.cuda().contiguous(), t)
        out.append(t)
    return out


def _valid(c):
    """Rows of the tiled layout that hold a token (a tile of fewer than 64 is stored as 64 rows)."""
    rows = tiling.tile_valid_rows(*c.grid, c.tile)
    return torch.from_numpy(np.pad(rows, ((0, 0), (0, c.plan.V - rows.shape[1])))).cuda()


def _natural(c, t):
    rows = c.tile[0] * c.tile[1] * c.tile[2]
    return tiling.unreorder(to64(t)[:, :, :, :rows], *c.grid, c.tile)


def _nan(shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("grid,rule", PAIRS)
def test_forward_both_layouts(bs, grid, rule):
    c = Case(bs, grid, rule)
    plan, ws = c.plan, c.plan.workspace("mod_forward")
    o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(plan, c.mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse)
    assert bs.attn_check_device_status(plan) == 0
    c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, c.k, c.v)))
    ot, lt = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
    bs.attn_forward_mod(plan, c.mod, *_tiled(bs, plan, c.q, c.k, c.v), c.idx, c.cnt, ot, ws, lse=lt)
    assert bs.attn_check_device_status(plan) == 0
    valid = _valid(c)
    back = torch.empty_like(o)
    bs.attn_unreorder(plan, ot, back)
    assert torch.equal(back, o)
    assert torch.all(ot[:, :, ~valid] == 0) and torch.all(torch.isneginf(lt[:, :, ~valid]))


@pytest.mark.parametrize("grid,rule", [p for p in PAIRS if p[0] != "token"] + [("token", "all")])
def test_backward(bs, grid, rule):
    c = Case(bs, grid, rule, seed=1)
    plan = c.plan
    q, k, v, do = _tiled(bs, plan, c.q, c.k, c.v, c.do)
    o, lse = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
    bs.attn_forward_mod(plan, c.mod, q, k, v, c.idx, c.cnt, o, plan.workspace("mod_forward"), lse=lse)
    grads = [_nan(plan.tiled_shape()) for _ in range(3)]
    ds = None if c.slopes is None else _nan((c.heads,), torch.float32)
    bs.attn_backward_mod(plan, c.mod, q, k, v, o, do, lse, c.idx, c.cnt, *grads, plan.workspace("mod_backward"),
                         d_slopes=ds)
    assert bs.attn_check_device_status(plan) == 0
    valid = _valid(c)
    for t in grads:
        assert torch.all(t[:, :, ~valid] == 0)
    _check_grads(c, grads, ds, *(to64(x) for x in (c.q, c.k, c.v, c.do)))


def _check_grads(c, grads, ds, q, k, v, do):
    nat = [_natural(c, t) for t in grads]
    for h in range(c.heads):
        dslope = mag = 0.0
        for b in range(c.B):
            r = c.oracle(b, h, *(x[b, :, h] for x in (q, k, v, do)))
            e = c.score_error(q[b, :, h], k[b, :, h])
            for name, got in zip(("dq", "dk", "dv"), nat):
                err = np.abs(got[b, :, h] - r[name])
                tol = (2.0 ** -8 * 1.02 + 4 * e) * r[name + "_mag"] + 2.0 ** -8 * np.abs(r[name]) + 1e-30
                assert np.all(err <= tol), (name, b, h, (err / tol).max())
            dslope += r["dslope"]
            mag += r["dslope_mag"]
        if ds is not None:
            assert abs(float(ds[h]) - dslope) <= (2.0 ** -16 + 4 * e) * mag + 1e-30


@pytest.mark.parametrize("grid", ["ragged", "tile688", "tile344", "seq400"])
@pytest.mark.parametrize("rule", ["hidden", "all"])
def test_hidden_rows_may_hold_anything(bs, grid, rule):
    c = Case(bs, grid, rule, seed=2)
    plan, ws = c.plan, c.plan.workspace("mod_forward")
    bad = c.spoil()
    o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(plan, c.mod, *(x.cuda() for x in bad[:3]), c.idx, c.cnt, o, ws, lse_nat=lse)
    c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, c.k, c.v)))
    res = []
    for xs in ((c.q, c.k, c.v, c.do), bad):
        q, k, v, do = _tiled(bs, plan, *xs)
        ot, lt = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
        bs.attn_forward_mod(plan, c.mod, q, k, v, c.idx, c.cnt, ot, ws, lse=lt)
        grads = [_nan(plan.tiled_shape()) for _ in range(3)]
        ds = None if c.slopes is None else _nan((c.heads,), torch.float32)
        bs.attn_backward_mod(plan, c.mod, q, k, v, ot, do, lt, c.idx, c.cnt, *grads, plan.workspace("mod_backward"),
                             d_slopes=ds)
        assert bs.attn_check_device_status(plan) == 0
        res.append([ot, lt, *grads] + ([] if ds is None else [ds]))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("grid", ["ragged", "ragged_d64", "tile688", "seq400"])
def test_without_a_workspace(bs, grid):
    """No CTAs share a query block then: the same tolerances."""
    c = Case(bs, grid, "cap", seed=7)
    o, lse = _nan(c.plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(c.plan, c.mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o, lse_nat=lse)
    assert bs.attn_check_device_status(c.plan) == 0
    c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, c.k, c.v)))


def test_large_and_falling_scores(bs):
    """Scores far apart within a row, so that references move and parts of a row's keys vanish."""
    for amp, grid in ((300.0, "seq400"), (300.0, "ragged"), (2000.0, "seq400")):
        c = Case(bs, grid, "off", seed=8, amp=amp)
        for order in (1, -1):  # the largest scores last, first
            k = c.k.double().numpy()
            k = torch.from_numpy(k * np.linspace(0, 1, c.L)[::order][None, :, None, None]).to(torch.bfloat16)
            for ws in (None, c.plan.workspace("mod_forward")):
                o, lse = _nan(c.plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
                bs.attn_forward_natural_mod(c.plan, c.mod, c.q.cuda(), k.cuda(), c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse)
                c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, k, c.v)))


@pytest.mark.parametrize("grid", ["ragged", "seq400", "tile688"])
def test_ids_in_any_order(bs, grid):
    c = Case(bs, grid, "all", seed=3, random_docs=True)
    o, lse = _nan(c.plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(c.plan, c.mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o,
                                c.plan.workspace("mod_forward"), lse_nat=lse)
    c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, c.k, c.v)))


@pytest.mark.parametrize("grid", ["ragged", "tile688"])
def test_everything_hidden(bs, grid):
    c = Case(bs, grid, "hidden", seed=4)
    doc = torch.full((c.B, c.L), -1, dtype=torch.int32, device="cuda")
    mod = bs.ScoreMod(softcap=5.0, doc=doc)
    q, k, v, do = _tiled(bs, c.plan, c.q, c.k, c.v, c.do)
    o, lse = _nan(c.plan.tiled_shape()), _nan(c.plan.tiled_shape()[:-1], torch.float32)
    bs.attn_forward_mod(c.plan, mod, q, k, v, c.idx, c.cnt, o, c.plan.workspace("mod_forward"), lse=lse)
    grads = [_nan(c.plan.tiled_shape()) for _ in range(3)]
    bs.attn_backward_mod(c.plan, mod, q, k, v, o, do, lse, c.idx, c.cnt, *grads, c.plan.workspace("mod_backward"))
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse)) and all(torch.all(x == 0) for x in grads)


@pytest.mark.parametrize("grid,rule", [("ragged", "all"), ("ragged_d64", "cap"), ("tile688", "all"), ("seq400", "bias")])
def test_forward_e4m3(bs, grid, rule):
    c = Case(bs, grid, rule, seed=5, fp8=True)
    plan, ws = c.plan, c.plan.workspace("mod_forward")
    codes, scales, values = [], [], []
    for x in (c.q, c.k):
        code, scale = e4m3.quantize_tiled(tiling.reorder(x.float().numpy(), *c.grid, c.tile))
        codes.append(torch.from_numpy(code).cuda())
        scales.append(torch.from_numpy(scale).cuda())
        values.append(tiling.unreorder(e4m3.dequantize_tiled(code, scale), *c.grid, c.tile).astype(np.float64))
    o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(plan, c.mod, *codes, c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse, q_scale=scales[0],
                                k_scale=scales[1])
    assert bs.attn_check_device_status(plan) == 0
    c.check_forward(to64(o), to64(lse), *values, to64(c.v))
    ot = _nan(plan.tiled_shape())
    bs.attn_forward_mod(plan, c.mod, *codes, *_tiled(bs, plan, c.v), c.idx, c.cnt, ot, ws, q_scale=scales[0],
                        k_scale=scales[1])
    back = torch.empty_like(o)
    bs.attn_unreorder(plan, ot, back)
    assert torch.equal(back, o)


@pytest.mark.parametrize("rule", ["bias", "all"])
def test_e4m3_tiles_of_tiny_values(bs, rule):
    """Scales whose product is no fp32 number: the scores are zero, the rest of the rules holds."""
    c = Case(bs, "ragged", rule, seed=5, fp8=True)
    plan, ws = c.plan, c.plan.workspace("mod_forward")
    codes, scales = [], []
    for x, tiny in ((c.q, 1e-36), (c.k, 1e-25)):
        code, scale = e4m3.quantize_tiled(tiling.reorder(x.float().numpy(), *c.grid, c.tile))
        codes.append(torch.from_numpy(code).cuda())
        scales.append((torch.from_numpy(scale) * tiny).cuda())
    o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
    bs.attn_forward_natural_mod(plan, c.mod, *codes, c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse, q_scale=scales[0],
                                k_scale=scales[1])
    assert bs.attn_check_device_status(plan) == 0
    zero = np.zeros(plan.natural_shape())
    c.check_forward(to64(o), to64(lse), zero, zero, to64(c.v))


# ---------------------------------------------------------------- routing

def _tile_lists(c):
    N = c.plan.N
    rows = [np.nonzero(c.tid == j)[0] for j in range(N)]
    return rows, [c.xyz[r] for r in rows]


@pytest.mark.parametrize("random_docs", [False, True])
@pytest.mark.parametrize("grid,rule", [("ragged", r) for r in RULES] + [("tile688", "all"), ("seq400", "all"),
                                                                       ("token", "all"), ("tile344", "all")])
def test_scores(bs, grid, rule, random_docs):
    c = Case(bs, grid, rule, seed=6, random_docs=random_docs)
    N = c.plan.N
    rows, xyz = _tile_lists(c)
    S = (4 * np.random.default_rng(7).standard_normal((c.B, c.heads, N, N))).astype(np.float32)
    S[0, 0, 0, 0] = -np.inf
    docs = None if c.doc is None else [[c.doc[b][r] for r in rows] for b in range(c.B)]
    want = rules.scores(S, xyz, c.slopes, DIST, c.cap, c.causal, c.prefix, docs)
    t = torch.from_numpy(S).cuda()
    out = _nan(t.shape, torch.float32)
    bs.attn_mod_scores(c.plan, c.mod, t, out, c.plan.workspace("mod_scores"))
    got = to64(out)
    low = want == rules.LOWEST
    assert np.array_equal(got == rules.LOWEST, low)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fine = ~low & ~inf
    # cap: 3e-7 of it; products, differences and sums of the bias: 2^-22 of their magnitude.
    tol = 3e-7 * c.cap + 2.0 ** -22 * (np.abs(S[fine]) + np.abs(want[fine] - S[fine]))
    assert np.all(np.abs(got[fine] - want[fine]) <= tol)
    bs.attn_mod_scores(c.plan, c.mod, t, t, c.plan.workspace("mod_scores"))  # in place
    assert torch.equal(t, out)


# ---------------------------------------------------------------- the whole layer

def _layer_plan(bs, rule, fp8=False, tile=(4, 4, 4), B=2, heads=3, D=128, grid=(9, 10, 13)):
    kw = {"topk": dict(rule="topk", k=5), "topp": dict(rule="topp", k=2, p=0.8), "window": dict(rule="window", win=(1, 1, 1))}
    return bs.Plan(B, heads, D, *grid, tile=tile, qk_fp8=fp8, **kw[rule])


def _layer_inputs(plan, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(plan.natural_shape(), generator=g).to(torch.bfloat16).cuda() for _ in range(3)]


def _layer_mod(bs, plan, hidden=False):
    g = np.random.default_rng(8)
    doc = np.sort(g.integers(0, 3, (plan.B, plan.L)), axis=1).astype(np.int32)
    if hidden:
        doc[:, plan.L - plan.L // 5:] = -1
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return bs.ScoreMod(softcap=12.0, slopes=dev(np.array([0.3, 0.1, 0.05], np.float32)), dist=(1.0, 0.5, 0.5),
                       causal=True, prefix=dev(np.array([2, 0], np.int32)), doc=dev(doc))


@pytest.mark.parametrize("rule,fp8,tile", [("topk", False, (4, 4, 4)), ("topp", False, (4, 4, 4)),
                                           ("window", False, (4, 4, 4)), ("topk", True, (4, 4, 4)),
                                           ("window", True, (6, 8, 8)), ("topk", False, (3, 4, 4))])
def test_layer_equals_its_steps(bs, rule, fp8, tile):
    plan = _layer_plan(bs, rule, fp8, tile)
    q, k, v = _layer_inputs(plan, 9)
    r, mod = bs.Rope(dims=(44, 42, 42), offset=(100, 0, 0)), _layer_mod(bs, plan)
    si, sc = plan.list_shapes()
    idx, cnt = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (si, sc))
    o, lse = _nan(plan.natural_shape()), _nan((plan.B, plan.heads, plan.L), torch.float32)
    bs.attn_layer_mod(plan, r, mod, q, k, v, o, plan.workspace("mod_layer"), lse_nat=lse, idx=idx, cnt=cnt)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    means = [torch.empty((plan.B, plan.heads, plan.N, plan.D), device="cuda") for _ in range(2)]
    bs.attn_rope(plan, r, q, qr, k, kr, *means)
    S = torch.empty((plan.B, plan.heads, plan.N, plan.N), device="cuda")
    idx2, cnt2 = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (si, sc))
    bs.attn_block_scores(plan, *means, S)
    bs.attn_mod_scores(plan, mod, S, S, plan.workspace("mod_scores"))
    bs.attn_select_from_scores(plan, S, idx2, cnt2)
    qs = ks = None
    if fp8:
        pair = []
        for x in (qr, kr):
            t, = _tiled(bs, plan, x)
            code = torch.empty(plan.tiled_shape(), dtype=torch.uint8, device="cuda")
            scale = torch.empty((plan.B, plan.heads, plan.N), device="cuda")
            bs.attn_quantize_e4m3(plan, t, code, scale)
            pair.append((code, scale))
        (qr, qs), (kr, ks) = pair
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    bs.attn_forward_natural_mod(plan, mod, qr, kr, v, idx2, cnt2, o2, plan.workspace("mod_forward"), lse_nat=lse2,
                                q_scale=qs, k_scale=ks)
    assert bs.attn_check_device_status(plan) == 0
    assert torch.equal(cnt, cnt2)
    live = torch.arange(plan.kmax, device="cuda") < cnt[..., None]
    assert torch.equal(idx[live], idx2[live])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rule,fp8", [("topk", False), ("topk", True), ("window", True), ("topp", False)])
@pytest.mark.parametrize("rotate", [True, False])
def test_layer_ignores_what_hidden_tokens_hold(bs, rule, fp8, rotate):
    plan = _layer_plan(bs, rule, fp8)
    q, k, v = _layer_inputs(plan, 10)
    mod = _layer_mod(bs, plan, hidden=True)
    r = bs.Rope(dims=(44, 42, 42)) if rotate else None
    outs = []
    for spoil in (False, True):
        if spoil:
            for x in (q, k, v):
                x[mod.doc < 0] = float("nan")
        o, lse = _nan(plan.natural_shape()), _nan((plan.B, plan.heads, plan.L), torch.float32)
        bs.attn_layer_mod(plan, r, mod, q, k, v, o, plan.workspace("mod_layer"), lse_nat=lse)
        assert bs.attn_check_device_status(plan) == 0
        outs.append((o, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.all(outs[0][0][mod.doc < 0] == 0)


def test_layer_without_rope_and_rules_is_attn_layer(bs):
    plan = _layer_plan(bs, "topk")
    q, k, v = _layer_inputs(plan, 11)
    o, want = _nan(plan.natural_shape()), _nan(plan.natural_shape())
    bs.attn_layer_mod(plan, None, None, q, k, v, o, plan.workspace("mod_layer"))
    bs.attn_layer(plan, q, k, v, want, plan.workspace("layer"))
    assert torch.equal(o, want)


def test_layer_and_training_step_in_a_graph_beside_another_stream(bs):
    plan = _layer_plan(bs, "topk")
    r, mod = bs.Rope(dims=(44, 42, 42)), _layer_mod(bs, plan, hidden=True)
    ins = [_layer_inputs(plan, 12 + s) for s in range(2)]
    si, sc = plan.list_shapes()

    class Step:
        def __init__(self):
            self.x = [t.clone() for t in ins[0]]
            self.o = torch.empty_like(self.x[0])
            self.idx, self.cnt = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (si, sc))
            self.t = [torch.zeros(plan.tiled_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(7)]
            self.lse = torch.zeros(plan.tiled_shape()[:-1], device="cuda")
            self.ds = torch.zeros(plan.heads, device="cuda")
            self.ws = [plan.workspace(w) for w in ("mod_layer", "mod_forward", "mod_backward")]

        def run(self):
            bs.attn_layer_mod(plan, r, mod, *self.x, self.o, self.ws[0], idx=self.idx, cnt=self.cnt)
            for x, t in zip(self.x, self.t):
                bs.attn_reorder(plan, x, t)
            bs.attn_forward_mod(plan, mod, *self.t[:3], self.idx, self.cnt, self.t[3], self.ws[1], lse=self.lse)
            bs.attn_backward_mod(plan, mod, *self.t[:3], self.t[3], self.t[2], self.lse, self.idx, self.cnt,
                                 *self.t[4:], self.ws[2], d_slopes=self.ds)

        def out(self):
            return [self.o, self.t[3], self.lse, *self.t[4:], self.ds]

    a, other, ref = Step(), Step(), Step()
    ref.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for xs in (ins[1], ins[0]):
        for x, y in zip(a.x, xs):
            x.copy_(y)
        graph.replay()
        with torch.cuda.stream(side):
            other.run()  # at the same time, with its own workspaces
        for x, y in zip(ref.x, xs):
            x.copy_(y)
        ref.run()
        torch.cuda.synchronize()
        assert bs.attn_check_device_status(plan) == 0
        assert all(torch.equal(x, y) for x, y in zip(a.out(), ref.out()))
    assert all(torch.equal(x, y) for x, y in zip(other.out(), ref.out()))
    del graph


# ---------------------------------------------------------------- refusals

def _mod_calls(bs, c, mod, ws="mod_forward"):
    plan = c.plan
    o = _nan(plan.natural_shape())
    bs.attn_forward_natural_mod(plan, mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o,
                                plan.workspace(ws) if ws else None)


def test_timeouts_and_bad_lists_are_reported(bs):
    c = Case(bs, "ragged", "all")
    plan, ws = c.plan, c.plan.workspace("mod_forward")
    run = lambda idx, o: bs.attn_forward_natural_mod(plan, c.mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), idx, c.cnt, o, ws)  # noqa: E731
    o = torch.empty(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    bs.attn_testing_force_timeout(True)
    try:
        run(c.idx, o)
        assert bs.attn_check_device_status(plan) == 4
    finally:
        bs.attn_testing_force_timeout(False)
    run(c.idx, o)  # and works again
    assert bs.attn_check_device_status(plan) == 0
    bad = c.idx.clone()
    bad[0, 1, 0, 0] = plan.N  # out of range: skipped and reported
    again = torch.empty_like(o)
    run(bad, again)
    assert bs.attn_check_device_status(plan) == 5
    assert torch.equal(again[1:], o[1:])


@pytest.mark.parametrize("kw", [dict(softcap=1e-7), dict(softcap=1e31), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                                dict(dist=(1.0, -1.0, 0.0)), dict(dist=(float("nan"), 0.0, 0.0)), dict(prefix=True)])
def test_bad_rules_are_refused(bs, kw):
    c = Case(bs, "ragged", "off")
    if "prefix" in kw:
        kw = dict(prefix=torch.zeros(c.B, dtype=torch.int32, device="cuda"))  # without causal
    with pytest.raises(bs.BsattnError) as e:
        _mod_calls(bs, c, bs.ScoreMod(**kw))
    assert e.value.code == 1


def test_bad_tensors_and_workspaces_are_refused(bs):
    c = Case(bs, "ragged", "docs")
    for mod in (bs.ScoreMod(slopes=torch.zeros(c.heads + 1, device="cuda")),
                bs.ScoreMod(slopes=torch.zeros(c.heads, dtype=torch.float64, device="cuda")),
                bs.ScoreMod(doc=torch.zeros((c.B, c.L + 1), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            _mod_calls(bs, c, mod)
    with pytest.raises(bs.BsattnError) as e:
        _mod_calls(bs, c, c.mod, ws=None)  # documents need the workspace
    assert e.value.code == 6
    _mod_calls(bs, c, bs.ScoreMod(softcap=3.0), ws=None)
    mod = bs.ScoreMod(softcap=3.0)
    q, k, v = _tiled(bs, c.plan, c.q, c.k, c.v)
    lse = torch.zeros(c.plan.tiled_shape()[:-1], device="cuda")
    back = lambda plan, mod, ws, **kw: bs.attn_backward_mod(plan, mod, q, k, v, v, v, lse, c.idx, c.cnt, q, k, v, ws, **kw)  # noqa: E731
    with pytest.raises(bs.BsattnError) as e:
        back(c.plan, mod, c.plan.workspace("backward")[:1024])
    assert e.value.code == 6
    with pytest.raises(bs.BsattnError) as e:
        back(c.plan, mod, c.plan.workspace("mod_backward"), d_slopes=torch.zeros(c.heads, device="cuda"))
    assert e.value.code == 1  # no slopes to differentiate
    f8 = Case(bs, "ragged", "off", fp8=True)
    with pytest.raises(bs.BsattnError) as e:
        back(f8.plan, mod, f8.plan.workspace("mod_backward"))
    assert e.value.code == 2
    lib, raw = bs._lib, ctypes.byref(mod.raw)
    p = ctypes.c_void_p(q.data_ptr())
    assert lib.attn_forward_mod(c.plan.handle, None, p, p, None, None, p, p, p, p, None, None, 0, None) == 1
    assert lib.attn_forward_mod(c.plan.handle, raw, p, p, None, None, None, p, p, p, None, None, 0, None) == 1
