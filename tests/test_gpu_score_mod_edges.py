"""Attention under score rules at its edges: references that move within a
step, rows that are not numbers, refusals, which come before any work, and
tensors of a description exchanged between calls."""
import math

import numpy as np
import pytest
import torch

from oracle import rules
from tests.helpers import to64
from tests.test_gpu_score_mod import Case, _nan, _tiled, bs  # noqa: F401  (bs: fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- references that move within a step

# Score levels of the first steps of the first query block's walk, for keys 0-31 and 32-63 of a step. A row's
# reference moves when a half's maximum is 70 powers of two (48.5) above the one that set it.
MOVES = {  # levels of the steps, moves in the (first, second) half
    "first": ([(-55, -55), (0, 0), (55, 55)], [(0, 0), (1, 0), (1, 0)]),
    "second": ([(-55, -55), (-55, 0), (0, 55)], [(0, 0), (0, 1), (0, 1)]),
    "both": ([(-55, -55), (0, 55)], [(0, 0), (1, 1)]),
    "at_once": ([(-55, 0), (55, 0)], [(0, 1), (1, 0)]),
}


def _moves(z):
    """Which halves of 32 scores (natural units, in the order of the walk) move a row's reference."""
    ref, out = -math.inf, []
    for half in z.reshape(-1, 32):
        top = half.max() / math.log(2.0)
        move = top > ref + 30.0
        out.append(int(move and ref > -math.inf))
        ref = top + 40.0 if move else ref
    return [tuple(x) for x in np.array(out).reshape(-1, 2).tolist()]


@pytest.mark.parametrize("moves", list(MOVES))
@pytest.mark.parametrize("grid", ["seq400", "seq300_wide"])  # D = 128 and 64
def test_references_that_move_within_a_step(bs, grid, moves):  # noqa: F811
    """Cap and bias together take a step in two halves; what the first half stored is scaled by the second. The
    scales are powers below 2^-70: a P or an O that missed one would outweigh all the rest."""
    levels, want = MOVES[moves]
    c = Case(bs, grid, "cap", seed=20)
    plan, (T, _, _) = c.plan, c.grid
    c.cap, c.slopes = 60.0, np.full(c.heads, 2.0 ** -10, np.float32)
    c.mod = bs.ScoreMod(softcap=c.cap, slopes=torch.from_numpy(c.slopes).cuda(), dist=(1.0, 0.5, 0.0))
    # The first block's walk: its own tile's chunks from the last to the first, then the others ascending.
    per, chunks = c.tile[0] // 64, -(-T // 64)
    walk = [*range(per)][::-1] + [*range(per, chunks)]
    g = np.random.default_rng(23)
    level = g.choice([-55.0, 0.0, 55.0], (chunks, 2))
    level[walk[:len(levels)]] = levels
    level = level.reshape(-1).repeat(32)[:T]
    u = np.where(g.random(c.D) < 0.5, -1.0, 1.0)
    k = (c.cap * np.arctanh(level / c.cap) / math.sqrt(c.D))[:, None] * u + 0.02 * g.standard_normal((T, c.D))
    draw = lambda x: torch.from_numpy(np.broadcast_to(x[None, :, None], plan.natural_shape()).copy()).to(torch.bfloat16)  # noqa: E731
    c.q, c.k = draw(u + 0.01 * g.standard_normal((T, c.D))), draw(k)
    z = c.cap * np.tanh(c.D ** -0.5 * to64(c.q)[0, 0, 0] @ to64(c.k)[0, :, 0].T / c.cap)
    z = z - 2.0 ** -10 * rules.distance(c.xyz[:1], c.xyz, (1.0, 0.5, 0.0))[0]
    steps = np.concatenate([z[64 * n:64 * n + 64] for n in walk if 64 * n + 64 <= T])
    assert _moves(steps)[:len(want)] == want
    for ws in (None, plan.workspace("mod_forward")):
        o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
        bs.attn_forward_natural_mod(plan, c.mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse)
        assert bs.attn_check_device_status(plan) == 0
        c.check_forward(to64(o), to64(lse), *(to64(x) for x in (c.q, c.k, c.v)))
        ot = _nan(plan.tiled_shape())
        bs.attn_forward_mod(plan, c.mod, *_tiled(bs, plan, c.q, c.k, c.v), c.idx, c.cnt, ot, ws)
        back = torch.empty_like(o)
        bs.attn_unreorder(plan, ot, back)
        assert torch.equal(back, o)


# ---------------------------------------------------------------- rows that are not numbers

@pytest.mark.parametrize("rule", ["cap", "bias", "all"])
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("grid", ["ragged", "seq400"])
def test_a_visible_row_that_is_not_a_number(bs, grid, shared, rule):  # noqa: F811
    """NaN in a visible query row: O, lse and dQ of that row are NaN, whether CTAs share its block or not; its
    lse is not the -inf of a row that sees no key. Other rows of O and dQ are what they are without it."""
    c = Case(bs, grid, rule, seed=21)
    plan, ws = c.plan, c.plan.workspace("mod_forward") if shared or c.doc is not None else None
    # The first token of the last batch that sees a key.
    b, h = c.B - 1, c.heads - 1
    r = c.oracle(b, h, *(to64(x)[b, :, h] for x in (c.q, c.k, c.v)))
    row = int((~(r["lse"] == -float("inf"))).nonzero()[0][0])
    bad = c.q.clone()
    bad[b, row, h, 5] = float("nan")
    res = []
    for q0 in (c.q, bad):
        o, lse = _nan(plan.natural_shape()), _nan((c.B, c.heads, c.L), torch.float32)
        bs.attn_forward_natural_mod(plan, c.mod, q0.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o, ws, lse_nat=lse)
        q, k, v, do = _tiled(bs, plan, q0, c.k, c.v, c.do)
        ot, lt = _nan(plan.tiled_shape()), _nan(plan.tiled_shape()[:-1], torch.float32)
        bs.attn_forward_mod(plan, c.mod, q, k, v, c.idx, c.cnt, ot, ws, lse=lt)
        grads = [_nan(plan.tiled_shape()) for _ in range(3)]
        bs.attn_backward_mod(plan, c.mod, q, k, v, ot, do, lt, c.idx, c.cnt, *grads, plan.workspace("mod_backward"))
        assert bs.attn_check_device_status(plan) == 0
        dq = torch.empty_like(o)
        bs.attn_unreorder(plan, grads[0], dq)
        res.append((o, dq, lse))
    (o0, dq0, lse0), (o1, dq1, lse1) = res
    assert torch.isnan(o1[b, row, h]).all() and torch.isnan(dq1[b, row, h]).all() and torch.isnan(lse1[b, h, row])
    for x, y in ((o0, o1), (dq0, dq1)):
        y[b, row, h] = x[b, row, h]
        assert torch.equal(x, y)
    lse1[b, h, row] = lse0[b, h, row]
    assert torch.equal(lse0, lse1)


# ---------------------------------------------------------------- refusals come before any work

def _marked(nbytes):
    return torch.full((int(nbytes),), 0xA5, dtype=torch.uint8, device="cuda")


def _docs(plan):
    return torch.zeros((plan.B, plan.L), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rule", ["topk", "window"])
def test_refused_frequencies_leave_everything_as_it_was(bs, rule):  # noqa: F811
    plan = bs.Plan(1, 2, 128, 4, 8, 8, rule=rule, k=2, win=(1, 1, 1))
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    o, ws = _nan(plan.natural_shape()), _marked(plan.mod_info.layer_workspace_bytes)
    r = bs.Rope(dims=(8, 8, 8), scaling="ntk", factor=(1.0, 1e300, 1.0))
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_layer_mod(plan, r, bs.ScoreMod(softcap=5.0, doc=_docs(plan)), x, x, x, o, ws)
    assert e.value.code == 1
    assert torch.isnan(o).all() and torch.all(ws == 0xA5)


BIG = {  # heads, D, grid, tile, window
    "tiles": (1, 64, (32769, 1, 1), (1, 1, 1), (0, 0, 0)),      # more than 32768 tiles
    "list": (1, 128, (1, 1033, 1), (1, 8, 1024), (0, 129, 0)),  # 16,640 steps of one block
}


@pytest.mark.parametrize("big", list(BIG))
@pytest.mark.parametrize("call", ["forward", "forward_natural", "layer", "layer_no_rules"])
def test_plans_too_large_for_the_forward(bs, big, call):  # noqa: F811
    heads, D, grid, tile, win = BIG[big]
    plan = bs.Plan(1, heads, D, *grid, rule="window", win=win, tile=tile)
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    o = _nan(plan.natural_shape())
    mod = bs.ScoreMod(softcap=5.0, doc=_docs(plan))
    layer = call.startswith("layer")
    ws = _marked(plan.mod_info.layer_workspace_bytes if layer else plan.mod_info.forward_workspace_bytes)
    si, sc = plan.list_shapes()
    idx, cnt = torch.zeros(si, dtype=torch.int32, device="cuda"), torch.zeros(sc, dtype=torch.int32, device="cuda")
    with pytest.raises(bs.BsattnError) as e:
        if layer:
            bs.attn_layer_mod(plan, bs.Rope(dims=(8, 8, 8)), mod if call == "layer" else None, x, x, x, o, ws)
        elif call == "forward_natural":
            bs.attn_forward_natural_mod(plan, mod, x, x, x, idx, cnt, o, ws)
        else:
            x = torch.empty(plan.tiled_shape(), dtype=torch.bfloat16, device="cuda")
            o = _nan(plan.tiled_shape())
            bs.attn_forward_mod(plan, mod, x, x, x, idx, cnt, o, ws)
    assert e.value.code == 2
    assert torch.isnan(o).all() and torch.all(ws == 0xA5)


def test_plans_too_large_for_the_backward(bs):  # noqa: F811
    """The dQ pass has room for its lists (128 steps), the dK, dV pass does not (8,192)."""
    plan = bs.Plan(1, 1, 128, 1, 505, 1, rule="window", win=(0, 0, 0), tile=(1, 8, 1024))
    x = torch.zeros(plan.tiled_shape(), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(plan.tiled_shape()[:-1], device="cuda")
    idx = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 1, 64, 1)
    cnt = torch.ones((1, 1, 64), dtype=torch.int32, device="cuda")
    grads = [_nan(plan.tiled_shape()) for _ in range(3)]
    ws = _marked(plan.mod_info.backward_workspace_bytes)
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_backward_mod(plan, bs.ScoreMod(softcap=5.0, doc=_docs(plan)), x, x, x, x, x, lse, idx, cnt, *grads, ws)
    assert e.value.code == 2
    assert all(torch.isnan(t).all() for t in grads) and torch.all(ws == 0xA5)


def test_more_heads_than_the_rules_on_scores_take(bs):  # noqa: F811
    plan = bs.Plan(300, 220, 64, 1, 1, 1, rule="topk", k=1)
    s = torch.zeros((plan.B, plan.heads, 1, 1), device="cuda")
    ws = _marked(plan.mod_info.scores_workspace_bytes)
    mod = bs.ScoreMod(softcap=5.0, doc=_docs(plan))
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_mod_scores(plan, mod, s, s, ws)
    assert e.value.code == 2 and torch.all(ws == 0xA5)
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    o, ws = _nan(plan.natural_shape()), _marked(plan.mod_info.layer_workspace_bytes)
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_layer_mod(plan, None, mod, x, x, x, o, ws)
    assert e.value.code == 2 and torch.isnan(o).all() and torch.all(ws == 0xA5)


# ---------------------------------------------------------------- tensors exchanged after construction

def test_exchanged_tensors_are_used(bs):  # noqa: F811
    c = Case(bs, "ragged", "all", seed=22)
    plan, ws = c.plan, c.plan.workspace("mod_forward")

    def run(mod):
        o = _nan(plan.natural_shape())
        bs.attn_forward_natural_mod(plan, mod, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.idx, c.cnt, o, ws)
        return o

    old = [torch.zeros_like(t) for t in (c.mod.slopes, c.mod.prefix, c.mod.doc)]
    mod = bs.ScoreMod(softcap=c.cap, slopes=old[0], dist=(1.0, 0.5, 0.0), causal=True, prefix=old[1], doc=old[2])
    first = run(mod)
    mod.slopes, mod.prefix, mod.doc = c.mod.slopes, c.mod.prefix, c.mod.doc
    want = run(c.mod)
    assert torch.equal(run(mod), want) and not torch.equal(first, want)
    mod.slopes = mod.prefix = mod.doc = None
    assert torch.equal(run(mod), run(bs.ScoreMod(softcap=c.cap, causal=True)))
    with pytest.raises(ValueError):
        mod.doc = c.mod.doc.cpu()
    pos = torch.randint(-1000, 1000, (2, plan.B, plan.L, 3), device="cuda").to(torch.int32)
    r, y = bs.Rope(dims=(8, 8, 8), pos=pos[0].clone()), [_nan(plan.natural_shape()) for _ in range(2)]
    r.pos = pos[1]
    bs.attn_rope(plan, r, c.q.cuda(), y[0])
    bs.attn_rope(plan, bs.Rope(dims=(8, 8, 8), pos=pos[1]), c.q.cuda(), y[1])
    assert torch.equal(y[0], y[1])
