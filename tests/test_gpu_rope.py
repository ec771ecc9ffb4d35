"""Rotary positions: attn_rope against the fp64 oracle.

Tolerances. The rotated value x c - y s is formed in fp32 from bf16 inputs:
sine and cosine carry at most about 2^-22 (argument rounded in turns, then two
units of the function), the products and the sum three roundings of 2^-24, so
the value is within 2^-20 (|x| + |y|) amplitude; the bf16 rounding adds half a
step, 2^-8 of the value. A mean of n values adds n roundings of 2^-24 of their
mean magnitude."""
import numpy as np
import pytest
import torch

from oracle import rope, tiling
from tests.helpers import to64

pytestmark = pytest.mark.gpu

GRIDS = {  # B, heads, D, (T, H, W), tile
    "token": (1, 1, 64, (1, 1, 1), (4, 4, 4)),
    "token40": (3, 40, 128, (1, 1, 1), (4, 4, 4)),
    "ragged": (2, 3, 128, (5, 6, 7), (4, 4, 4)),
    "tile688": (1, 2, 64, (7, 9, 10), (6, 8, 8)),
    "tile344": (1, 2, 128, (5, 6, 7), (3, 4, 4)),
    "sequence": (2, 5, 64, (131, 1, 1), (64, 1, 1)),
    "wide": (1, 17, 64, (1, 3, 200), (1, 1, 128)),
}
ROPES = [
    dict(dims=(44, 42, 42), layout="interleaved"),
    dict(dims=(44, 42, 42), layout="half"),
    dict(dims=(0, 64, 0), layout="half", scaling="ntk", factor=(1.0, 4.0, 1.0)),
    dict(dims=(6, 10, 2), layout="interleaved", offset=(1 << 30, 7, -5), scaling="linear", factor=(8.0, 2.0, 0.5)),
    dict(dims=(6, 10, 2), layout="half", amplitude=1.25),
    dict(dims=(16, 8, 8), layout="half", scaling="by_parts", factor=(4.0, 2.0, 2.0), original=(256.0, 64.0, 64.0)),
    dict(dims=(2, 0, 0), layout="half"),
]


@pytest.fixture(scope="module")
def bs():
    from block_sparse_attention_reorder_b200 import bsattn
    assert torch.cuda.is_available()
    return bsattn


def _draw(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def _want(x, kw, T, H, W, pos=None, transpose=False):
    kw = dict(kw)
    layout, amp, offset = kw.pop("layout"), kw.pop("amplitude", 1.0), kw.pop("offset", (0, 0, 0))
    f, axis = rope.frequencies(**kw)
    at = rope.grid_positions(T, H, W, offset) if pos is None else pos.astype(np.int64)
    y = rope.rotate(to64(x), at, f, axis, layout, amp, transpose)
    R = f.size
    mag = np.abs(to64(x))
    if layout == "half":
        mag[..., :R], mag[..., R:2 * R] = (mag[..., :R] + mag[..., R:2 * R],) * 2
    else:
        mag[..., 0:2 * R:2], mag[..., 1:2 * R:2] = (mag[..., 0:2 * R:2] + mag[..., 1:2 * R:2],) * 2
    return y, 2.0 ** -20 * mag * max(1.0, amp)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("r", range(len(ROPES)))
@pytest.mark.parametrize("grid", list(GRIDS))
def test_rope_against_oracle(bs, grid, r, transpose):
    B, heads, D, (T, H, W), tile = GRIDS[grid]
    kw = ROPES[r]
    if sum(kw["dims"]) > D:
        pytest.skip("more features than the head has")
    plan = bs.Plan(B, heads, D, T, H, W, rule="window", tile=tile)
    x = [_draw(plan.natural_shape(), 10 * r + i) for i in range(2)]
    out = [torch.full(plan.natural_shape(), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bs.attn_rope(plan, bs.Rope(**kw), x[0].cuda(), out[0], x[1].cuda(), out[1], transpose=transpose)
    for a, b in zip(x, out):
        y, tol = _want(a, kw, T, H, W, transpose=transpose)
        err = np.abs(to64(b) - y)
        assert np.all(err <= 2.0 ** -8 * np.abs(y) + tol), (err.max(), (err - 2.0 ** -8 * np.abs(y)).max())


@pytest.mark.parametrize("r", [0, 1, 3, 4, 5])
@pytest.mark.parametrize("grid", ["token40", "ragged", "tile688", "tile344", "sequence"])
def test_tile_means(bs, grid, r):
    B, heads, D, (T, H, W), tile = GRIDS[grid]
    kw = ROPES[r]
    if sum(kw["dims"]) > D:
        pytest.skip("more features than the head has")
    plan = bs.Plan(B, heads, D, T, H, W, rule="window", tile=tile)
    x = [_draw(plan.natural_shape(), 50 + i) for i in range(2)]
    shape = (B, heads, plan.N, D)
    for both in (True, False):  # means of one tensor only take another launch
        y = [torch.empty(plan.natural_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        z = [torch.empty_like(t) for t in y]
        means = [torch.full(shape, float("nan"), device="cuda") for _ in range(2)]
        bs.attn_rope(plan, bs.Rope(**kw), x[0].cuda(), y[0], x[1].cuda(), y[1], pooled0=means[0],
                     pooled1=means[1] if both else None)
        bs.attn_rope(plan, bs.Rope(**kw), x[0].cuda(), z[0], x[1].cuda(), z[1])
        for i in range(2 if both else 1):
            assert torch.equal(y[i], z[i])  # the rotation does not depend on the means
            want, tol = _want(x[i], kw, T, H, W)
            n = plan.V
            mag = tiling.pool_mean(np.abs(want), T, H, W, tile)
            bound = tiling.pool_mean(tol, T, H, W, tile) + (n + 2) * 2.0 ** -24 * mag
            assert np.all(np.abs(to64(means[i]) - tiling.pool_mean(want, T, H, W, tile)) <= bound)
        if not both:
            assert torch.isnan(means[1]).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("grid", ["ragged", "tile344", "sequence"])
def test_explicit_positions_in_place_and_one_tensor(bs, grid, layout):
    B, heads, D, (T, H, W), tile = GRIDS[grid]
    plan = bs.Plan(B, heads, D, T, H, W, rule="window", tile=tile)
    g = np.random.default_rng(5)
    pos = g.integers(-2 ** 31, 2 ** 31, (B, plan.L, 3)).astype(np.int32)
    kw = dict(dims=(20, 12, 10), layout=layout)
    x = _draw(plan.natural_shape(), 6)
    t = x.cuda()
    bs.attn_rope(plan, bs.Rope(pos=torch.from_numpy(pos).cuda(), **kw), t, t)
    y, tol = _want(x, kw, T, H, W, pos=pos)
    assert np.all(np.abs(to64(t) - y) <= 2.0 ** -8 * np.abs(y) + tol)


def test_own_stream_and_graph(bs):
    plan = bs.Plan(1, 12, 128, 16, 28, 52, rule="topk", k=46)
    r = bs.Rope(dims=(44, 42, 42))
    x = [_draw(plan.natural_shape(), 7 + i).cuda() for i in range(2)]
    want = torch.empty_like(x[0])
    bs.attn_rope(plan, r, x[0], want)
    side, y = torch.cuda.Stream(), torch.empty_like(x[0])
    side.wait_stream(torch.cuda.current_stream())
    bs.attn_rope(plan, r, x[0], y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    src = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.attn_rope(plan, r, src, y)
    src.copy_(x[1])
    graph.replay()
    bs.attn_rope(plan, r, x[1], want)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("kw", [
    dict(dims=(44, 42, 44)), dict(dims=(0, 0, 0)), dict(dims=(3, 1, 0)), dict(dims=(-2, 4, 2)), dict(dims=(8, 8, 8), base=1.0),
    dict(dims=(8, 8, 8), base=float("inf")), dict(dims=(8, 8, 8), layout=2), dict(dims=(8, 8, 8), scaling=4),
    dict(dims=(8, 8, 8), scaling="linear", factor=(1.0, 0.0, 1.0)), dict(dims=(8, 8, 8), scaling="by_parts"),
    dict(dims=(8, 8, 8), scaling="by_parts", original=(9.0, 9.0, 9.0), slow=4.0, fast=4.0),
    dict(dims=(8, 8, 8), scaling="by_parts", original=(9.0, 0.0, 9.0)), dict(dims=(8, 8, 8), amplitude=float("nan")),
])
def test_bad_descriptions_are_refused(bs, kw):
    plan = bs.Plan(1, 1, 128, 2, 2, 2, rule="window")
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    kw = dict(kw)
    if kw.get("scaling") == "by_parts" and "original" not in kw:
        kw["original"] = (-1.0, 1.0, 1.0)
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_rope(plan, bs.Rope(**kw), x, x)
    assert e.value.code == 1


@pytest.mark.parametrize("kw", [
    dict(dims=(8, 8, 8), scaling="ntk", factor=(1.0, 1e300, 1.0)), dict(dims=(8, 8, 8), amplitude=1e39),
    dict(dims=(8, 8, 8), scaling="linear", factor=(1e-310, 1.0, 1.0)),
    dict(dims=(8, 8, 8), scaling="by_parts", original=(9.0, 9.0, 9.0), slow=4.0, fast=8.0, factor=(1.0, 1.0, 1e-310)),
])
def test_frequencies_without_a_value_are_refused(bs, kw):
    plan = bs.Plan(1, 1, 128, 2, 2, 2, rule="window")
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_rope(plan, bs.Rope(**kw), x, x)
    assert e.value.code == 1
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_layer_mod(plan, bs.Rope(**kw), None, x, x, x, torch.empty_like(x), plan.workspace("mod_layer"))
    assert e.value.code == 1


def test_bad_tensors_are_refused(bs):
    plan = bs.Plan(1, 1, 64, 2, 2, 2, rule="window")
    x = torch.zeros(plan.natural_shape(), dtype=torch.bfloat16, device="cuda")
    r = bs.Rope(dims=(8, 0, 0))
    means = torch.zeros((1, 1, 1, 64), device="cuda")
    for bad in (x.float(), x[:, :4], x.cpu()):
        with pytest.raises(ValueError):
            bs.attn_rope(plan, r, x, bad)
    for kw in (dict(x1=x), dict(y1=x), dict(pooled1=means)):
        with pytest.raises(bs.BsattnError) as e:
            bs.attn_rope(plan, r, x, x, **kw)
        assert e.value.code == 1
    pos = torch.zeros((1, 4, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        bs.attn_rope(plan, bs.Rope(dims=(8, 0, 0), pos=pos), x, x)
    raw = torch.zeros(64 * 8 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 64 * 8].view(plan.natural_shape())
    with pytest.raises(bs.BsattnError) as e:
        bs.attn_rope(plan, r, raw, x)
    assert e.value.code == 1
