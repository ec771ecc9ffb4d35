"""Pins of the rotary and score-rule oracles (CPU only)."""
import numpy as np
import pytest

from oracle import attention, rope, rules


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dims", [(4, 2, 2), (2, 0, 4)])
def test_rotated_products_depend_on_the_difference_of_positions(layout, dims):
    g = np.random.default_rng(1)
    x, y = g.standard_normal((2, 1, 1, 1, 10))
    f, axis = rope.frequencies(dims)
    p, q, s = g.integers(-50, 50, (3, 1, 3))
    at = lambda v, pos: rope.rotate(v, pos, f, axis, layout)[0, 0, 0]  # noqa: E731
    assert at(x, p) @ at(y, q) == pytest.approx(at(x, p + s) @ at(y, q + s), abs=1e-12)
    np.testing.assert_array_equal(at(x, p)[sum(dims):], x[0, 0, 0, sum(dims):])


def test_first_pair_turns_by_the_position_itself():
    f, axis = rope.frequencies((2, 0, 0))
    x = np.zeros((1, 1, 1, 4))
    x[..., 0] = 1.0
    got = rope.rotate(x, np.array([[3, 0, 0]]), f, axis)[0, 0, 0]
    np.testing.assert_allclose(got, [np.cos(3), np.sin(3), 0, 0], atol=1e-15)


def test_scalings():
    dims, s = (8, 0, 0), (4.0, 1.0, 1.0)
    f0, _ = rope.frequencies(dims)
    np.testing.assert_allclose(rope.frequencies(dims, scaling="linear", factor=s)[0], f0 / 4)
    ntk = rope.frequencies(dims, scaling="ntk", factor=s)[0]
    assert ntk[0] == f0[0] and ntk[-1] == pytest.approx(f0[-1] / 4)  # the ends: kept, interpolated
    parts = rope.frequencies(dims, scaling="by_parts", factor=s, original=(2000.0, 1, 1), slow=1.0, fast=32.0)[0]
    assert parts[0] == f0[0] and parts[-1] == pytest.approx(f0[-1] / 4)
    assert np.all((parts <= f0) & (parts >= f0 / 4))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_transpose_is_the_gradient(layout):
    g = np.random.default_rng(2)
    x, up = g.standard_normal((2, 1, 3, 1, 8))
    f, axis = rope.frequencies((2, 2, 2))
    pos = g.integers(0, 9, (3, 3))
    grad = rope.rotate(up, pos, f, axis, layout, 1.3, transpose=True)
    for at in [(0, 0, 0, 0), (0, 1, 0, 3), (0, 2, 0, 5), (0, 2, 0, 7)]:
        d = np.zeros_like(x)
        d[at] = 1e-4
        diff = ((rope.rotate(x + d, pos, f, axis, layout, 1.3) - rope.rotate(x - d, pos, f, axis, layout, 1.3)) * up).sum()
        assert grad[at] == pytest.approx(diff / 2e-4, abs=1e-9)


def _case(seed=3):
    g = np.random.default_rng(seed)
    xyz = rope.grid_positions(3, 2, 2)
    n = len(xyz)
    q, k, v, do = g.standard_normal((4, n, 4))
    doc = np.array([0] * 5 + [1] * 5 + [-1] * 2)
    seen = rules.visible(xyz, xyz, True, 1, doc, doc) & (g.random((n, n)) < 0.8)
    return xyz, q, k, v, do, doc, seen, rules.distance(xyz, xyz, (1.0, 0.5, 0.25))


def test_rules_off_is_masked_attention():
    _, q, k, v, _, _, seen, _ = _case()
    o, lse = attention.dense_masked(q, k, v, seen, 0.5)
    r = rules.attend(q, k, v, seen, 0.5)
    np.testing.assert_allclose(r["o"], o, atol=1e-14)
    np.testing.assert_allclose(r["lse"], lse, atol=1e-14)


def test_rules_against_a_loop():
    xyz, q, k, v, _, doc, _, far = _case()
    cap, slope, pre = 2.0, 0.3, 1
    r = rules.attend(q, k, v, rules.visible(xyz, xyz, True, pre, doc, doc), 0.5, cap, slope, far)
    for i in range(len(q)):
        w = np.zeros(len(k))
        for j in range(len(k)):
            ti, tj = xyz[i][0], xyz[j][0]
            if doc[i] != doc[j] or doc[j] < 0 or not (tj <= ti or tj < pre):
                continue
            d = abs(xyz[i][0] - xyz[j][0]) + 0.5 * abs(xyz[i][1] - xyz[j][1]) + 0.25 * abs(xyz[i][2] - xyz[j][2])
            w[j] = np.exp(cap * np.tanh(0.5 * (q[i] @ k[j]) / cap) - slope * d)
        if w.sum() == 0:
            assert np.all(r["o"][i] == 0) and r["lse"][i] == -np.inf
        else:
            np.testing.assert_allclose(r["o"][i], (w / w.sum()) @ v, atol=1e-12)
            assert r["lse"][i] == pytest.approx(np.log(w.sum()), abs=1e-12)


def test_gradients_against_central_differences():
    _, q, k, v, do, _, seen, far = _case()
    args = dict(scale=0.5, cap=2.0, far=far)
    r = rules.attend(q, k, v, seen, slope=0.3, do=do, **args)
    loss = lambda q, k, v, s: (rules.attend(q, k, v, seen, slope=s, **args)["o"] * do).sum()  # noqa: E731
    h = 1e-5
    for name, which in (("dq", 0), ("dk", 1), ("dv", 2)):
        for at in [(0, 0), (4, 2), (7, 1), (11, 3)]:
            lo, hi = [q.copy(), k.copy(), v.copy()], [q.copy(), k.copy(), v.copy()]
            lo[which][at] -= h
            hi[which][at] += h
            assert r[name][at] == pytest.approx((loss(*hi, 0.3) - loss(*lo, 0.3)) / (2 * h), abs=1e-8)
    assert r["dslope"] == pytest.approx((loss(q, k, v, 0.3 + h) - loss(q, k, v, 0.3 - h)) / (2 * h), abs=1e-8)


def test_hidden_tile_pairs_hide_every_token_pair():
    """Pairs set to the lowest value have no visible token pair; with ids that do not decrease, no others have none."""
    T, H, W = 6, 2, 3
    xyz = rope.grid_positions(T, H, W)
    tiles = [np.nonzero(xyz[:, 0] // 2 == t)[0] for t in range(3)]
    g = np.random.default_rng(4)
    doc = np.sort(g.integers(0, 4, T * H * W))
    out = rules.scores(np.zeros((1, 1, 3, 3)), [xyz[t] for t in tiles], causal=True, prefix=[1],
                       docs=[[doc[t] for t in tiles]])
    ok = rules.visible(xyz, xyz, True, 1, doc, doc)
    by_doc = rules.visible(xyz, xyz, doc_q=doc, doc_k=doc)
    by_time = rules.visible(xyz, xyz, True, 1)
    for i in range(3):
        for j in range(3):
            pair = np.ix_(tiles[i], tiles[j])
            if out[0, 0, i, j] == rules.LOWEST:
                assert not ok[pair].any()
            else:
                assert by_doc[pair].any() and by_time[pair].any()
