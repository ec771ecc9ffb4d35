"""Rotary positions, and block-sparse attention whose scores are capped, biased
by distance and masked by document and prefix: measured cases.

`run` computes each operator in elementary torch operations, or, with `own`
set, by the framework's entry points. Kinds of case (`"op"`):

rope    Q and K of one layer rotated by their grid positions, with the tile
        means of the result; or the gradient of that (`"transpose"`).
scores  the block scores of a layer under the layer's cap, bias and masks.
attend  attention over kept tile pairs with cap, bias and masks.
train   the same on tiled tensors, forward and backward.
layer   rotation, tile window and attention in one call.
"""
import math

import numpy as np
import torch

own = False

LOWEST = torch.finfo(torch.float32).min
LOG2E = 1.4426950408889634


def _case(name, op, grid, heads, D, B=1, tile=(4, 4, 4), topk=0, win=None, cap=0.0, bias=False, causal=False, docs=0,
          hidden=False, half=False, dims=(0, 0, 0), scaling="none", positions=False, transpose=False, pooled=False, fp8=False):
    c = {"op": op, "B": B, "heads": heads, "D": D, "T": grid[0], "H": grid[1], "W": grid[2], "tile_t": tile[0],
         "tile_h": tile[1], "tile_w": tile[2], "topk": topk, "win_t": -1, "win_h": -1, "win_w": -1, "cap": cap,
         "bias": bias, "causal": causal, "docs": docs, "hidden": hidden, "half": half, "dim_t": dims[0],
         "dim_h": dims[1], "dim_w": dims[2], "scaling": scaling, "positions": positions, "transpose": transpose,
         "pooled": pooled, "fp8": fp8}
    if win is not None:
        c["win_t"], c["win_h"], c["win_w"] = win
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One new token of a 40-head layer at a far position: the smallest call, all latency.
        _case("rope_one_token", "rope", (1, 1, 1), 40, 128, dims=(44, 42, 42)),
        # Q and K of the Wan-1.3B-shaped layer, with the tile means that its routing reads.
        _case("rope_wan1.3b", "rope", (16, 28, 52), 12, 128, dims=(44, 42, 42), pooled=True),
        # The gradient through the rotation at the Wan-14B size: half layout, part of the head, longer clips.
        _case("rope_wan14b_gradient", "rope", (21, 45, 80), 40, 128, half=True, dims=(32, 24, 24), scaling="by_parts",
              transpose=True),
        # Routing of a two-head toy layer: latency.
        _case("scores_tiny", "scores", (8, 16, 16), 2, 64, cap=20.0, causal=True),
        # Routing of the Wan-14B layer over three packed clips, each causal in time.
        _case("scores_wan14b", "scores", (21, 45, 80), 40, 128, cap=30.0, bias=True, causal=True, docs=3),
        # A packed token sequence (a grid of one column), causal within each of eleven documents, some padding behind.
        _case("attend_packed", "attend", (16384, 1, 1), 8, 128, tile=(64, 1, 1), win=(255, 0, 0), causal=True, docs=11,
              hidden=True),
        # The e4m3 tile-window layer's attention (480p grid) with capped scores and a bias for near tokens.
        _case("attend_window_fp8", "attend", (21, 30, 52), 12, 128, win=(1, 1, 0), cap=30.0, bias=True, fp8=True),
        # Frame-causal attention with a visible prefix, Wan-14B shape in the 384-token tiles.
        _case("attend_wan14b_t688", "attend", (21, 45, 80), 40, 128, tile=(6, 8, 8), topk=24, cap=50.0, causal=True),
        # A training step on a small ragged batch with documents and hidden tokens.
        _case("train_ragged", "train", (7, 10, 13), 3, 128, B=2, topk=5, cap=15.0, bias=True, causal=True, docs=2,
              hidden=True),
        # A training step of the Wan-1.3B-shaped layer with cap and bias.
        _case("train_wan1.3b", "train", (16, 28, 52), 12, 128, topk=46, cap=30.0, bias=True),
        # The toy layer with every rule on: latency of the whole call.
        _case("layer_tiny", "layer", (8, 16, 16), 2, 64, win=(1, 1, 1), cap=20.0, bias=True, causal=True, docs=2,
              dims=(24, 20, 20), positions=True),
        # Rotation, a (3,3,1) tile window and frame-causal capped attention in one call, 480p grid.
        _case("layer_window", "layer", (21, 30, 52), 12, 128, win=(1, 1, 0), cap=30.0, causal=True, dims=(44, 42, 42)),
    ]


def draw(rng):
    op = rng.choice(["rope", "scores", "attend", "attend", "train", "layer"])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    D = rng.choice([64, 128])
    heads, B = log(1, 16), rng.choice([1, 1, 2])
    kw = dict(cap=rng.choice([0.0, rng.uniform(8.0, 60.0)]), bias=rng.random() < 0.5, causal=rng.random() < 0.5,
              docs=rng.choice([0, 0, log(1, 12)]))
    kw["hidden"] = kw["docs"] > 0 and rng.random() < 0.5
    if not (kw["cap"] or kw["bias"] or kw["causal"] or kw["docs"]):
        kw["cap"] = 30.0
    grid, tile = (log(1, 24), log(3, 44), log(3, 60)), rng.choice([(4, 4, 4), (4, 4, 4), (6, 8, 8), (2, 4, 8), (3, 4, 4)])
    if rng.random() < 0.25:
        grid, tile = (log(1, 12000), 1, 1), (64, 1, 1)
    n = [-(-g // t) for g, t in zip(grid, tile)]
    N = n[0] * n[1] * n[2]
    if op in ("rope", "layer"):
        pairs = [rng.randrange(0, D // 6 + 1) for _ in range(3)]
        pairs[rng.randrange(3)] += 1
        kw.update(half=rng.random() < 0.5, dims=tuple(2 * p for p in pairs), positions=rng.random() < 0.3,
                  scaling=rng.choice(["none", "linear", "ntk", "by_parts"]))
    if op == "rope":
        kw.update(transpose=rng.random() < 0.3)
        kw["pooled"] = not kw["transpose"] and rng.random() < 0.5
        kw.update(cap=0.0, bias=False, causal=False, docs=0, hidden=False)
    elif op != "scores":
        if op == "layer" or rng.random() < 0.4:
            most = 2 if tile[0] < 6 else 1
            kw["win"] = (N - 1, 0, 0) if tile[0] == 64 else tuple(rng.randint(0, most) for _ in range(3))
        else:
            kw["topk"] = max(1, min(N, 64 if tile[0] < 6 else 24, int(N * rng.uniform(0.1, 0.6))))
        kw["fp8"] = op == "attend" and rng.random() < 0.3
    return _case("", op, grid, heads, D, B=B, tile=tile, **kw)


# ------------------------------------------------------------------ geometry

def _tiles(c):
    tile = (c["tile_t"], c["tile_h"], c["tile_w"])
    n = tuple(-(-g // t) for g, t in zip((c["T"], c["H"], c["W"]), tile))
    return tile, n, n[0] * n[1] * n[2], max(64, tile[0] * tile[1] * tile[2])


def _geometry(c, device):
    """Coordinates of every token, its tile and row, the token of every (tile, row) slot (L where there is none)."""
    (tt, th, tw), (nt, nh, nw), N, V = _tiles(c)
    n = torch.arange(c["T"] * c["H"] * c["W"], device=device)
    t, h, w = n // (c["H"] * c["W"]), n // c["W"] % c["H"], n % c["W"]
    tile = (t // tt * nh + h // th) * nw + w // tw
    row = (t % tt * th + h % th) * tw + w % tw
    slot = torch.full((N * V,), n.numel(), device=device)
    slot[tile * V + row] = n
    return {"coord": torch.stack((t, h, w), -1), "tile": tile, "place": tile * V + row, "slot": slot}


def _freqs(c):
    """Angle per unit of position for each pair, and the pair's axis, in 64 bits."""
    f, axis = [], []
    for a, (d, s) in enumerate(zip((c["dim_t"], c["dim_h"], c["dim_w"]), _FACTOR)):
        i = np.arange(d // 2, dtype=np.float64)
        base = 10000.0
        if c["scaling"] == "ntk" and d > 2:
            base = base * s ** (d / (d - 2.0))
        g = base ** (-2.0 * i / max(d, 1))
        if c["scaling"] == "linear":
            g = g / s
        elif c["scaling"] == "by_parts":
            keep = np.clip((_ORIGINAL[a] * g / (2 * np.pi) - _SLOW) / (_FAST - _SLOW), 0.0, 1.0)
            g = g * (keep + (1.0 - keep) / s)
        f.append(g)
        axis.append(np.full(d // 2, a))
    return np.concatenate(f), np.concatenate(axis).astype(np.int64)


_FACTOR, _ORIGINAL, _SLOW, _FAST = (4.0, 2.0, 2.0), (256.0, 64.0, 64.0), 1.0, 32.0
_OFFSET = (70001, 3, 5)  # a stream's window: far along time
_DIST = (1.0, 0.5, 0.25)


def _field(gen, c, rows):
    """Smooth latent-like features plus noise, natural layout, bf16."""
    T, H, W, B, heads, D = c["T"], c["H"], c["W"], c["B"], c["heads"], c["D"]
    low = torch.randn((B, heads * D, max(1, T // 3), max(1, H // 5), max(1, W // 5)), generator=gen, device="cuda")
    x = torch.nn.functional.interpolate(low, size=(T, H, W), mode="trilinear")
    x = x + 0.5 * torch.randn(x.shape, generator=gen, device="cuda")
    return x.mul_(rows).permute(0, 2, 3, 4, 1).reshape(B, T * H * W, heads, D).to(torch.bfloat16).contiguous()


def _to_tiles(x, slot):
    """Natural [B, L, heads, D] -> [B, heads, N * V, D], zeros where a slot holds no token."""
    x = torch.cat((x, torch.zeros_like(x[:, :1])), 1)
    return x[:, slot].transpose(1, 2)


def _lists(c, g, q, k):
    """Kept key tiles of every (batch, head, query tile): a tile window, or the k largest products of tile means."""
    (_, n, N, V), B, heads = _tiles(c), c["B"], c["heads"]
    if c["win_t"] >= 0:
        at = np.stack(np.unravel_index(np.arange(N), n), -1)
        win = np.array([c["win_t"], c["win_h"], c["win_w"]])
        keep = (np.abs(at[:, None] - at[None]) <= win).all(-1)
        cnt, kmax = keep.sum(1), int(np.prod(np.minimum(2 * win + 1, np.array(n))))
        idx = np.argsort(~keep, axis=1, kind="stable")[:, :kmax]
        idx = torch.from_numpy(idx.astype(np.int32)).cuda().expand(B, heads, N, kmax).contiguous()
        return idx, torch.from_numpy(cnt.astype(np.int32)).cuda().expand(B, heads, N).contiguous()
    mean = lambda x: _to_tiles(x, g["slot"]).reshape(B, heads, N, V, -1).float().mean(3)  # noqa: E731
    s = mean(q) @ mean(k).transpose(-1, -2)
    idx = s.topk(c["topk"], -1).indices.sort(-1).values.to(torch.int32).contiguous()
    return idx, torch.full((B, heads, N), c["topk"], dtype=torch.int32, device="cuda")


def _codes(c, g, x):
    """e4m3 codes of natural x in the tiled layout, and a scale per (batch, head, tile)."""
    _, _, N, V = _tiles(c)
    t = _to_tiles(x, g["slot"]).reshape(c["B"], c["heads"], N, V, c["D"]).float()
    scale = t.abs().amax((3, 4)) / 448.0
    scale = torch.where(scale > 0, scale, 1.0)
    codes = (t / scale[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).contiguous(), scale


def _decoded(codes, scale, dtype):
    """The values of e4m3 tile codes, [B, heads, N * V, D]."""
    return (codes.view(torch.float8_e4m3fn).to(dtype) * scale[..., None, None].to(dtype)).flatten(2, 3)


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)
    L, (tile, n, N, V) = c["T"] * c["H"] * c["W"], _tiles(c)
    s = {"case": c, "g": _geometry(c, "cuda")}
    cpu = np.random.RandomState(seed % (1 << 31))
    # The rules: slopes halving over the heads, a prefix of up to a third of the frames, documents cut at random frames.
    s["slopes"] = s["prefix"] = s["doc"] = None
    if c["bias"]:
        s["slopes"] = torch.tensor([2.0 ** (-6.0 * (h + 1) / c["heads"]) for h in range(c["heads"])], device="cuda")
    if c["causal"]:
        s["prefix"] = torch.from_numpy(cpu.randint(0, c["T"] // 3 + 1, c["B"]).astype(np.int32)).cuda()
    start = np.zeros((c["B"], L), np.int64)  # first frame of each token's document
    if c["docs"]:
        frame = np.arange(L) // (c["H"] * c["W"])
        doc = np.zeros((c["B"], L), np.int32)
        for b in range(c["B"]):
            cuts = np.sort(cpu.randint(0, c["T"] + 1, c["docs"] - 1))
            doc[b] = np.searchsorted(cuts, frame, side="right")
            start[b] = np.concatenate(([0], cuts))[doc[b]]
            if c["hidden"]:
                doc[b, L - cpu.randint(0, L // 8 + 1):] = -1
        s["doc"] = torch.from_numpy(doc).cuda()
    s["pos"] = None
    if c["positions"]:
        p = s["g"]["coord"].to(torch.int32).expand(c["B"], L, 3).clone()
        p[..., 0] -= torch.from_numpy(start).cuda().to(torch.int32)
        s["pos"] = p.contiguous()
    if c["op"] == "scores":
        s["S"] = 3.0 * torch.randn((c["B"], c["heads"], N, N), generator=gen, device="cuda")
    else:
        s["q"], s["k"] = _field(gen, c, 2.0), _field(gen, c, 1.0)
        if c["op"] != "rope":
            s["v"] = _field(gen, c, 1.0)
        if c["op"] != "rope":
            s["idx"], s["cnt"] = _lists(c, s["g"], s["q"], s["k"])
        if c["fp8"]:
            for x in ("q", "k"):
                s[x], s[x + "s"] = _codes(c, s["g"], s[x])
        if c["op"] == "train":
            do = torch.randn(s["q"].shape, generator=gen, device="cuda").to(torch.bfloat16)
            for name, x in (("q", s["q"]), ("k", s["k"]), ("v", s["v"]), ("do", do)):
                s[name] = _to_tiles(x, s["g"]["slot"]).reshape(c["B"], c["heads"], N, V, c["D"]).contiguous()
    if own:
        _own_prepare(s)
    return s


# ------------------------------------------------------------------ the framework's calls

def _own_prepare(s):
    from block_sparse_attention_reorder_b200 import bsattn
    c = s["case"]
    tile, n, N, V = _tiles(c)
    if c["win_t"] >= 0:
        rule = dict(rule="window", win=(c["win_t"], c["win_h"], c["win_w"]))
    else:
        rule = dict(rule="topk", k=c["topk"]) if c["topk"] else dict(rule="window", win=(0, 0, 0))
    plan = bsattn.Plan(c["B"], c["heads"], c["D"], c["T"], c["H"], c["W"], tile=tile, qk_fp8=c["fp8"], **rule)
    s["bsattn"], s["plan"] = bsattn, plan
    if c["op"] in ("rope", "layer"):
        s["rope"] = bsattn.Rope(dims=(c["dim_t"], c["dim_h"], c["dim_w"]), layout="half" if c["half"] else "interleaved",
                                scaling=c["scaling"], factor=_FACTOR, original=_ORIGINAL, slow=_SLOW, fast=_FAST,
                                offset=_OFFSET, pos=s["pos"])
    if c["op"] != "rope":
        s["mod"] = bsattn.ScoreMod(softcap=c["cap"], slopes=s["slopes"], dist=_DIST, causal=c["causal"],
                                   prefix=s["prefix"], doc=s["doc"])
    if c["op"] == "rope":
        s["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"])]
        if c["pooled"]:
            s["out"] += [torch.empty((c["B"], c["heads"], N, c["D"]), device="cuda") for _ in range(2)]
    elif c["op"] == "scores":
        s["out"], s["ws"] = torch.empty_like(s["S"]), plan.workspace("mod_scores")
    elif c["op"] == "train":
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:-1], device="cuda")
        s["grads"] = [torch.empty_like(s["q"]) for _ in range(3)]
        s["dslopes"] = torch.empty(c["heads"], device="cuda") if c["bias"] else None
        s["ws"], s["bws"] = plan.workspace("mod_forward"), plan.workspace("mod_backward")
    else:
        s["o"] = torch.empty_like(s["v"])
        s["lse"] = torch.empty((c["B"], c["heads"], s["v"].shape[1]), device="cuda")
        s["ws"] = plan.workspace("mod_forward" if c["op"] == "attend" else "mod_layer")


def _own_run(s):
    b, plan, c = s["bsattn"], s["plan"], s["case"]
    if c["op"] == "rope":
        o = s["out"]
        b.attn_rope(plan, s["rope"], s["q"], o[0], s["k"], o[1], pooled0=o[2] if c["pooled"] else None,
                    pooled1=o[3] if c["pooled"] else None, transpose=c["transpose"])
        return o
    if c["op"] == "scores":
        b.attn_mod_scores(plan, s["mod"], s["S"], s["out"], s["ws"])
        return [s["out"]]
    if c["op"] == "attend":
        b.attn_forward_natural_mod(plan, s["mod"], s["q"], s["k"], s["v"], s["idx"], s["cnt"], s["o"], s["ws"],
                                   lse_nat=s["lse"], q_scale=s.get("qs"), k_scale=s.get("ks"))
        return [s["o"], s["lse"]]
    if c["op"] == "layer":
        b.attn_layer_mod(plan, s["rope"], s["mod"], s["q"], s["k"], s["v"], s["o"], s["ws"], lse_nat=s["lse"])
        return [s["o"], s["lse"]]
    b.attn_forward_mod(plan, s["mod"], s["q"], s["k"], s["v"], s["idx"], s["cnt"], s["o"], s["ws"], lse=s["lse"])
    b.attn_backward_mod(plan, s["mod"], s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["idx"], s["cnt"],
                        *s["grads"], s["bws"], d_slopes=s["dslopes"])
    return [s["o"], s["lse"], *s["grads"]] + ([s["dslopes"]] if c["bias"] else [])


# ------------------------------------------------------------------ the plain forms

def _plain_rope(s, x):
    """Rotated x in fp32 (natural layout)."""
    c = s["case"]
    f, axis = _freqs(c)
    R = 2 * f.size
    if s["pos"] is not None:
        p = s["pos"].double()
    else:
        p = (s["g"]["coord"] + torch.tensor(_OFFSET, device="cuda")).double()[None]
    ang = p[..., torch.from_numpy(axis).cuda()] * torch.from_numpy(f).cuda()  # [B or 1, L, pairs]
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    if c["transpose"]:
        sin = -sin
    x = x.float()
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if c["half"] else (x[..., 0:R:2], x[..., 1:R:2])
    y = x.clone()
    u, w = a * cos - b * sin, a * sin + b * cos
    if c["half"]:
        y[..., :R // 2], y[..., R // 2:R] = u, w
    else:
        y[..., 0:R:2], y[..., 1:R:2] = u, w
    return y


def _plain_mean(s, y):
    (_, _, N, V), c = _tiles(s["case"]), s["case"]
    real = (s["g"]["slot"] < y.shape[1]).reshape(N, V).sum(1).float()
    t = _to_tiles(y, s["g"]["slot"]).reshape(c["B"], c["heads"], N, V, c["D"])
    return t.sum(3) / real[:, None]


def _plain_scores(s):
    c, g, S = s["case"], s["g"], s["S"]
    _, _, N, V = _tiles(c)
    out = c["cap"] * torch.tanh(S / c["cap"]) if c["cap"] else S.clone()
    slot = g["slot"].reshape(N, V)
    real = slot < g["coord"].shape[0]
    xyz = g["coord"].float()[slot.clamp_max(g["coord"].shape[0] - 1)] * real[..., None]
    if c["bias"]:
        mid = xyz.sum(1) / real.sum(1, keepdim=True)
        far = ((mid[:, None] - mid[None]).abs() * torch.tensor(_DIST, device="cuda")).sum(-1)
        out = out - s["slopes"][:, None, None] * far
    ok = torch.ones((c["B"], 1, N, N), dtype=torch.bool, device="cuda")
    if c["causal"]:
        first = torch.where(real, xyz[..., 0], math.inf).amin(1)
        last = torch.where(real, xyz[..., 0], -math.inf).amax(1)
        ok = ok & ((first[None, :] <= last[:, None]) | (first[None, None, None] < s["prefix"][:, None, None, None]))
    if s["doc"] is not None:
        d = torch.cat((s["doc"], torch.full_like(s["doc"][:, :1], -1)), 1)[:, slot].float()
        lo, hi = torch.where(d >= 0, d, math.inf).amin(2), d.amax(2)
        ok = ok & ((lo[:, None, :] <= hi[:, :, None]) & (lo[:, :, None] <= hi[:, None, :]))[:, None]
    return torch.where(ok, out, LOWEST)


def _plain_attend(s, q, k, v, do=None):
    """Attention over kept tiles on tiled fp32 tensors [B, heads, N * V, D], a few (batch, head) pairs at a time:
    O, lse and, with the gradient of O, dQ, dK, dV and the slopes' gradient per (batch, head)."""
    c, g = s["case"], s["g"]
    (_, _, N, V), D, heads = _tiles(c), c["D"], c["heads"]
    BH, kmax, L, dev = c["B"] * heads, s["idx"].shape[-1], g["coord"].shape[0], q.device
    q, k, v = (x.reshape(BH, N, V, D) for x in (q, k, v))
    idx, cnt = s["idx"].reshape(BH, N, kmax).long(), s["cnt"].reshape(BH, N)
    slot = g["slot"].reshape(N, V)
    real = slot < L
    xyz = g["coord"].float()[slot.clamp_max(L - 1)]
    doc = torch.where(real, 0, -1)[None].expand(c["B"], N, V)
    if s["doc"] is not None:
        doc = torch.cat((s["doc"], torch.full_like(s["doc"][:, :1], -1)), 1)[:, slot]
    scale, out = 1.0 / math.sqrt(D), [[] for _ in range(6)]
    step = max(1, (1 << 29) // (N * V * kmax * V))
    for at in range(0, BH, step):
        e = torch.arange(at, min(at + step, BH), device=dev)
        b, j = e // heads, idx[at:at + step]
        take = lambda x: x[at:at + step][torch.arange(e.numel(), device=dev)[:, None, None], j].reshape(e.numel(), N, kmax * V, D)  # noqa: E731
        K, Vv = take(k), take(v)
        z = scale * (q[e] @ K.transpose(-1, -2))
        th = None
        if c["cap"]:
            th = torch.tanh(z / c["cap"])
            z = c["cap"] * th
        far = None
        if c["bias"]:
            far = torch.zeros_like(z)
            for a in range(3):
                far += _DIST[a] * (xyz[None, :, :, None, a] - xyz[j, :, a].reshape(e.numel(), N, 1, kmax * V)).abs()
            z = z - s["slopes"][e % heads][:, None, None, None] * far
        dk_, dq_ = doc[b[:, None, None], j].reshape(e.numel(), N, 1, kmax * V), doc[b][..., None]
        ok = (dq_ == dk_) & (dk_ >= 0)
        ok &= (torch.arange(kmax, device=dev) < cnt[e][..., None]).repeat_interleave(V, -1)[:, :, None]
        if c["causal"]:
            tk = xyz[j, :, 0].reshape(e.numel(), N, 1, kmax * V)
            ok &= (tk <= xyz[None, :, :, None, 0]) | (tk < s["prefix"][b][:, None, None, None])
        z = torch.where(ok, z, -math.inf)
        top = z.amax(-1, keepdim=True)
        p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
        tot = p.sum(-1, keepdim=True)
        p = p / torch.where(tot > 0, tot, 1.0)
        o = p @ Vv
        out[0].append(o)
        out[1].append((top + torch.log(tot))[..., 0])
        if do is None:
            continue
        G = do.reshape(BH, N, V, D)[e]
        dz = p * (G @ Vv.transpose(-1, -2) - (G * o).sum(-1, keepdim=True))
        if far is not None:
            out[5].append(-(dz * far).sum((1, 2, 3)))
        ds = scale * (dz * (1.0 - th * th) if th is not None else dz)
        out[2].append(ds @ K)
        for to, x, y in ((3, ds, q[e]), (4, p, G)):
            part = (x.transpose(-1, -2) @ y).reshape(e.numel() * N * kmax, V, D)
            put = torch.zeros((e.numel() * N, V, D), device=dev)
            put.index_add_(0, (j + N * torch.arange(e.numel(), device=dev)[:, None, None]).reshape(-1), part)
            out[to].append(put.reshape(e.numel(), N, V, D))
    return [torch.cat(x) if x else None for x in out]


def run(s):
    if own:
        return _own_run(s)
    c = s["case"]
    if c["op"] == "scores":
        return [_plain_scores(s)]
    if c["op"] == "rope":
        y = [_plain_rope(s, s["q"]), _plain_rope(s, s["k"])]
        return [x.to(torch.bfloat16) for x in y] + ([_plain_mean(s, x) for x in y] if c["pooled"] else [])
    if c["op"] == "train":
        o, lse, *grads, dsl = _plain_attend(s, *(s[x].float() for x in ("q", "k", "v", "do")))
        out = [o.reshape(s["q"].shape).to(torch.bfloat16), lse.reshape(s["q"].shape[:-1])]
        out += [x.reshape(s["q"].shape).to(torch.bfloat16) for x in grads]
        return out + ([dsl.reshape(c["B"], c["heads"]).sum(0)] if c["bias"] else [])
    q, k = s["q"], s["k"]
    if c["op"] == "layer":  # the rotated Q and K are bf16 tensors
        q, k = (_plain_rope(s, x).to(torch.bfloat16) for x in (q, k))
    if c["fp8"]:
        q, k = _decoded(q, s["qs"], torch.float32), _decoded(k, s["ks"], torch.float32)
    else:
        q, k = (_to_tiles(x.float(), s["g"]["slot"]) for x in (q, k))
    o, lse = _plain_attend(s, q, k, _to_tiles(s["v"].float(), s["g"]["slot"]))[:2]
    o = o.reshape(c["B"], c["heads"], -1, c["D"])[:, :, s["g"]["place"]].transpose(1, 2)
    return [o.to(torch.bfloat16).contiguous(), lse.reshape(c["B"], c["heads"], -1)[:, :, s["g"]["place"]]]


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(s, name):
    """Each pair as a complex number, turned."""
    c = s["case"]
    x = s[name].double()
    f, axis = _freqs(c)
    n = f.size
    at = s["pos"].double() if s["pos"] is not None else s["g"]["coord"].double()[None] + torch.tensor(_OFFSET, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       (-1.0 if c["transpose"] else 1.0) * at[..., axis] * torch.from_numpy(f).cuda())
    first = torch.arange(n, device="cuda") * (1 if c["half"] else 2)
    second = first + (n if c["half"] else 1)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, :, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_rules(s, b, h, rows, cols):
    """(distance, visibility) of token rows against token columns of one (batch, head), from their coordinates."""
    c, xyz = s["case"], s["g"]["coord"].double()
    far = sum(w * (xyz[rows, None, a] - xyz[None, cols, a]).abs() for a, w in enumerate(_DIST))
    ok = torch.ones((rows.numel(), cols.numel()), dtype=torch.bool, device="cuda")
    if c["causal"]:
        ok &= (xyz[None, cols, 0] <= xyz[rows, None, 0]) | (xyz[None, cols, 0] < float(s["prefix"][b]))
    if s["doc"] is not None:
        ok &= (s["doc"][b, rows][:, None] == s["doc"][b, cols][None]) & (s["doc"][b, cols] >= 0)[None]
    return far, ok


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    (_, _, N, V), L, D = _tiles(c), c["T"] * c["H"] * c["W"], c["D"]
    tile, place = s["g"]["tile"], s["g"]["place"]
    if c["op"] == "rope":
        y = [_exact_rope(s, x) for x in ("q", "k")]
        if not c["pooled"]:
            return y
        cnt = torch.zeros(N, dtype=torch.float64, device="cuda").index_add_(0, tile, torch.ones(L, dtype=torch.float64, device="cuda"))
        return y + [(torch.zeros((c["B"], N, c["heads"], D), dtype=torch.float64, device="cuda").index_add_(1, tile, x)
                     / cnt[:, None, None]).transpose(1, 2) for x in y]
    if c["op"] == "scores":
        z = s["S"].double()
        if c["cap"]:
            z = c["cap"] * (1.0 - 2.0 / (torch.exp(2.0 * z / c["cap"]) + 1.0))
        xyz, n = s["g"]["coord"].double(), torch.bincount(tile, minlength=N).double()
        if c["bias"]:
            for a, w in enumerate(_DIST):
                m = torch.bincount(tile, weights=xyz[:, a], minlength=N) / n
                z = z - s["slopes"].double()[:, None, None] * w * (m[:, None] - m[None]).abs()
        for b in range(c["B"]):
            ends = lambda val, how, start: torch.full((N,), start, dtype=torch.float64, device="cuda").scatter_reduce(0, tile, val, how)  # noqa: E731
            hide = torch.zeros((N, N), dtype=torch.bool, device="cuda")
            if c["causal"]:
                lo, hi = ends(xyz[:, 0], "amin", math.inf), ends(xyz[:, 0], "amax", -math.inf)
                hide |= (lo[None] > hi[:, None]) & (lo[None] >= float(s["prefix"][b]))
            if s["doc"] is not None:
                d = s["doc"][b].double()
                lo, hi = ends(torch.where(d < 0, math.inf, d), "amin", math.inf), ends(d, "amax", -1.0)
                hide |= (lo[None] > hi[:, None]) | (lo[:, None] > hi[None])
            z[b].masked_fill_(hide, float(LOWEST))
        return [z]
    if c["B"] * c["heads"] * float(L) * L > 1.2e11:
        return None
    train = c["op"] == "train"
    if train:
        q, k, v, do = (s[x].double().reshape(c["B"], c["heads"], N * V, D)[:, :, place] for x in ("q", "k", "v", "do"))
    elif c["fp8"]:
        q, k = (_decoded(s[x], s[x + "s"], torch.float64)[:, :, place] for x in ("q", "k"))
        v = s["v"].double().transpose(1, 2)
    else:
        q, k, v = ((_exact_rope(s, x).to(torch.bfloat16) if c["op"] == "layer" and x != "v" else s[x]).double().transpose(1, 2)
                   for x in ("q", "k", "v"))
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(q) for _ in range(3)] if train else []
    dslopes = torch.zeros(c["heads"], dtype=torch.float64, device="cuda")
    cols, scale = torch.arange(L, device="cuda"), D ** -0.5
    for b in range(c["B"]):
        for h in range(c["heads"]):
            kept = torch.zeros((N, N), dtype=torch.bool, device="cuda")
            live = torch.arange(s["idx"].shape[-1], device="cuda") < s["cnt"][b, h][:, None]
            kept[torch.nonzero(live)[:, 0], s["idx"][b, h][live].long()] = True
            for rows in cols.split(max(1, (1 << 28) // L)):
                far, ok = _exact_rules(s, b, h, rows, cols)
                ok &= kept[tile[rows]][:, tile]
                x = q[b, h, rows] @ k[b, h].T * scale
                z, slope_of = x, 1.0
                if c["cap"]:
                    ex = torch.exp(-2.0 * x.abs() / c["cap"])
                    z, slope_of = x.sign() * c["cap"] * (1 - ex) / (1 + ex), 4 * ex / (1 + ex) ** 2
                if c["bias"]:
                    z = z - s["slopes"][h].double() * far
                z = z.masked_fill(~ok, -math.inf)
                lse[b, h, rows] = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[b, h, rows].nan_to_num(neginf=0.0)[:, None])
                o[b, h, rows] = p @ v[b, h]
                if train:
                    dp = do[b, h, rows] @ v[b, h].T
                    dz = p * (dp - (p * dp).sum(-1, keepdim=True))
                    dslopes[h] -= (dz * far).sum()
                    ds = dz * slope_of * scale
                    grads[0][b, h, rows] = ds @ k[b, h]
                    grads[1][b, h] += ds.T @ q[b, h, rows]
                    grads[2][b, h] += p.T @ do[b, h, rows]
    if not train:
        return [o.transpose(1, 2).contiguous(), lse]
    full = lambda x, fill: torch.full((c["B"], c["heads"], N * V) + x.shape[3:], fill, dtype=torch.float64, device="cuda").index_copy_(2, place, x)  # noqa: E731
    out = [full(o, 0.0), full(lse, -math.inf)] + [full(x, 0.0) for x in grads]
    out = [x.reshape((c["B"], c["heads"], N, V) + x.shape[3:]) for x in out]
    return out + ([dslopes] if c["bias"] else [])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    (_, n, N, V), L, D = _tiles(c), c["T"] * c["H"] * c["W"], c["D"]
    rows = c["B"] * c["heads"] * L
    if c["op"] == "rope":
        pooled = 2 * 4 * c["B"] * c["heads"] * N * D if c["pooled"] else 0
        return {"bytes": 2 * 2 * 2 * rows * D + pooled, "flops": 2 * 3 * rows * (c["dim_t"] + c["dim_h"] + c["dim_w"])}
    if c["op"] == "scores":
        e = c["B"] * c["heads"] * N * N
        return {"bytes": 8 * e, "flops": e * (2 + 8 * bool(c["cap"]) + 2 * c["bias"])}
    if c["win_t"] >= 0:  # kept tile pairs of a clipped window
        pairs = 1
        for m, w in zip(n, (c["win_t"], c["win_h"], c["win_w"])):
            pairs *= sum(min(m - 1, i + w) - max(0, i - w) + 1 for i in range(m))
    else:
        pairs = N * c["topk"]
    share = (0.5 + 0.5 / max(1, c["T"])) if c["causal"] else 1.0  # of the kept token pairs: about what the rules leave
    share /= max(1, c["docs"]) if c["win_t"] >= 0 else 1
    seen = c["B"] * c["heads"] * pairs * (L / N) ** 2 * share
    lists = 4 * c["B"] * c["heads"] * (pairs + N) if c["op"] != "layer" else 0
    if c["op"] == "train":
        return {"bytes": (4 + 1 + 3) * 2 * rows * D + 8 * rows + 2 * lists, "flops": 14 * D * seen}
    qk = 2 if c["fp8"] else 4
    return {"bytes": (qk + 4) * rows * D + 4 * rows + lists, "flops": 4 * D * seen}
