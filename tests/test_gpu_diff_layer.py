"""The differential-attention layer as it is used: a fused projection's Q, K and V
rotated into cube order, lambda, attention over windows and global tokens, each
head normalised, raster order; and the gradients all the way back. Against the
same chain in 64 bits with torch's autograd.

Bounds, in 2-norms relative to the reference: every stored tensor is rounded once
(U = half a step), and so are the attention's weights; each such rounding moves a
result by at most U of the tensors it combines. Forward: rotated Q, K, V, weights,
output, normalised output: 6 roundings on the way. Backward: those, and dy in cube
order, the norm's dx, dS, dQ/dK/dV, the rotation back: 12. Logits of order 4 and
the norm's division by the output's own size (about its rounding's size in units)
multiply by less than 2 each: 4 x 6 U and 4 x 12 U. fp32: 2^-24 (sums of a few
hundred terms) in place of U.
"""
import pytest
import torch

import diff_ref
from helpers import check_no_device_error
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
GRID, CUBE, GGRID = (3, 6, 10), (2, 4, 4), (2, 3, 5)     # partial cubes
H = 3


def rotate64(x, pos, split, scales, layout):
    """[rows, heads, w] float64, differentiable."""
    out, base = [], 0
    for a, d in enumerate(split):
        k = torch.arange(d // 2, dtype=torch.float64, device=x.device)
        phi = (pos[:, a].double() * scales[a])[:, None, None] * 10000.0 ** (-2 * k / d)
        seg = x[..., base:base + d]
        p, q = (seg[..., :d // 2], seg[..., d // 2:]) if layout == "half" else (seg[..., 0::2], seg[..., 1::2])
        a1, a2 = p * phi.cos() - q * phi.sin(), p * phi.sin() + q * phi.cos()
        out.append(torch.cat([a1, a2], -1) if layout == "half" else torch.stack([a1, a2], -1).flatten(-2))
        base += d
    return torch.cat(out + [x[..., base:]], -1)


def positions(grid):
    return torch.stack(torch.meshgrid(*(torch.arange(e) for e in grid), indexing="ij"), -1).reshape(-1, 3).to(DEV)


def setup(hd, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(hd)
    n, m = GRID[0] * GRID[1] * GRID[2], GGRID[0] * GGRID[1] * GGRID[2]
    t = {"d": torch.randn(n, 3 * H, hd, generator=g, device=DEV).to(DT[dtype]),
         "g": torch.randn(m, 3 * H, hd, generator=g, device=DEV).to(DT[dtype]),
         "dy_d": torch.randn(n, H, hd, generator=g, device=DEV).to(DT[dtype]),
         "dy_g": torch.randn(m, H, hd, generator=g, device=DEV).to(DT[dtype])}
    t["vec"] = [(0.3 * torch.randn(H, hd // 2, generator=g, device=DEV)).to(DT[dtype]) for _ in range(4)]
    t["gamma"] = 0.5 + 0.1 * torch.randn(H * hd, generator=g, device=DEV)
    return t, n, m


def layer(t, n, m, hd, split, layout):
    """The calls of a training step; returns outputs and gradients in raster order."""
    dt, e = t["d"].dtype, lambda r: torch.empty(r, H, hd, dtype=t["d"].dtype, device=DEV)
    scales = {"d": (1.0, 1.0, 1.0), "g": (1.0, 2.0, 2.0)}
    maps = lambda x: x.view(x.shape[0], 2 * H, hd // 2)  # noqa: E731
    cols = lambda x, i: x[:, i * H:(i + 1) * H]  # noqa: E731
    wide = lambda x, i: x.view(x.shape[0], 6 * H, hd // 2)[:, 2 * i * H:2 * (i + 1) * H]  # noqa: E731
    rot = {s: atlas.make_rotary(10000.0, split, scales[s], layout=layout) for s in "dg"}
    grid, cube, order = {"d": GRID, "g": GGRID}, {"d": CUBE, "g": None}, {"d": "reorder", "g": "raster"}
    rows = {"d": n, "g": m}
    q, k, v, o, s, y, r = ({p: e(rows[p]) for p in "dg"} for _ in range(7))
    for p in "dg":
        atlas.rotary([(wide(t[p], 0), maps(q[p])), (wide(t[p], 1), maps(k[p])), (wide(t[p], 2), maps(v[p]), False)],
                     grid[p], rot[p], cube=cube[p], order=order[p])
    lam, dlam = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    atlas.diff_lambda(*t["vec"], 0.5, lam)
    off = atlas.cube_window_offsets(GRID, CUBE).to(DEV)
    lse = torch.empty(1, H, 2, n + m, device=DEV)
    kw = {"window_offsets": off}
    atlas.diff_attn(q["d"], k["d"], v["d"], q["g"], k["g"], v["g"], lam, o["d"], o["g"], s["d"], s["g"], lse, **kw)
    stats, flat = {p: torch.empty(rows[p], H, 2, device=DEV) for p in "dg"}, lambda x: x.view(x.shape[0], H * hd)
    for p in "dg":
        atlas.group_norm(flat(o[p]), t["gamma"], None, flat(y[p]), 1, H, stats=stats[p])
    atlas.cube_unorder(y["d"], r["d"], GRID, CUBE)
    out = {"y_d": r["d"], "y_g": y["g"]}
    # back
    dy, do = {"d": e(n), "g": t["dy_g"]}, {p: e(rows[p]) for p in "dg"}
    atlas.cube_reorder(t["dy_d"], dy["d"], GRID, CUBE)
    dgamma = {p: torch.empty(H * hd, device=DEV) for p in "dg"}
    for p in "dg":
        atlas.group_norm_bwd(flat(dy[p]), flat(o[p]), t["gamma"], None, stats[p], flat(do[p]), dgamma[p], None, 1, H)
    dq, dk, dv = ({p: e(rows[p]) for p in "dg"} for _ in range(3))
    atlas.diff_attn_bwd(q["d"], k["d"], v["d"], o["d"], s["d"], do["d"], q["g"], k["g"], v["g"], o["g"], s["g"],
                        do["g"], lam, lse, dq["d"], dk["d"], dv["d"], dq["g"], dk["g"], dv["g"], dlam, **kw)
    dvec = [torch.empty_like(x) for x in t["vec"]]
    atlas.diff_lambda_bwd(*t["vec"], dlam, *dvec)
    for p in "dg":
        back = torch.empty_like(t[p])
        atlas.rotary([(maps(dq[p]), wide(back, 0)), (maps(dk[p]), wide(back, 1)), (maps(dv[p]), wide(back, 2), False)],
                     grid[p], rot[p], cube=cube[p], order={"d": "unorder", "g": "raster"}[p], transpose=True)
        out["dqkv_" + p] = back
    out["dgamma"], out["dvec"] = dgamma["d"] + dgamma["g"], torch.cat(dvec)
    assert cols(t["d"], 0).dtype == dt
    return out


def reference(t, n, m, hd, split, layout):
    x = {p: t[p].double().requires_grad_() for p in "dg"}
    vec = [v.double().requires_grad_() for v in t["vec"]]
    gamma = t["gamma"].double().requires_grad_()
    scales = {"d": (1.0, 1.0, 1.0), "g": (1.0, 2.0, 2.0)}
    q, k, v = [], [], []
    for p, grid in (("d", GRID), ("g", GGRID)):
        halves = x[p].reshape(x[p].shape[0], 6 * H, hd // 2)
        pos = positions(grid)
        for i, into in ((0, q), (1, k)):
            into.append(rotate64(halves[:, 2 * i * H:2 * (i + 1) * H], pos, split, scales[p], layout))
        v.append(x[p][:, 2 * H:])
    q, k, v = torch.cat(q), torch.cat(k), torch.cat(v)
    pos = positions(GRID)
    cube = ((pos // torch.tensor(CUBE, device=DEV)) * torch.tensor([10000, 100, 1], device=DEV)).sum(1)
    mask = torch.zeros(n + m, n + m, dtype=torch.bool, device=DEV)
    mask[:n, :n] = cube[:, None] == cube[None, :]
    mask[:, n:] = True
    p = []
    for i in range(2):
        s = torch.einsum("qhc,khc->hqk", q[:, i::2], k[:, i::2]) * (hd // 2) ** -0.5
        p.append(torch.softmax(s.masked_fill(~mask, float("-inf")), -1))
    lam = (vec[0] * vec[1]).sum(1).exp() - (vec[2] * vec[3]).sum(1).exp() + 0.5
    o = torch.einsum("hqk,khc->qhc", p[0] - lam[:, None, None] * p[1], v)
    y = (o - o.mean(-1, keepdim=True)) / (o.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    y = y * gamma.reshape(H, hd)
    (y * torch.cat([t["dy_d"], t["dy_g"]]).double()).sum().backward()
    return {"y_d": y[:n], "y_g": y[n:], "dqkv_d": x["d"].grad, "dqkv_g": x["g"].grad, "dgamma": gamma.grad,
            "dvec": torch.cat([a.grad for a in vec])}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,split", [(64, (8, 12, 12)), (128, (16, 14, 22))])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_layer(hd, split, layout, dtype):
    t, n, m = setup(hd, dtype)
    got = layer(t, n, m, hd, split, layout)
    torch.cuda.synchronize()
    check_no_device_error()
    want = reference(t, n, m, hd, split, layout)
    u = diff_ref.unit(DT[dtype]) if dtype == "bf16" else 2.0 ** -24 * 16
    for name, w in want.items():
        err = float((got[name].double() - w).norm() / w.norm())
        assert err <= 4 * (6 if name.startswith("y") else 12) * u, (name, err)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_in_a_graph(dtype):
    """One captured step (no call made before it on these shapes) replays the
    eager step's bits, on new inputs too."""
    t, n, m = setup(64, dtype)
    args = (n, m, 64, (8, 12, 12), "half")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    off = atlas.cube_window_offsets(GRID, CUBE)      # (host; its copy to the device is not captured)
    real = atlas.cube_window_offsets
    dev_off = off.to(DEV)
    atlas.cube_window_offsets = lambda *a: dev_off
    try:
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = layer(t, *args)
        for p in "dg":
            t[p].copy_(torch.flip(t[p], (0,)))
        g.replay()
        torch.cuda.synchronize()
        eager = layer(t, *args)
    finally:
        atlas.cube_window_offsets = real
    torch.cuda.synchronize()
    check_no_device_error()
    for name in out:
        assert torch.equal(out[name], eager[name]), name
