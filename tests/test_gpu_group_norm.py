"""Group norm, channels last, with its activation and gradients, against a
64-bit reference (bounds in diff_ref.py)."""
import pytest
import torch

import diff_ref
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rnd(*shape, seed=0, dtype=torch.float32, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


CASES = [
    # samples, rows, channels, groups
    (1, 1, 1, 1),            # one value: zero variance
    (2, 1, 7, 7),            # groups of one value
    (5, 1, 2, 1),
    (3, 1001, 60, 12),       # groups of five channels
    (2, 37, 5, 1),           # rows of ten bytes (bf16)
    (1, 700, 24, 8),
    (301, 1, 1280, 10),      # heads of 128, one token each
    (9, 1, 5120, 40),
    (33, 1, 512, 8),         # heads of 64
    (40, 1, 96, 1),          # a whole token
    (64, 1, 160, 2),         # 80 channels: no power of two
    (7, 3, 256, 4),          # three rows a sample
    (2, 4096, 64, 32),       # many rows, two channels a group
    (1, 20011, 128, 32),
    (3, 5000, 320, 32),      # groups of ten
    (2, 2500, 2048, 4),      # more than one slice of columns
    (2, 600, 5120, 4),       # slices of several rows a block
    (1, 3, 8200, 1),
]


def run(x, gamma, beta, rows, groups, act, dy):
    S = x.shape[0] // rows
    y, dx = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    stats = torch.full((S, groups, 2), 9.0, device=DEV)
    dg, db = (torch.full((x.shape[1],), 9.0, device=DEV) for _ in range(2))
    atlas.group_norm(x, gamma, beta, y, rows, groups, activation=act, stats=stats)
    atlas.group_norm_bwd(dy, x, gamma, beta, stats, dx, dg, db, rows, groups, activation=act)
    return y, stats, dx, dg, db


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_reference(case, act, dtype):
    S, R, C, K = case
    x = (rnd(S * R, C) + rnd(1, C, seed=1)).to(DT[dtype])
    dy = rnd(S * R, C, seed=2, dtype=DT[dtype])
    gamma, beta = 1 + 0.2 * rnd(C, seed=3), 0.2 * rnd(C, seed=4)
    y, stats, dx, dg, db = run(x, gamma, beta, R, K, act, dy)
    r = diff_ref.group_norm(x.double(), gamma.double(), beta.double(), R, K, 1e-5, act == "silu",
                            DT[dtype], dy.double())
    for name, got in (("mean", stats[..., 0]), ("rstd", stats[..., 1]), ("y", y), ("dx", dx),
                      ("dgamma", dg), ("dbeta", db)):
        diff_ref.check(name, got.double(), r[name], r[name + "_bound"])
    again = run(x, gamma, beta, R, K, act, dy)
    assert all(torch.equal(a, b) for a, b in zip((y, stats, dx, dg, db), again))


@pytest.mark.parametrize("case", [(2, 37, 64, 4), (64, 1, 256, 4), (1, 3000, 60, 12)], ids=str)
def test_without_affine_and_in_place(case):
    S, R, C, K = case
    x, dy = rnd(S * R, C), rnd(S * R, C, seed=1)
    stats = torch.empty(S, K, 2, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    atlas.group_norm(x, None, None, y, R, K, stats=stats, activation="silu")
    atlas.group_norm_bwd(dy, x, None, None, stats, dx, None, None, R, K, activation="silu")
    r = diff_ref.group_norm(x.double(), None, None, R, K, 1e-5, True, torch.float32, dy.double())
    diff_ref.check("y", y.double(), r["y"], r["y_bound"])
    diff_ref.check("dx", dx.double(), r["dx"], r["dx_bound"])
    over = x.clone()
    atlas.group_norm(over, None, None, over, R, K, activation="silu")
    assert torch.equal(over, y)
    for into in ("dy", "x"):
        a, b = x.clone(), dy.clone()
        dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        atlas.group_norm_bwd(b, a, None, None, stats, b if into == "dy" else a, dg, db, R, K,
                             activation="silu")
        assert torch.equal(b if into == "dy" else a, dx)
        diff_ref.check("dgamma", dg.double(), r["dgamma"], r["dgamma_bound"])


@pytest.mark.parametrize("case", [(1, 4000, 64, 4), (50, 1, 256, 4), (2, 100, 40, 8)], ids=str)
def test_large_mean(case):
    """Values of mean 1000 and deviation 1: the variance is not lost in the squares'
    cancellation (relative error of rstd bounded by the mean's own rounding)."""
    S, R, C, K = case
    x = 1000 + rnd(S * R, C)
    y, stats, *_ = run(x, None, None, R, K, "none", rnd(S * R, C, seed=1))
    r = diff_ref.group_norm(x.double(), None, None, R, K, 1e-5, False, torch.float32)
    # centred sums: x - pivot is exact to 2^-24 of 1000 in a value of order 1
    assert float((stats[..., 1].double() / r["rstd"] - 1).abs().max()) <= 2.0 ** -10
    diff_ref.check("y", y.double(), r["y"], r["y_bound"])


@pytest.mark.parametrize("case", [(1, 900, 64, 4), (20, 1, 128, 4), (3, 50, 30, 3)], ids=str)
def test_constant_and_non_finite(case):
    """A constant group gives beta exactly; NaN stays in its (sample, group)."""
    S, R, C, K = case
    x = rnd(S * R, C)
    cg = C // K
    x[:R, :cg] = 3.0
    x[R * (S - 1):, C - cg:][R // 2, 0] = float("nan")
    beta = rnd(C, seed=1)
    y = torch.empty_like(x)
    atlas.group_norm(x, None, beta, y, R, K)
    assert torch.equal(y[:R, :cg], beta[:cg].expand(R, cg))
    bad = torch.isnan(y)
    assert bool(bad[R * (S - 1):, C - cg:].all())
    bad[R * (S - 1):, C - cg:] = False
    assert not bad.any()


def test_gradient_against_differences():
    """Central differences of the forward call in fp32: step h, truncation h^2
    and rounding 2^-22 |sum| / h, both below the bound used."""
    S, R, C, K = 2, 6, 12, 3
    x, dy = rnd(S * R, C), rnd(S * R, C, seed=1)
    gamma, beta = 1 + 0.2 * rnd(C, seed=2), 0.2 * rnd(C, seed=3)
    _, _, dx, dg, db = run(x, gamma, beta, R, K, "silu", dy)

    def loss(a, g, b):
        y = torch.empty_like(a)
        atlas.group_norm(a, g, b, y, R, K, activation="silu")
        return float((y.double() * dy.double()).sum())

    h = 2.0 ** -6
    for t, grad, picks in ((0, dx, ((0, 0), (5, 7), (11, 11))), (1, dg, ((3,), (11,))),
                           (2, db, ((0,), (6,)))):
        for at in picks:
            args = [[x, gamma, beta], [x, gamma, beta]]
            ends = []
            for sign, a in zip((1, -1), args):
                a[t] = a[t].clone()
                a[t][at] += sign * h
                ends.append(loss(*a))
            # truncation f''' h^2 / 6: at unit variance the third derivatives of a
            # group's values (or of silu over a channel's rows) add up to below 48 max |dy|
            tol = 8 * h * h * float(dy.abs().max()) + 2.0 ** -22 * float(dy.abs().sum()) / h
            assert abs((ends[0] - ends[1]) / (2 * h) - float(grad[at])) <= tol


def test_graph_and_streams():
    S, R, C, K = 2, 3000, 64, 4
    x, dy = rnd(S * R, C, dtype=torch.bfloat16), rnd(S * R, C, seed=1, dtype=torch.bfloat16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty(S, K, 2, device=DEV)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)

    def step():
        atlas.group_norm(x, None, None, y, R, K, activation="silu", stats=stats)
        atlas.group_norm_bwd(dy, x, None, None, stats, dx, dg, db, R, K, activation="silu")

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    x.copy_(rnd(S * R, C, seed=7, dtype=torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    first = [t.clone() for t in (y, dx, stats, dg, db)]
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, stats, dg, db)))
