"""The differential-attention layer's kernels where a block takes several units,
tiles or samples in turn, and what they write: nothing outside their outputs."""
import numpy as np
import pytest
import torch

import diff_ref
from helpers import check_no_device_error
from test_gpu_diff_attn import DEV, DT, GRADS, against_reference, make, rnd, run
from test_gpu_rotary import expect, grid_pos, inputs
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu
SMS = 148   # of a B200: one attention block each


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- several units a block ------------------------------------------------------

MIXED = [0, 300, 301, 428, 430, 557, 686, 900, 905, 1100, 1101, 1300, 1500, 1530, 1660, 1900, 2100, 2400, 2560]
SHORT = list(range(0, 2560, 20)) + [2560]
LAYOUTS = {
    # window offsets (fixed windows where they are even), global ranges
    "windows of 256": (list(range(0, 2561, 256)), None),
    "windows of 20": (SHORT, None),
    "windows of 20, aligned": (SHORT, [i * 130 // 128 for i in range(129)]),
    "mixed offsets": (MIXED, None),
    "mixed offsets, aligned": (MIXED, [i * 130 // 18 for i in range(19)]),
}


def layout_of(name):
    windows, shares = LAYOUTS[name]
    kw = {"global_window_offsets": int32(shares)} if shares else {}
    if name.startswith("mixed"):
        kw["window_offsets"] = int32(windows)
    else:
        kw["window_len"] = windows[1]
    return windows, shares, kw


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_attention_over_several_units_a_block(layout, hd):
    """528 units of 128 rows: every block walks three or four, forward and backward."""
    B, N, G, H = 2, 2560, 130, 12
    assert B * H * (N // 128 + 2) > 3 * SMS
    windows, shares, kw = layout_of(layout)
    t = make(B, N, G, H, hd, "bf16", seed=11)
    lam = 0.3 + 0.2 * rnd(H, seed=5)
    out = run(t, lam, B, N, G, H, **kw)
    against_reference(t, out, lam, B, N, G, H, hd, "bf16", windows, shares)
    again = run(t, lam, B, N, G, H, **kw)
    for n in out:
        assert torch.equal(out[n], again[n]), n


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("layout", ["windows of 20, aligned", "mixed offsets, aligned"])
def test_non_finite_rows_over_several_units_a_block(layout, hd):
    """NaN and infinities in every seventh window of every head and problem: those
    windows' rows show them, the other rows' bits stay, in whichever unit a block
    comes to them."""
    B, N, G, H = 2, 2560, 130, 12
    windows, shares, kw = layout_of(layout)
    t = make(B, N, G, H, hd, "bf16", seed=12)
    lam = 0.3 + 0.2 * rnd(H, seed=5)
    clean = run(t, lam, B, N, G, H, **kw)
    for name, value in (("v", "inf"), ("k", "nan"), ("q", "nan"), ("do", "-inf")):
        bad = {n: x.clone() for n, x in t.items()}
        hit = torch.zeros(B, N, dtype=torch.bool, device=DEV)
        for w in range(0, len(windows) - 1, 7):
            a, b = windows[w], windows[w + 1]
            rows = bad[name + "_d"].view(B, N, H, hd)[:, a:b]
            rows[:, (b - a) // 2, :, 5] = float(value)
            hit[:, a:b] = True
        hit = hit.flatten()
        out = run(bad, lam, B, N, G, H, **kw)
        for n in ("o", "s") + GRADS:
            assert torch.equal(out[n + "_d"][~hit], clean[n + "_d"][~hit]), (name, n)
            assert torch.equal(out["o_g"], clean["o_g"]) and torch.equal(out["dq_g"], clean["dq_g"])
        if name in ("v", "k"):   # (windows of 128 rows and more: the value's channel)
            assert not bool(torch.isfinite(out["o_d"][hit][..., 5]).any()), name
            assert not bool(torch.isfinite(out["s_d"][hit][..., 5]).any()) or name == "k"
            assert not bool(torch.isfinite(out["dq_d"][hit][..., 5]).any()), name
        if name in ("q", "do"):
            assert not bool(torch.isfinite(out["dk_d"][hit][..., 5]).any()), name


# ---- several tiles a block, several tokens and samples a thread -------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("order", ["raster", "reorder", "unorder"])
def test_rotary_over_several_tiles_a_block(order, layout, dtype):
    """85,000 rows of 64 pairs: 2,657 tiles of 32 rows for 1,184 blocks."""
    grid, cube, hd, split = (5, 100, 170), (2, 16, 24), 128, (44, 42, 42)
    rows = int(np.prod(grid))
    assert rows // 32 > 2 * 8 * SMS
    perm = diff_ref.cube_rows(grid, cube)
    rot = atlas.make_rotary(10000.0, split, (2.0, 1.0, 0.5), layout=layout)
    x = inputs(rows, 1, hd, dtype)
    y = torch.full_like(x, 7.0)
    moved = torch.full_like(x, 7.0)
    atlas.rotary([(x, y), (x, moved, False)], grid, rot, cube=cube, order=order)
    want, bound = expect(x, grid_pos(grid, 1), dtype, perm, order, 10000.0, split, (2.0, 1.0, 0.5), layout)
    diff_ref.check("y", y.double().cpu(), want, bound)
    at = torch.from_numpy(perm).to(DEV)
    if order == "reorder":
        assert torch.equal(moved, x[at])
    elif order == "unorder":
        assert torch.equal(moved[at], x)
    else:
        assert torch.equal(moved, x)


NORMS = [
    # samples, rows, channels, groups
    (80001, 1, 128, 1),      # heads: 16 tokens at a time, 592 blocks of 4 (forward) or 2 in flight
    (9001, 1, 1280, 10),     # heads: a token at a time and slice
    (1500, 3, 256, 4),       # resident: more samples than blocks
    (1300, 37, 60, 12),      # resident, groups of five channels
    (700, 1, 96, 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("case", NORMS, ids=str)
def test_norm_over_several_tokens_and_samples_a_block(case, act, dtype):
    S, R, C, K = case
    x = (rnd(S * R, C) + rnd(1, C, seed=1)).to(DT[dtype])
    dy = rnd(S * R, C, seed=2, dtype=DT[dtype])
    gamma, beta = 1 + 0.2 * rnd(C, seed=3), 0.2 * rnd(C, seed=4)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(S, K, 2, device=DEV)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    atlas.group_norm(x, gamma, beta, y, R, K, activation=act, stats=stats)
    atlas.group_norm_bwd(dy, x, gamma, beta, stats, dx, dg, db, R, K, activation=act)
    r = diff_ref.group_norm(x.double(), gamma.double(), beta.double(), R, K, 1e-5, act == "silu",
                            DT[dtype], dy.double())
    for name, got in (("mean", stats[..., 0]), ("rstd", stats[..., 1]), ("y", y), ("dx", dx),
                      ("dgamma", dg), ("dbeta", db)):
        diff_ref.check(name, got.double(), r[name], r[name + "_bound"])


# ---- nothing outside the outputs ----------------------------------------------------

class Guarded:
    """Tensors inside larger buffers whose other bytes must stay."""
    PAD = 4096

    def __init__(self):
        self.all = []

    def empty(self, shape, dtype=torch.float32):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((n + 2 * self.PAD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((buf, n))
        return buf[self.PAD:self.PAD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert bool((buf[:self.PAD] == 0xA5).all()) and bool((buf[self.PAD + n:] == 0xA5).all()), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("case", [
    # problems, detail rows, window (or offsets), global rows, heads
    (1, 1, 1, 1, 1), (2, 387, 129, 1, 2), (3, 0, 1, 333, 1), (1, 130, 1, 5, 1), (1, 2304, 768, 260, 1),
    (2, 600, [0, 200, 456, 457, 600], 130, 2), (1, 7, [0, 7], 0, 3), (1, 2100, [0, 700, 1400, 2100], 300, 1),
], ids=str)
def test_attention_writes_its_outputs_alone(case, hd, dtype):
    """Every output, and a workspace of exactly the size that the library states."""
    B, N, L, G, H = case
    kw = {"window_offsets": int32(L)} if isinstance(L, list) else {"window_len": L}
    t, dt = make(B, N, G, H, hd, dtype), DT[dtype]
    lam = torch.full((H,), 0.4, device=DEV)
    want = run(t, lam, B, N, G, H, **kw)
    g = Guarded()
    o = {f"{n}_{p}": g.empty((B * rows, H, hd), dt) for n in ("o", "s") + GRADS for p, rows in (("d", N), ("g", G))}
    o["lse"], o["dlam"] = g.empty((B, H, 2, N + G)), g.empty((H,))
    work = g.empty((atlas.diff_attn_bwd_workspace(B, N, G, H, hd, atlas.BF16 if dtype == "bf16" else atlas.FP32),),
                   torch.uint8)
    atlas.diff_attn(t["q_d"], t["k_d"], t["v_d"], t["q_g"], t["k_g"], t["v_g"], lam, o["o_d"], o["o_g"],
                    o["s_d"], o["s_g"], o["lse"], batch=B, **kw)
    atlas.diff_attn_bwd(t["q_d"], t["k_d"], t["v_d"], o["o_d"], o["s_d"], t["do_d"], t["q_g"], t["k_g"],
                        t["v_g"], o["o_g"], o["s_g"], t["do_g"], lam, o["lse"], o["dq_d"], o["dk_d"],
                        o["dv_d"], o["dq_g"], o["dk_g"], o["dv_g"], o["dlam"], work, batch=B, **kw)
    g.check()
    check_no_device_error()
    for n in want:
        assert torch.equal(o[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1), (301, 1, 1280, 10), (3, 1001, 60, 12), (2, 37, 5, 1),
                                  (7, 3, 256, 4), (1, 20011, 128, 32), (2, 600, 5120, 4), (300, 2000, 64, 1)],
                         ids=str)
def test_norm_writes_its_outputs_alone(case, dtype):
    S, R, C, K = case
    g, dt = Guarded(), DT[dtype]
    x, dy = rnd(S * R, C, dtype=dt), rnd(S * R, C, seed=1, dtype=dt)
    y, dx, stats = g.empty((S * R, C), dt), g.empty((S * R, C), dt), g.empty((S, K, 2))
    dg, db = g.empty((C,)), g.empty((C,))
    works = [g.empty((atlas.group_norm_workspace(x, R, K, b),), torch.uint8) for b in (False, True)]
    atlas.group_norm(x, None, None, y, R, K, activation="silu", stats=stats, workspace=works[0])
    atlas.group_norm_bwd(dy, x, None, None, stats, dx, dg, db, R, K, activation="silu", workspace=works[1])
    g.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_writes_its_rows_alone(layout, dtype):
    """Destinations that are columns of a wider buffer: its other columns, and what
    lies before and behind it, stay."""
    grid, cube, hd = (3, 17, 19), (2, 5, 8), 64
    rows, g, dt = int(np.prod(grid)), Guarded(), DT[dtype]
    wide = g.empty((rows, 7, hd), dt)
    wide.fill_(3.0)
    src = [inputs(rows, h, hd, dtype, seed=h) for h in (2, 3)]
    rot = atlas.make_rotary(10000.0, (10, 26, 20), layout=layout)
    for order in ("raster", "reorder", "unorder"):
        atlas.rotary([(src[0], wide[:, 1:3]), (src[1], wide[:, 3:6], False)], grid, rot, cube=cube, order=order)
        g.check()
        assert bool((wide[:, 0] == 3.0).all()) and bool((wide[:, 6] == 3.0).all())
