"""Rotary positions, general form, against a 64-bit reference (bounds in
diff_ref.py: one output rounding plus the fp32 rotation)."""
import numpy as np
import pytest
import torch

import diff_ref
from helpers import f64
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(rows, heads, hd, dtype, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(rows, heads, hd, generator=g, device=DEV).to(DT[dtype])


def grid_pos(grid, batch):
    p = np.stack(np.meshgrid(*(np.arange(e) for e in grid), indexing="ij"), -1).reshape(-1, 3)
    return np.tile(p, (batch, 1))


def expect(x, pos, dtype, order_rows, order, theta, split, scales, layout, transpose=False, **kw):
    """(reference, bound) of the call; x in the input's order."""
    mag = kw.get("magnitude", 1.0)
    x = f64(x)
    if order == "unorder":
        y = np.empty_like(x)
        y[order_rows] = x
        x = y
    y, err = diff_ref.rotary(x, pos, theta, split, scales, layout, transpose=transpose, **kw)
    rot = sum(split)
    err[..., :rot] += diff_ref.unit(DT[dtype]) * np.abs(y[..., :rot])
    if order == "reorder":
        y, err = y[order_rows], err[order_rows]
    assert mag > 0
    return torch.from_numpy(y), torch.from_numpy(err)


CASES = [
    # grid, cube, batch, hd, split, layout
    ((4, 8, 8), (2, 4, 4), 1, 64, (16, 24, 24), "interleaved"),
    ((4, 8, 8), (2, 4, 4), 1, 64, (16, 24, 24), "half"),
    ((3, 5, 7), (2, 4, 4), 2, 128, (44, 42, 42), "half"),
    ((3, 5, 7), (2, 4, 4), 3, 128, (44, 42, 42), "interleaved"),
    ((2, 3, 5), (4, 9, 9), 1, 96, (6, 10, 2), "half"),          # part of the head, cube over the grid
    ((2, 3, 5), (1, 1, 1), 1, 96, (6, 10, 2), "interleaved"),
    ((1, 1, 1), (1, 1, 1), 1, 32, (2, 0, 0), "half"),           # one token, one pair
    ((1, 1, 37), (1, 1, 5), 1, 8, (0, 0, 8), "interleaved"),
    ((1, 1, 3), (1, 1, 1), 1, 512, (512, 0, 0), "half"),        # the widest head
    ((2, 2, 2), (1, 1, 1), 1, 64, (0, 0, 0), "half"),           # nothing rotates
    ((7, 31, 33), (3, 16, 16), 1, 80, (26, 26, 26), "half"),    # several tiles per block
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["raster", "reorder", "unorder"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[3]}-{c[4]}-{c[5]}")
def test_against_reference(case, order, dtype):
    grid, cube, batch, hd, split, layout = case
    rows = batch * int(np.prod(grid))
    n = int(np.prod(grid))
    perm = np.concatenate([b * n + diff_ref.cube_rows(grid, cube) for b in range(batch)])
    rot = atlas.make_rotary(10000.0, split, (2.0, 1.0, 0.5), layout=layout, magnitude=1.25)
    src = [inputs(rows, h, hd, dtype, seed=h) for h in (3, 1, 2)]
    dst = [torch.full_like(s, 7.0) for s in src]
    atlas.rotary([(src[0], dst[0]), (src[1], dst[1]), (src[2], dst[2], False)], grid, rot, cube=cube,
                 order=order, batch=batch)
    pos = grid_pos(grid, batch)
    for s, d in zip(src[:2], dst[:2]):
        want, bound = expect(s, pos, dtype, perm, order, 10000.0, split, (2.0, 1.0, 0.5), layout,
                             magnitude=1.25)
        diff_ref.check("y", f64(d), want, bound)
        tail = sum(split)   # the channels behind the rotated part: bit-exact
        plain = s if order == "raster" else torch.empty_like(s)
        if order == "reorder":
            plain = s[torch.from_numpy(perm).to(DEV)]
        if order == "unorder":
            plain[torch.from_numpy(perm).to(DEV)] = s
        assert torch.equal(d[..., tail:], plain[..., tail:])
    moved = src[2] if order == "raster" else torch.empty_like(src[2])
    if order == "reorder":
        moved = src[2][torch.from_numpy(perm).to(DEV)]
    if order == "unorder":
        moved[torch.from_numpy(perm).to(DEV)] = src[2]
    assert torch.equal(dst[2], moved)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("scaling", ["none", "ntk", "by_parts"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_positions_and_scaling(layout, scaling, dtype):
    """Positions per token: negative, zero, far beyond 2^24; scaled frequencies."""
    rows, hd, split = 53, 64, (32, 12, 4)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-1000, 200000, (rows, 3), generator=g, dtype=torch.int32)
    pos[0] = torch.tensor([0, 0, 0])
    pos[1] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1])
    kw = dict(scaling=scaling, factor=(8.0, 2.0, 1.0), original=(4096.0, 64.0, 16.0),
              magnitude=1.2)
    rot = atlas.make_rotary(10000.0, split, (1.0, 4.0, 1.0), layout=layout, **kw)
    x = inputs(rows, 2, hd, dtype)
    y = torch.empty_like(x)
    atlas.rotary([(x, y)], (1, 1, rows), rot, positions=pos.to(DEV))
    want, bound = expect(x, pos.numpy().astype(np.float64), dtype, None, "raster", 10000.0, split,
                         (1.0, 4.0, 1.0), layout, **kw)
    diff_ref.check("y", f64(y), want, bound)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradient(layout):
    """transpose is the gradient: against the formula, and against differences
    of the forward call (linear in x, so a difference is exact up to rounding)."""
    grid, hd, split = (2, 3, 4), 32, (8, 6, 10)
    rows = 24
    rot = atlas.make_rotary(100.0, split, layout=layout, magnitude=1.1)
    cube = (1, 2, 3)
    perm = diff_ref.cube_rows(grid, cube)
    x, dy = inputs(rows, 2, hd, "fp32", 1), inputs(rows, 2, hd, "fp32", 2)
    dx = torch.empty_like(x)
    atlas.rotary([(dy, dx)], grid, rot, cube=cube, order="unorder", transpose=True)
    want, bound = expect(dy, grid_pos(grid, 1), "fp32", perm, "unorder", 100.0, split, (1, 1, 1), layout,
                         transpose=True, magnitude=1.1)
    diff_ref.check("dx", f64(dx), want, bound)

    def loss(v):
        y = torch.empty_like(v)
        atlas.rotary([(v, y)], grid, rot, cube=cube, order="reorder")
        return float((y.double() * dy.double()).sum())

    for row, head, c in ((0, 0, 0), (5, 1, 9), (23, 0, 31), (11, 1, 20)):
        e = torch.zeros_like(x)
        e[row, head, c] = 1.0
        # <dy, R e> with coefficients of 2^-20 relative error, a sum of two terms
        assert abs(loss(e) - float(dx[row, head, c])) <= 2.0 ** -18 * 1.1 * float(dy.abs().max())


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_slices_and_in_place(layout, dtype):
    """Q, K, V as column slices of one fused buffer: out of it, and in place in it."""
    rows, hd, split = 39, 64, (20, 18, 22)
    grid = (3, 13, 1)
    whole = inputs(rows, 7, hd, dtype)
    parts = [whole[:, 0:4], whole[:, 4:6], whole[:, 6:7]]
    rot = atlas.make_rotary(10000.0, split, layout=layout)
    out = [torch.empty(rows, p.shape[1], hd, dtype=whole.dtype, device=DEV) for p in parts]
    atlas.rotary([(parts[0], out[0]), (parts[1], out[1]), (parts[2], out[2], False)], grid, rot)
    for p, o in zip(parts[:2], out[:2]):
        want, bound = expect(p, grid_pos(grid, 1), dtype, None, "raster", 10000.0, split, (1, 1, 1), layout)
        diff_ref.check("y", f64(o), want, bound)
    assert torch.equal(out[2], parts[2])
    atlas.rotary([(parts[0], parts[0]), (parts[1], parts[1]), (parts[2], parts[2], False)], grid, rot)
    for p, o in zip(parts, out):
        assert torch.equal(p, o)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_non_finite_stays_in_its_pair(layout):
    """Inf and NaN in a channel reach its pair and nothing else; unrotated
    channels keep their bits, NaN payloads included."""
    rows, hd, split = 8, 32, (6, 4, 6)
    x = torch.ones(rows, 1, hd, device=DEV, dtype=torch.bfloat16)
    x[3, 0, 0] = float("inf")
    x.view(torch.int16)[4, 0, 20] = 0x7fc5
    y = torch.empty_like(x)
    rot = atlas.make_rotary(10000.0, split, layout=layout)
    atlas.rotary([(x, y)], (2, 2, 2), rot)
    bad = ~torch.isfinite(y.float())
    partner = 1 if layout == "interleaved" else 3
    assert bad[3, 0, 0] and bad[3, 0, partner]
    bad[3, 0, 0] = bad[3, 0, partner] = bad[4, 0, 20] = False
    assert not bad.any()
    assert int(y.view(torch.int16)[4, 0, 20]) == 0x7fc5


def test_matches_the_framework_rope():
    """INTERLEAVED over the whole head is atlas_rope3d / atlas_cube_reorder up
    to their coefficients' fp32 roundings."""
    grid, cube, hd, split = (4, 8, 8), (2, 4, 4), 64, (16, 24, 24)
    x = inputs(256, 2, hd, "fp32")
    a, b = torch.empty_like(x), torch.empty_like(x)
    atlas.cube_reorder(x, a, grid, cube, atlas.make_rope(10000.0, split, (4.0, 1.0, 1.0)))
    atlas.rotary([(x, b)], grid, atlas.make_rotary(10000.0, split, (4.0, 1.0, 1.0)), cube=cube,
                 order="reorder")
    assert float((a - b).abs().max()) <= 2.0 ** -19 * 2 * float(x.abs().max())


def test_streams_and_graph():
    """Captured without a first call, replayed on new inputs; a side stream."""
    grid, hd, split = (3, 5, 7), 128, (44, 42, 42)
    rot = atlas.make_rotary(10000.0, split, layout="half")
    x = inputs(105, 2, hd, "bf16")
    y, z = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        atlas.rotary([(x, y)], grid, rot, cube=(2, 4, 4), order="reorder")
    x.copy_(inputs(105, 2, hd, "bf16", seed=9))
    g.replay()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    atlas.rotary([(x, z)], grid, rot, cube=(2, 4, 4), order="reorder", stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_small_part_of_a_wide_head(layout, dtype):
    """A quarter of a 512-channel head rotates, in many tiles: the vectors behind
    the rotated part touch no coefficient."""
    rows, hd, split = 12000, 512, (128, 0, 0)
    rot = atlas.make_rotary(10000.0, split, layout=layout)
    x = inputs(rows, 1, hd, dtype)
    y = torch.empty_like(x)
    atlas.rotary([(x, y)], (1, 1, rows), rot, positions=torch.arange(rows, dtype=torch.int32, device=DEV))
    pick = torch.tensor([0, 1, 31, 32, 5000, 11999])
    pos = np.zeros((len(pick), 3))
    pos[:, 0] = pick.numpy()
    want, bound = expect(x[pick], pos, dtype, None, "raster", 10000.0, split, (1, 1, 1), layout)
    diff_ref.check("y", f64(y[pick]), want, bound)
    assert torch.equal(y[..., 128:], x[..., 128:])
