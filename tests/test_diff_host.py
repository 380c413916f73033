"""Refusals of the differential-attention layer's calls (no GPU needed): every
case fails validation before any CUDA call; fake pointers are never read."""
import ctypes

import pytest
import torch

from video_dit_windowed_b200 import atlas, build

FAKE = 0x7F0000000000
STEP = 1 << 32
E = atlas


@pytest.fixture(scope="module")
def lib():
    build.build()
    return atlas.lib()


def at(i):
    return FAKE + i * STEP


# ---- rotary ------------------------------------------------------------------

def rotary(lib, tensors=None, batch=1, grid=(2, 3, 5), cube=(1, 2, 2), order=1, positions=None, axes=0,
           hd=64, dtype=atlas.BF16, n=None, rot=None, **kw):
    tensors = tensors if tensors is not None else [dict()]
    items = (atlas.RotaryTensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        d = dict(src=at(2 * i), dst=at(2 * i + 1), src_stride=0, dst_stride=0, heads=2, rotate=1)
        d.update(t)
        for k, v in d.items():
            setattr(items[i], k, v)
    r = atlas.make_rotary(10000.0, (16, 24, 24), **kw) if rot is None else rot
    return lib.atlas_rotary_apply(items, len(tensors) if n is None else n, batch, atlas.Grid3(*grid),
                                  ctypes.byref(atlas.Cube3(*cube)) if cube else None, order, positions,
                                  axes, hd, dtype, ctypes.byref(r), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tensors=[dict(src=None)]), E.ERR_NULL),
    (dict(tensors=[dict(dst=None)]), E.ERR_NULL),
    (dict(cube=None), E.ERR_NULL),
    (dict(n=0), E.ERR_SHAPE),
    (dict(n=9), E.ERR_SHAPE),
    (dict(batch=0), E.ERR_SHAPE),
    (dict(batch=1 << 31), E.ERR_SHAPE),
    (dict(grid=(0, 1, 1)), E.ERR_SHAPE),
    (dict(grid=(1 << 20, 1 << 10, 4)), E.ERR_SHAPE),
    (dict(cube=(0, 1, 1)), E.ERR_SHAPE),
    (dict(tensors=[dict(heads=0)]), E.ERR_SHAPE),
    (dict(tensors=[dict(heads=65536)]), E.ERR_SHAPE),
    (dict(tensors=[dict(src_stride=64)]), E.ERR_SHAPE),
    (dict(tensors=[dict(dst_stride=-128)]), E.ERR_SHAPE),
    (dict(tensors=[dict(src_stride=130)]), E.ERR_ALIGN),
    (dict(tensors=[dict(src=FAKE + 8)]), E.ERR_ALIGN),
    (dict(tensors=[dict(dst=at(1) + 2)]), E.ERR_ALIGN),
    (dict(hd=60), E.ERR_ALIGN),
    (dict(positions=at(20) + 2, axes=3), E.ERR_ALIGN),
    (dict(hd=576), E.ERR_UNSUPPORTED),
    (dict(dtype=5), E.ERR_UNSUPPORTED),
    (dict(order=3), E.ERR_UNSUPPORTED),
    (dict(positions=at(20), axes=2), E.ERR_UNSUPPORTED),
    (dict(positions=at(20), axes=1), E.ERR_UNSUPPORTED),   # d_h and d_w need their own positions
    (dict(hd=32), E.ERR_UNSUPPORTED),                      # 64 channels rotate
    (dict(scaling="ntk", factor=(0.5, 1, 1)), E.ERR_UNSUPPORTED),
    (dict(scaling="ntk", factor=(1, float("nan"), 1)), E.ERR_UNSUPPORTED),
    (dict(scaling="by_parts", original=(0, 1, 1)), E.ERR_UNSUPPORTED),
    (dict(scaling="by_parts", original=(8, 8, 8), beta_fast=1.0, beta_slow=1.0), E.ERR_UNSUPPORTED),
    (dict(magnitude=float("inf")), E.ERR_UNSUPPORTED),
    (dict(rot=atlas.make_rotary(0.0, (16, 24, 24))), E.ERR_UNSUPPORTED),
    (dict(rot=atlas.make_rotary(1e4, (15, 24, 24))), E.ERR_UNSUPPORTED),
    (dict(rot=atlas.make_rotary(1e4, (-2, 24, 24))), E.ERR_UNSUPPORTED),
    (dict(rot=atlas.make_rotary(1e4, (2, 2, 2), (float("nan"), 1, 1))), E.ERR_UNSUPPORTED),
    (dict(tensors=[dict(dst=at(0))]), E.ERR_ALIAS),                       # reorder in place
    (dict(order=0, tensors=[dict(dst=at(0), src_stride=256)]), E.ERR_ALIAS),
    (dict(tensors=[dict(), dict(dst=at(1))]), E.ERR_ALIAS),               # two destinations
    (dict(tensors=[dict(), dict(src=at(1) + 1024)]), E.ERR_ALIAS),        # one reads what another writes
    (dict(order=0, tensors=[dict(dst=at(0) + 128, src_stride=384, dst_stride=384)]), E.ERR_ALIAS),
    (dict(positions=at(1) + 64, axes=3), E.ERR_ALIAS),
], ids=str)
def test_rotary_refusals(lib, kw, status):
    assert rotary(lib, **kw) == status


def test_rotary_layout_and_scaling_codes(lib):
    for field in ("layout", "scaling"):
        r = atlas.make_rotary(1e4, (16, 24, 24))
        setattr(r, field, 9)
        assert rotary(lib, rot=r) == atlas.ERR_UNSUPPORTED


def test_rotary_accepts_columns_of_one_buffer(lib):
    """Disjoint columns of one buffer are no overlap: past the checks, the call
    stops only at the missing device."""
    cols = [dict(src=FAKE + i * 256, dst=FAKE + i * 256, src_stride=384, dst_stride=384, heads=2)
            for i in range(3)]
    if not torch.cuda.is_available():
        assert rotary(lib, tensors=cols, order=0) == atlas.ERR_DEVICE


# ---- differential attention ----------------------------------------------------

def diff(lib, bwd=False, n_d=64, n_g=32, heads=2, hd=64, L=32, dtype=atlas.BF16, n_lam=2, layout=True,
         scale=0.0, batch=1, offsets=None, n_win=0, shares=None, **over):
    names = ["q_d", "k_d", "v_d", "o_d", "s_d", "do_d", "q_g", "k_g", "v_g", "o_g", "s_g", "do_g",
             "lam", "lse", "work", "dq_d", "dk_d", "dv_d", "dq_g", "dk_g", "dv_g", "dlam"]
    p = {n: at(i) for i, n in enumerate(names)}
    p.update(over)
    ly = atlas.AttnLayout(batch, L, offsets, n_win, shares)
    lyp = ctypes.byref(ly) if layout else None
    if not bwd:
        return lib.atlas_diff_attn(p["q_d"], p["k_d"], p["v_d"], n_d, p["q_g"], p["k_g"], p["v_g"], n_g,
                                   lyp, heads, hd, scale, dtype, p["lam"], n_lam, p["o_d"], p["o_g"],
                                   p["s_d"], p["s_g"], p["lse"], None)
    return lib.atlas_diff_attn_bwd(p["q_d"], p["k_d"], p["v_d"], p["o_d"], p["s_d"], p["do_d"], n_d,
                                   p["q_g"], p["k_g"], p["v_g"], p["o_g"], p["s_g"], p["do_g"], n_g, lyp,
                                   heads, hd, scale, dtype, p["lam"], n_lam, p["lse"], p["work"],
                                   p["dq_d"], p["dk_d"], p["dv_d"], p["dq_g"], p["dk_g"], p["dv_g"],
                                   p["dlam"], None)


BOTH = [
    (dict(layout=False), E.ERR_NULL),
    (dict(lam=None), E.ERR_NULL),
    (dict(q_d=None), E.ERR_NULL),
    (dict(v_g=None), E.ERR_NULL),
    (dict(o_d=None), E.ERR_NULL),
    (dict(n_lam=3), E.ERR_SHAPE),
    (dict(n_lam=0), E.ERR_SHAPE),
    (dict(L=48), E.ERR_SHAPE),
    (dict(n_d=-1), E.ERR_SHAPE),
    (dict(batch=0), E.ERR_SHAPE),
    (dict(heads=0), E.ERR_SHAPE),
    (dict(offsets=at(40), n_win=65), E.ERR_SHAPE),
    (dict(offsets=at(40) + 2, n_win=3), E.ERR_ALIGN),
    (dict(shares=at(41), n_win=5), E.ERR_SHAPE),
    (dict(hd=96), E.ERR_UNSUPPORTED),
    (dict(hd=32), E.ERR_UNSUPPORTED),
    (dict(dtype=3), E.ERR_UNSUPPORTED),
    (dict(scale=float("inf")), E.ERR_UNSUPPORTED),
    (dict(lam=at(12) + 2), E.ERR_ALIGN),
    (dict(q_d=at(0) + 8), E.ERR_ALIGN),
    (dict(o_g=at(9) + 8), E.ERR_ALIGN),
    (dict(lse=at(13) + 1), E.ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", BOTH, ids=str)
@pytest.mark.parametrize("bwd", [False, True])
def test_diff_refusals(lib, kw, status, bwd):
    assert diff(lib, bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(s_d=None), E.ERR_NULL),                        # one of the two sides
    (dict(o_d=at(0)), E.ERR_ALIAS),
    (dict(o_d=at(9)), E.ERR_ALIAS),
    (dict(s_g=at(4)), E.ERR_ALIAS),
    (dict(lse=at(3)), E.ERR_ALIAS),
    (dict(lse=at(12)), E.ERR_ALIAS),
    (dict(o_d=at(40), offsets=at(40), n_win=3), E.ERR_ALIAS),
], ids=str)
def test_diff_forward_refusals(lib, kw, status):
    assert diff(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), E.ERR_NULL),
    (dict(work=None), E.ERR_NULL),
    (dict(dlam=None), E.ERR_NULL),
    (dict(s_d=None), E.ERR_NULL),
    (dict(dv_g=None), E.ERR_NULL),
    (dict(work=at(14) + 4), E.ERR_ALIGN),
    (dict(dq_d=at(15) + 8), E.ERR_ALIGN),
    (dict(dlam=at(21) + 2), E.ERR_ALIGN),
    (dict(dq_d=at(0)), E.ERR_ALIAS),
    (dict(dk_g=at(17)), E.ERR_ALIAS),
    (dict(work=at(13)), E.ERR_ALIAS),
    (dict(dlam=at(12)), E.ERR_ALIAS),
    (dict(dlam=at(14) + 64), E.ERR_ALIAS),
], ids=str)
def test_diff_backward_refusals(lib, kw, status):
    assert diff(lib, True, **kw) == status


def test_diff_workspace(lib):
    rows = 4 * (2 * 2 * 3 * 107 + 3 * 64)
    assert atlas.diff_attn_bwd_workspace(2, 100, 7, 3, 64, atlas.FP32) == rows
    assert atlas.diff_attn_bwd_workspace(2, 100, 7, 3, 64, atlas.BF16) == rows   # too short to cut
    # 40 long units of one head: cut into parts of dV and dK sums
    base, cut = 4 * (2 * 85680 + 64), 4 * 5040 * 2 * 128
    for dtype in (atlas.BF16, atlas.FP32):
        extra = atlas.diff_attn_bwd_workspace(1, 80640, 5040, 1, 128, dtype) - base
        assert extra > cut and extra % cut == 0
    for bad in ((0, 1, 1, 1, 64), (1, -1, 1, 1, 64), (1, 1, 1, 0, 64), (1, 1 << 31, 0, 1, 64),
                (2, 1 << 30, 0, 1, 64), (1, 1, 1, 1, 32)):
        assert atlas.diff_attn_bwd_workspace(*bad, atlas.BF16) == 0
    assert atlas.diff_attn_bwd_workspace(1, 1, 1, 1, 64, 7) == 0


def test_lambda_refusals(lib):
    def fwd(v=(at(0), at(1), at(2), at(3)), n=2, d=32, init=0.5, dt=atlas.BF16, lam=at(4)):
        return lib.atlas_diff_lambda(*v, n, d, init, dt, lam, None)

    def bwd(dl=at(4), dv=(at(5), at(6), at(7), at(8)), dt=atlas.FP32, n=2, d=32):
        return lib.atlas_diff_lambda_bwd(at(0), at(1), at(2), at(3), n, d, dl, dt, *dv, None)

    assert fwd(v=(at(0), None, at(2), at(3))) == E.ERR_NULL
    assert fwd(lam=None) == E.ERR_NULL
    assert fwd(n=0) == E.ERR_SHAPE and fwd(d=0) == E.ERR_SHAPE
    assert fwd(dt=7) == E.ERR_UNSUPPORTED and fwd(init=float("nan")) == E.ERR_UNSUPPORTED
    assert fwd(lam=at(4) + 2) == E.ERR_ALIGN and fwd(v=(at(0) + 1, at(1), at(2), at(3))) == E.ERR_ALIGN
    assert fwd(lam=at(1) + 4) == E.ERR_ALIAS
    assert bwd(dl=None) == E.ERR_NULL and bwd(dv=(None, at(6), at(7), at(8))) == E.ERR_NULL
    assert bwd(dv=(at(5) + 2, at(6), at(7), at(8))) == E.ERR_ALIGN
    assert bwd(dv=(at(0), at(6), at(7), at(8))) == E.ERR_ALIAS
    assert bwd(dv=(at(5), at(5), at(7), at(8))) == E.ERR_ALIAS
    assert bwd(n=0) == E.ERR_SHAPE


# ---- group norm -----------------------------------------------------------------

def norm(lib, bwd=False, samples=2, rows=8, channels=64, groups=4, eps=1e-5, act=1, dtype=atlas.BF16,
         **over):
    names = ["x", "gamma", "beta", "y", "stats", "work", "dy", "dgamma", "dbeta"]
    p = {n: at(i) for i, n in enumerate(names)}
    p.update(over)
    if not bwd:
        return lib.atlas_group_norm(p["x"], p["gamma"], p["beta"], p["y"], samples, rows, channels, groups,
                                    eps, act, dtype, p["stats"], p["work"], None)
    return lib.atlas_group_norm_bwd(p["dy"], p["x"], p["gamma"], p["beta"], p["stats"], p["y"],
                                    p["dgamma"], p["dbeta"], samples, rows, channels, groups, act, dtype,
                                    p["work"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), E.ERR_NULL),
    (dict(y=None), E.ERR_NULL),
    (dict(samples=0), E.ERR_SHAPE),
    (dict(rows=0), E.ERR_SHAPE),
    (dict(channels=0), E.ERR_SHAPE),
    (dict(groups=0), E.ERR_SHAPE),
    (dict(groups=5), E.ERR_SHAPE),
    (dict(samples=1 << 20, rows=1 << 12), E.ERR_SHAPE),
    (dict(channels=1 << 32), E.ERR_SHAPE),
    (dict(dtype=4), E.ERR_UNSUPPORTED),
    (dict(act=2), E.ERR_UNSUPPORTED),
    (dict(x=at(0) + 8), E.ERR_ALIGN),
    (dict(gamma=at(1) + 2), E.ERR_ALIGN),
    (dict(stats=at(4) + 2), E.ERR_ALIGN),
    (dict(y=at(0) + 16), E.ERR_ALIAS),
    (dict(y=at(1)), E.ERR_ALIAS),
    (dict(y=at(4)), E.ERR_ALIAS),
], ids=str)
def test_norm_refusals(lib, kw, status, bwd):
    assert norm(lib, bwd, **kw) == status


def test_norm_more_refusals(lib):
    assert norm(lib, eps=-1.0) == E.ERR_UNSUPPORTED and norm(lib, eps=float("nan")) == E.ERR_UNSUPPORTED
    assert norm(lib, stats=at(0)) == E.ERR_ALIAS
    assert norm(lib, True, dy=None) == E.ERR_NULL and norm(lib, True, stats=None) == E.ERR_NULL
    assert norm(lib, True, dgamma=at(8)) == E.ERR_ALIAS and norm(lib, True, dbeta=at(0)) == E.ERR_ALIAS
    assert norm(lib, True, dgamma=at(7) + 1) == E.ERR_ALIGN


# ---- the binding's own checks (host tensors are refused before anything runs) ---

def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        atlas.rotary([(x, x)], (1, 1, 4), atlas.make_rotary(1e4, (64, 0, 0)))
    with pytest.raises(ValueError):
        atlas.diff_attn(None, None, None, x, x, x, torch.ones(2), None, x)
    with pytest.raises(ValueError):
        atlas.diff_lambda(x[0], x[0], x[0], x[0], 0.5, torch.ones(2))
    with pytest.raises(ValueError):
        atlas.group_norm(x[:, 0], None, None, x[:, 0], 1, 1)


def test_rotary_rows_of_a_tensor():
    """Row strides as the library takes them: 0 there means contiguous, so a tensor
    whose rows share memory is refused."""
    x = torch.zeros(6, 3, 8)
    assert atlas._rows(x)[1] == 24 and atlas._rows(x[:, 1:])[1] == 24 and atlas._rows(x[::2])[1] == 48
    assert atlas._rows(x[:1].expand(1, 3, 8))[1] == 24
    for bad in (x[:1].expand(6, 3, 8), x[:, :1].expand(6, 3, 8), x.transpose(0, 1), x[..., ::2],
                x.as_strided((6, 3, 8), (8, 8, 1))):
        with pytest.raises(ValueError):
            atlas._rows(bad)
