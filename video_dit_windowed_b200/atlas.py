"""ctypes binding of ``libatlas.so`` (declared in ``include/atlas.h``).

Argument marshalling only: shapes, dtypes and device pointers are read off
torch tensors (torch is used for device memory and streams) and passed to the
C-ABI; every step of the path runs in the library's CUDA kernels. There is no
CPU fallback: if the library has not been built, the first call raises.

Passages (page title, section) for each call are given in the header; in
short: "Technische Samenvatting: AtlasVid" (gist.science), Methodologie 1
Fase 1 (temporally scaled RoPE), Fase 2 (cube reorder, window attention) and
Methodologie 2 (asymmetric hierarchical attention, position alignment).
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; ATLAS_LIBRARY may name another build of the same C-ABI.
LIB_PATH = os.environ.get("ATLAS_LIBRARY") or os.path.join(HERE, "libatlas.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_ALIAS, ERR_CUDA, \
    ERR_TIMEOUT, ERR_DEVICE, ERR_CAPACITY = range(10)
BF16, FP32 = 0, 1


class Grid3(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("W", ctypes.c_int64)]


class Cube3(ctypes.Structure):
    _fields_ = [("ct", ctypes.c_int32), ("ch", ctypes.c_int32), ("cw", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_double), ("d_t", ctypes.c_int32), ("d_h", ctypes.c_int32),
                ("d_w", ctypes.c_int32), ("scale_t", ctypes.c_double),
                ("scale_h", ctypes.c_double), ("scale_w", ctypes.c_double)]


class AttnLayout(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("window_len", ctypes.c_int64),
                ("window_offsets", ctypes.c_void_p), ("n_windows", ctypes.c_int64),
                ("global_window_offsets", ctypes.c_void_p)]


class Rotary(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_double), ("d_t", ctypes.c_int32), ("d_h", ctypes.c_int32),
                ("d_w", ctypes.c_int32), ("scale_t", ctypes.c_double),
                ("scale_h", ctypes.c_double), ("scale_w", ctypes.c_double),
                ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("factor_t", ctypes.c_double), ("factor_h", ctypes.c_double),
                ("factor_w", ctypes.c_double), ("original_t", ctypes.c_double),
                ("original_h", ctypes.c_double), ("original_w", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("magnitude", ctypes.c_double), ("transpose", ctypes.c_int32)]


class RotaryTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p),
                ("src_stride", ctypes.c_int64), ("dst_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("rotate", ctypes.c_int32)]


ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}
ROTARY_SCALINGS = {"none": 0, "ntk": 1, "by_parts": 2}
ORDERS = {"raster": 0, "reorder": 1, "unorder": 2}
ACTIVATIONS = {"none": 0, "silu": 1}


def make_rotary(theta, split, scales=(1.0, 1.0, 1.0), *, layout="interleaved", scaling="none",
                factor=(1.0, 1.0, 1.0), original=(0.0, 0.0, 0.0), beta_fast=32.0, beta_slow=1.0,
                magnitude=1.0) -> Rotary:
    """Parameters of ``rotary``: ``split`` (d_t, d_h, d_w) channels rotate (the
    first ones of a head), positions are multiplied by ``scales``; ``layout``
    "interleaved" or "half"; ``scaling`` "none", "ntk" or "by_parts" with the
    axes' extension ``factor`` and trained lengths ``original``."""
    return Rotary(float(theta), *(int(v) for v in split), *(float(v) for v in scales),
                  ROTARY_LAYOUTS[layout], ROTARY_SCALINGS[scaling], *(float(v) for v in factor),
                  *(float(v) for v in original), float(beta_fast), float(beta_slow),
                  float(magnitude), 0)


def make_rope(theta, split, scales) -> Rope:
    d_t, d_h, d_w = (int(v) for v in split)
    s_t, s_h, s_w = (float(v) for v in scales)
    return Rope(float(theta), d_t, d_h, d_w, s_t, s_h, s_w)


class AtlasError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


def _declare(lib):
    lib.atlas_cube_reorder.restype = ctypes.c_int
    lib.atlas_cube_reorder.argtypes = [_vp, _vp, Grid3, Cube3, _i32, _i32, ctypes.c_int,
                                       ctypes.POINTER(Rope), _vp]
    lib.atlas_cube_reorder_noalloc.restype = ctypes.c_int
    lib.atlas_cube_reorder_noalloc.argtypes = lib.atlas_cube_reorder.argtypes
    lib.atlas_cube_unorder.restype = ctypes.c_int
    lib.atlas_cube_unorder.argtypes = [_vp, _vp, Grid3, Cube3, _i32, _i32, ctypes.c_int, _vp]
    lib.atlas_rope3d.restype = ctypes.c_int
    lib.atlas_rope3d.argtypes = [_vp, _vp, Grid3, _i32, _i32, ctypes.c_int,
                                 ctypes.POINTER(Rope), _vp]
    lib.atlas_local_global_attn.restype = ctypes.c_int
    lib.atlas_local_global_attn.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64,
                                            _i32, _i32, ctypes.c_float, ctypes.c_int, _vp, _vp,
                                            _vp, _vp]
    lib.atlas_local_global_attn_windows.restype = ctypes.c_int
    lib.atlas_local_global_attn_windows.argtypes = [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                                    _i64, _i32, _i32, ctypes.c_float, ctypes.c_int,
                                                    _vp, _vp, _vp, _vp]
    lib.atlas_local_global_attn_ex.restype = ctypes.c_int
    lib.atlas_local_global_attn_ex.argtypes = [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64,
                                               ctypes.POINTER(AttnLayout), _i32, _i32,
                                               ctypes.c_float, ctypes.c_int, _vp, _vp, _vp, _vp]
    lib.atlas_local_global_attn_bwd.restype = ctypes.c_int
    lib.atlas_local_global_attn_bwd.argtypes = (
        [_vp] * 5 + [_i64] + [_vp] * 5 + [_i64, ctypes.POINTER(AttnLayout), _i32, _i32,
                                         ctypes.c_float, ctypes.c_int, _vp, _vp] + [_vp] * 7)
    lib.atlas_qkv_proj_reorder.restype = ctypes.c_int
    lib.atlas_qkv_proj_reorder.argtypes = [_vp, _vp, _i64, Grid3, Cube3, _i32, _i32, _i32,
                                           ctypes.c_int, ctypes.POINTER(Rope), _vp, _vp, _vp,
                                           _vp]
    lib.atlas_out_proj_unorder.restype = ctypes.c_int
    lib.atlas_out_proj_unorder.argtypes = [_vp, _vp, _i64, Grid3, Cube3, _i32, _i32,
                                           ctypes.c_int, _vp, _vp]
    for name in ("atlas_aligned_global_reorder", "atlas_aligned_global_unorder"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [_vp, _vp, _i64, Grid3, Cube3, Grid3, _i32, _i32, ctypes.c_int,
                       ctypes.POINTER(Rope), _vp]
    lib.atlas_aligned_global_offsets.restype = ctypes.c_int
    lib.atlas_aligned_global_offsets.argtypes = [Grid3, Cube3, Grid3, _vp, _i64,
                                                 ctypes.POINTER(_i64)]
    lib.atlas_aligned_global_cube.restype = ctypes.c_int
    lib.atlas_aligned_global_cube.argtypes = [Grid3, Cube3, Grid3, ctypes.POINTER(Cube3)]
    lib.atlas_cube_reorder_batched.restype = ctypes.c_int
    lib.atlas_cube_reorder_batched.argtypes = [_vp, _vp, _i64, Grid3, Cube3, _i32, _i32,
                                               ctypes.c_int, ctypes.POINTER(Rope), _vp]
    lib.atlas_cube_unorder_batched.restype = ctypes.c_int
    lib.atlas_cube_unorder_batched.argtypes = [_vp, _vp, _i64, Grid3, Cube3, _i32, _i32,
                                               ctypes.c_int, _vp]
    lib.atlas_cube_unorder_rope.restype = ctypes.c_int
    lib.atlas_cube_unorder_rope.argtypes = [_vp, _vp, _i64, Grid3, Cube3, _i32, _i32,
                                            ctypes.c_int, ctypes.POINTER(Rope), _vp]
    lib.atlas_rope3d_batched.restype = ctypes.c_int
    lib.atlas_rope3d_batched.argtypes = [_vp, _vp, _i64, Grid3, _i32, _i32, ctypes.c_int,
                                         ctypes.POINTER(Rope), _vp]
    lib.atlas_rotary_apply.restype = ctypes.c_int
    lib.atlas_rotary_apply.argtypes = [ctypes.POINTER(RotaryTensor), _i32, _i64, Grid3,
                                       ctypes.POINTER(Cube3), ctypes.c_int, _vp, _i32, _i32,
                                       ctypes.c_int, ctypes.POINTER(Rotary), _vp]
    lib.atlas_diff_lambda.restype = ctypes.c_int
    lib.atlas_diff_lambda.argtypes = [_vp] * 4 + [_i32, _i32, ctypes.c_double, ctypes.c_int, _vp,
                                                  _vp]
    lib.atlas_diff_lambda_bwd.restype = ctypes.c_int
    lib.atlas_diff_lambda_bwd.argtypes = [_vp] * 4 + [_i32, _i32, _vp, ctypes.c_int] + [_vp] * 5
    lib.atlas_diff_attn.restype = ctypes.c_int
    lib.atlas_diff_attn.argtypes = [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64,
                                    ctypes.POINTER(AttnLayout), _i32, _i32, ctypes.c_float,
                                    ctypes.c_int, _vp, _i32] + [_vp] * 6
    lib.atlas_diff_attn_bwd.restype = ctypes.c_int
    lib.atlas_diff_attn_bwd.argtypes = (
        [_vp] * 6 + [_i64] + [_vp] * 6 + [_i64, ctypes.POINTER(AttnLayout), _i32, _i32,
                                         ctypes.c_float, ctypes.c_int, _vp, _i32] + [_vp] * 10)
    lib.atlas_diff_attn_bwd_workspace.restype = _i64
    lib.atlas_diff_attn_bwd_workspace.argtypes = [_i64, _i64, _i64, _i32, _i32, ctypes.c_int]
    lib.atlas_group_norm.restype = ctypes.c_int
    lib.atlas_group_norm.argtypes = [_vp] * 4 + [_i64, _i64, _i64, _i32, ctypes.c_double,
                                                 ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]
    lib.atlas_group_norm_bwd.restype = ctypes.c_int
    lib.atlas_group_norm_bwd.argtypes = [_vp] * 8 + [_i64, _i64, _i64, _i32, ctypes.c_int,
                                                     ctypes.c_int, _vp, _vp]
    lib.atlas_group_norm_workspace.restype = _i64
    lib.atlas_group_norm_workspace.argtypes = [_i64, _i64, _i64, _i32, ctypes.c_int, _i32]
    lib.atlas_cube_window_offsets.restype = ctypes.c_int
    lib.atlas_cube_window_offsets.argtypes = [Grid3, Cube3, _vp, _i64, ctypes.POINTER(_i64)]
    lib.atlas_status_string.restype = ctypes.c_char_p
    lib.atlas_status_string.argtypes = [ctypes.c_int]
    lib.atlas_last_device_error.restype = ctypes.c_int
    lib.atlas_last_device_error.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.atlas_debug_stall_next_attention.restype = ctypes.c_int
    lib.atlas_debug_stall_next_attention.argtypes = []
    lib.atlas_release_caches.restype = ctypes.c_int
    lib.atlas_release_caches.argtypes = []
    lib.atlas_cached_rope_tables.restype = ctypes.c_int64
    lib.atlas_cached_rope_tables.argtypes = []
    lib.atlas_version.restype = ctypes.c_int32
    lib.atlas_version.argtypes = []
    return lib


def lib():
    """The loaded library. Raises if ``libatlas.so`` has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m video_dit_windowed_b200.build` (no CPU fallback exists)")
            _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    return lib().atlas_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise AtlasError(status, where)


# ---------------------------------------------------------------------------
# torch-facing wrappers (torch only supplies pointers, shapes and streams)
# ---------------------------------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(t, stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def cube_reorder(src, dst, grid, cube, rope: Rope | None = None, stream=None):
    """Raster -> cube order of ``src`` [T*H*W, heads, head_dim] into ``dst``;
    with ``rope`` the rows are also rotated by 3D RoPE at their grid position."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_reorder(
        _ptr(src), _ptr(dst), Grid3(*grid), Cube3(*cube), heads, hd, _dtype_code(src),
        ctypes.byref(rope) if rope is not None else None, _stream(src, stream))
    _check(st, "atlas_cube_reorder")
    return dst


def cube_reorder_noalloc(src, dst, grid, cube, rope: Rope | None = None, stream=None):
    """``cube_reorder`` through the entry point that allocates no device
    memory (its RoPE table sits in a fixed 32768-pair array shared by all
    calls on the device; overlapping calls race, see include/atlas.h)."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_reorder_noalloc(
        _ptr(src), _ptr(dst), Grid3(*grid), Cube3(*cube), heads, hd, _dtype_code(src),
        ctypes.byref(rope) if rope is not None else None, _stream(src, stream))
    _check(st, "atlas_cube_reorder_noalloc")
    return dst


def cube_unorder(src, dst, grid, cube, stream=None):
    """Cube order -> raster order (exact inverse of ``cube_reorder``)."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_unorder(_ptr(src), _ptr(dst), Grid3(*grid), Cube3(*cube), heads, hd,
                                  _dtype_code(src), _stream(src, stream))
    _check(st, "atlas_cube_unorder")
    return dst


def rope3d(src, dst, grid, rope: Rope, stream=None):
    """3D RoPE of raster-ordered tokens (``dst`` may be ``src``)."""
    n, heads, hd = src.shape
    st = lib().atlas_rope3d(_ptr(src), _ptr(dst), Grid3(*grid), heads, hd, _dtype_code(src),
                            ctypes.byref(rope), _stream(src, stream))
    _check(st, "atlas_rope3d")
    return dst


def local_global_attn(q_d, k_d, v_d, window_len, q_g, k_g, v_g, o_d, o_g, lse=None,
                      softmax_scale: float = 0.0, stream=None):
    """Asymmetric global-local attention; detail tensors in cube order.
    ``q_d`` (or ``q_g``) may have 0 rows. Returns (o_d, o_g, lse)."""
    ref = q_d if q_d is not None and q_d.shape[0] > 0 else q_g
    heads, hd = ref.shape[1], ref.shape[2]
    n_d = q_d.shape[0] if q_d is not None else 0
    n_g = q_g.shape[0] if q_g is not None else 0
    nz = lambda t, n: _ptr(t) if (t is not None and n > 0) else None
    st = lib().atlas_local_global_attn(
        nz(q_d, n_d), nz(k_d, n_d), nz(v_d, n_d), n_d, int(window_len),
        nz(q_g, n_g), nz(k_g, n_g), nz(v_g, n_g), n_g, heads, hd, float(softmax_scale),
        _dtype_code(ref), nz(o_d, n_d), nz(o_g, n_g), _ptr(lse), _stream(ref, stream))
    _check(st, "atlas_local_global_attn")
    return o_d, o_g, lse


def cube_window_offsets(grid, cube):
    """Window boundaries of the cube order as a host int32 tensor [n+1]
    (partial cubes at the far edges included)."""
    import torch
    n = _i64(0)
    _check(lib().atlas_cube_window_offsets(Grid3(*grid), Cube3(*cube), None, 0, ctypes.byref(n)),
           "atlas_cube_window_offsets")
    out = torch.empty(n.value + 1, dtype=torch.int32)
    _check(lib().atlas_cube_window_offsets(Grid3(*grid), Cube3(*cube),
                                           ctypes.c_void_p(out.data_ptr()), out.numel(),
                                           ctypes.byref(n)), "atlas_cube_window_offsets")
    return out


def local_global_attn_windows(q_d, k_d, v_d, window_offsets, q_g, k_g, v_g, o_d, o_g,
                              lse=None, softmax_scale: float = 0.0, stream=None):
    """Like ``local_global_attn`` with variable-length windows given by the
    device int32 tensor ``window_offsets`` [n_windows + 1]."""
    ref = q_d if q_d is not None and q_d.shape[0] > 0 else q_g
    heads, hd = ref.shape[1], ref.shape[2]
    n_d = q_d.shape[0] if q_d is not None else 0
    n_g = q_g.shape[0] if q_g is not None else 0
    nz = lambda t, n: _ptr(t) if (t is not None and n > 0) else None
    st = lib().atlas_local_global_attn_windows(
        nz(q_d, n_d), nz(k_d, n_d), nz(v_d, n_d), n_d, nz(window_offsets, n_d),
        window_offsets.numel() - 1 if window_offsets is not None else 0,
        nz(q_g, n_g), nz(k_g, n_g), nz(v_g, n_g), n_g, heads, hd, float(softmax_scale),
        _dtype_code(ref), nz(o_d, n_d), nz(o_g, n_g), _ptr(lse), _stream(ref, stream))
    _check(st, "atlas_local_global_attn_windows")
    return o_d, o_g, lse


def local_global_attn_ex(q_d, k_d, v_d, q_g, k_g, v_g, o_d, o_g, lse=None, *, batch=1,
                         window_len=0, window_offsets=None, global_window_offsets=None,
                         softmax_scale: float = 0.0, stream=None):
    """General layout: ``batch`` problems stacked along the rows (detail
    tensors [batch*N, heads, D], global [batch*G, heads, D], lse [batch,
    heads, N+G]); windows of ``window_len`` rows or the device int32
    ``window_offsets`` of one problem; with ``global_window_offsets`` (device
    int32 [n_windows+1], one problem) the queries of window w see only those
    global keys (the aligned variant)."""
    ref = q_d if q_d is not None and q_d.shape[0] > 0 else q_g
    heads, hd = ref.shape[1], ref.shape[2]
    n_d = (q_d.shape[0] if q_d is not None else 0) // batch
    n_g = (q_g.shape[0] if q_g is not None else 0) // batch
    nz = lambda t, n: _ptr(t) if (t is not None and n > 0) else None
    if window_offsets is not None:
        n_win = window_offsets.numel() - 1
    elif global_window_offsets is not None:
        n_win = global_window_offsets.numel() - 1
    else:
        n_win = 0
    wo = _ptr(window_offsets) if window_offsets is not None else None
    gwo = _ptr(global_window_offsets) if global_window_offsets is not None else None
    ly = AttnLayout(int(batch), int(window_len), wo.value if wo is not None else None,
                    int(n_win), gwo.value if gwo is not None else None)
    st = lib().atlas_local_global_attn_ex(
        nz(q_d, n_d), nz(k_d, n_d), nz(v_d, n_d), n_d, nz(q_g, n_g), nz(k_g, n_g), nz(v_g, n_g),
        n_g, ctypes.byref(ly), heads, hd, float(softmax_scale), _dtype_code(ref),
        nz(o_d, n_d), nz(o_g, n_g), _ptr(lse), _stream(ref, stream))
    _check(st, "atlas_local_global_attn_ex")
    return o_d, o_g, lse


def local_global_attn_bwd(q_d, k_d, v_d, o_d, do_d, q_g, k_g, v_g, o_g, do_g, lse,
                          dq_d, dk_d, dv_d, dq_g, dk_g, dv_g, delta=None, *, batch=1,
                          window_len=0, window_offsets=None, global_window_offsets=None,
                          softmax_scale: float = 0.0, stream=None):
    """Gradients of ``local_global_attn_ex`` (same layout arguments): fills
    dq_*, dk_*, dv_* from the forward's inputs, outputs ``o_*``, its ``lse``
    [batch, heads, N+G] and the output gradients ``do_*``. ``delta`` (fp32,
    shape of lse) is the workspace; allocated here when not given."""
    import torch
    ref = q_d if q_d is not None and q_d.shape[0] > 0 else q_g
    heads, hd = ref.shape[1], ref.shape[2]
    n_d = (q_d.shape[0] if q_d is not None else 0) // batch
    n_g = (q_g.shape[0] if q_g is not None else 0) // batch
    if delta is None:
        delta = torch.empty_like(lse)
    nz = lambda t, n: _ptr(t) if (t is not None and n > 0) else None
    if window_offsets is not None:
        n_win = window_offsets.numel() - 1
    elif global_window_offsets is not None:
        n_win = global_window_offsets.numel() - 1
    else:
        n_win = 0
    wo = _ptr(window_offsets) if window_offsets is not None else None
    gwo = _ptr(global_window_offsets) if global_window_offsets is not None else None
    ly = AttnLayout(int(batch), int(window_len), wo.value if wo is not None else None,
                    int(n_win), gwo.value if gwo is not None else None)
    st = lib().atlas_local_global_attn_bwd(
        nz(q_d, n_d), nz(k_d, n_d), nz(v_d, n_d), nz(o_d, n_d), nz(do_d, n_d), n_d,
        nz(q_g, n_g), nz(k_g, n_g), nz(v_g, n_g), nz(o_g, n_g), nz(do_g, n_g), n_g,
        ctypes.byref(ly), heads, hd, float(softmax_scale), _dtype_code(ref), _ptr(lse),
        _ptr(delta), nz(dq_d, n_d), nz(dk_d, n_d), nz(dv_d, n_d), nz(dq_g, n_g),
        nz(dk_g, n_g), nz(dv_g, n_g), _stream(ref, stream))
    _check(st, "atlas_local_global_attn_bwd")
    return dq_d, dk_d, dv_d, dq_g, dk_g, dv_g


def qkv_proj_reorder(x, w, grid, cube, q, k, v, rope: Rope | None = None, batch=1,
                     stream=None):
    """[Q | K | V] = x w^T with RoPE on Q and K and every row written at its
    cube position. x [batch*T*H*W, C] raster order; w [3*heads*head_dim, C];
    q, k, v [batch*T*H*W, heads, head_dim] (outputs)."""
    heads, hd = q.shape[1], q.shape[2]
    st = lib().atlas_qkv_proj_reorder(
        _ptr(x), _ptr(w), int(batch), Grid3(*grid), Cube3(*cube), x.shape[1], heads, hd,
        _dtype_code(x), ctypes.byref(rope) if rope is not None else None, _ptr(q), _ptr(k),
        _ptr(v), _stream(x, stream))
    _check(st, "atlas_qkv_proj_reorder")
    return q, k, v


def out_proj_unorder(o, w, grid, cube, y, batch=1, stream=None):
    """y = unorder(o) w^T: o [batch*T*H*W, heads, head_dim] (or [rows, C_in])
    in cube order, w [C_out, C_in], y [batch*T*H*W, C_out] raster order."""
    rows = o.shape[0]
    c_in = o.numel() // rows if rows else w.shape[1]
    st = lib().atlas_out_proj_unorder(_ptr(o), _ptr(w), int(batch), Grid3(*grid), Cube3(*cube),
                                      c_in, y.shape[1], _dtype_code(o), _ptr(y),
                                      _stream(o, stream))
    _check(st, "atlas_out_proj_unorder")
    return y


def aligned_global_reorder(src, dst, grid, cube, global_grid, rope: Rope | None = None,
                           batch=1, stream=None):
    """Global-proxy tokens (raster order of ``global_grid``) into the aligned
    order of ``grid`` cut into ``cube``; any grid ratios."""
    n, heads, hd = src.shape
    st = lib().atlas_aligned_global_reorder(
        _ptr(src), _ptr(dst), int(batch), Grid3(*grid), Cube3(*cube), Grid3(*global_grid), heads,
        hd, _dtype_code(src), ctypes.byref(rope) if rope is not None else None,
        _stream(src, stream))
    _check(st, "atlas_aligned_global_reorder")
    return dst


def aligned_global_unorder(src, dst, grid, cube, global_grid, rope: Rope | None = None,
                           batch=1, stream=None):
    """Inverse of ``aligned_global_reorder`` (optionally rotating, e.g. by the
    transposed RoPE for gradients)."""
    n, heads, hd = src.shape
    st = lib().atlas_aligned_global_unorder(
        _ptr(src), _ptr(dst), int(batch), Grid3(*grid), Cube3(*cube), Grid3(*global_grid), heads,
        hd, _dtype_code(src), ctypes.byref(rope) if rope is not None else None,
        _stream(src, stream))
    _check(st, "atlas_aligned_global_unorder")
    return dst


def aligned_global_offsets(grid, cube, global_grid):
    """Global key range of every detail window in the aligned order, as a
    host int32 tensor [n_windows + 1]."""
    import torch
    n = _i64(0)
    args = (Grid3(*grid), Cube3(*cube), Grid3(*global_grid))
    _check(lib().atlas_aligned_global_offsets(*args, None, 0, ctypes.byref(n)),
           "atlas_aligned_global_offsets")
    out = torch.empty(n.value + 1, dtype=torch.int32)
    _check(lib().atlas_aligned_global_offsets(*args, ctypes.c_void_p(out.data_ptr()),
                                              out.numel(), ctypes.byref(n)),
           "atlas_aligned_global_offsets")
    return out


def aligned_global_cube(grid, cube, global_grid):
    """The global-grid cube whose cubes are the aligned sets of the detail
    cubes (ratios must be integers dividing the cube)."""
    out = Cube3()
    _check(lib().atlas_aligned_global_cube(Grid3(*grid), Cube3(*cube), Grid3(*global_grid),
                                           ctypes.byref(out)), "atlas_aligned_global_cube")
    return (out.ct, out.ch, out.cw)


def cube_reorder_batched(src, dst, batch, grid, cube, rope: Rope | None = None, stream=None):
    """``cube_reorder`` of ``batch`` problems stacked along the rows."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_reorder_batched(
        _ptr(src), _ptr(dst), int(batch), Grid3(*grid), Cube3(*cube), heads, hd,
        _dtype_code(src), ctypes.byref(rope) if rope is not None else None, _stream(src, stream))
    _check(st, "atlas_cube_reorder_batched")
    return dst


def cube_unorder_batched(src, dst, batch, grid, cube, stream=None):
    """``cube_unorder`` of ``batch`` problems stacked along the rows."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_unorder_batched(_ptr(src), _ptr(dst), int(batch), Grid3(*grid),
                                          Cube3(*cube), heads, hd, _dtype_code(src),
                                          _stream(src, stream))
    _check(st, "atlas_cube_unorder_batched")
    return dst


def cube_unorder_rope(src, dst, grid, cube, rope: Rope, batch=1, stream=None):
    """Cube -> raster order with each row rotated at its raster position
    (with negated scales: the gradient of ``cube_reorder`` with RoPE)."""
    n, heads, hd = src.shape
    st = lib().atlas_cube_unorder_rope(_ptr(src), _ptr(dst), int(batch), Grid3(*grid),
                                       Cube3(*cube), heads, hd, _dtype_code(src),
                                       ctypes.byref(rope), _stream(src, stream))
    _check(st, "atlas_cube_unorder_rope")
    return dst


def transpose_rope(rope: Rope) -> Rope:
    """The same RoPE with negated position scales: rotation by -phi, the
    transpose (and inverse) of ``rope``."""
    return Rope(rope.theta, rope.d_t, rope.d_h, rope.d_w, -rope.scale_t, -rope.scale_h,
                -rope.scale_w)


def rope3d_batched(src, dst, batch, grid, rope: Rope, stream=None):
    """``rope3d`` of ``batch`` problems stacked along the rows."""
    n, heads, hd = src.shape
    st = lib().atlas_rope3d_batched(_ptr(src), _ptr(dst), int(batch), Grid3(*grid), heads, hd,
                                    _dtype_code(src), ctypes.byref(rope), _stream(src, stream))
    _check(st, "atlas_rope3d_batched")
    return dst


# ---------------------------------------------------------------------------
# Differential-attention layer: rotary positions, attention, group norm.
# These calls check shapes, types and devices here (the C-ABI cannot see
# them), run on the tensors' device whatever the current one is, and take
# `stream` as the stream of that device to enqueue on.
# ---------------------------------------------------------------------------

def _require(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _on(dev: int, *tensors):
    """Every tensor (None skipped) on CUDA device ``dev``."""
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError("tensors must live on one CUDA device")


def _fp32(n, what, *tensors):
    import torch
    for t in tensors:
        if t is not None and (t.dtype != torch.float32 or t.numel() != n):
            raise ValueError(f"{what}: fp32 of {n} elements expected")


def _at(t):
    """Device address of a contiguous tensor (None: NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _run(where, dev, stream, fn, *args):
    """fn(*args, stream) with device ``dev`` current; raises on a status."""
    import torch
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _run(where, dev, stream, fn, *args)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    status = fn(*args, stream.cuda_stream)
    if status != OK:
        raise AtlasError(status, where)


def _work(workspace, ref, stream, nbytes):
    """The caller's workspace once checked, or a new one whose memory goes back
    to the pool of the stream using it."""
    import torch
    if workspace is not None:
        _on(ref.get_device(), workspace)
        _require(workspace.numel() * workspace.element_size() >= nbytes,
                 "the workspace is smaller than the call needs")
        return workspace
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=ref.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=ref.device)


def _rows(t):
    """(address, row stride in elements) of [rows, heads, head_dim] whose rows
    are contiguous, as a slice of a wider buffer's columns is."""
    n, heads, hd = t.shape
    s0, s1, s2 = t.stride()
    # (a row stride of 0, an expanded tensor's, would mean contiguous rows below)
    _require((hd == 1 or s2 == 1) and (heads == 1 or s1 == hd) and (n <= 1 or s0 >= heads * hd),
             "tensors must be [rows, heads, head_dim] with contiguous rows, none of them shared")
    return t.data_ptr(), s0 if n > 1 else heads * hd


def rotary(tensors, grid, rot: Rotary, *, cube=None, order="raster", positions=None,
           transpose=False, batch=1, stream=None):
    """Rotary positions of several tensors of the same tokens in one launch.

    tensors: (src, dst) or (src, dst, rotate) of [batch*T*H*W, heads,
    head_dim] each (the heads may differ; rows may be strided); rotate False
    only moves the rows. order "reorder" / "unorder" also takes the rows from
    raster to cube order or back (``cube``). positions: int32 [batch*T*H*W]
    or [.., 1 or 3], by raster row, instead of the grid index. transpose
    rotates back: the gradient's map. Returns the destinations."""
    import torch
    _require(len(tensors) > 0, "at least one tensor")
    ref = tensors[0][0]
    dev, dtype, hd = ref.get_device(), ref.dtype, ref.shape[-1]
    rows = int(batch) * grid[0] * grid[1] * grid[2]
    items = (RotaryTensor * len(tensors))()
    for item, t in zip(items, tensors):
        src, dst = t[0], t[1]
        _on(dev, src, dst)
        _require(src.dim() == 3 and src.shape == dst.shape and src.shape[0] == rows and
                 src.shape[2] == hd, "rotary: src and dst of [batch*T*H*W, heads, head_dim], one "
                 "head_dim for all")
        _require(src.dtype == dtype and dst.dtype == dtype, "rotary: one dtype for all")
        item.src, item.src_stride = _rows(src)
        item.dst, item.dst_stride = _rows(dst)
        item.heads, item.rotate = src.shape[1], int(bool(t[2]) if len(t) > 2 else True)
    axes = 0
    if positions is not None:
        _on(dev, positions)
        _require(positions.dtype == torch.int32 and positions.dim() in (1, 2) and
                 positions.shape[0] == rows, "rotary: positions are int32 [batch*T*H*W(, axes)]")
        axes = positions.shape[1] if positions.dim() == 2 else 1
    if bool(rot.transpose) != bool(transpose):
        rot = Rotary.from_buffer_copy(rot)
        rot.transpose = int(bool(transpose))
    c = ctypes.byref(Cube3(*cube)) if cube is not None else None
    _run("atlas_rotary_apply", dev, stream, lib().atlas_rotary_apply, items, len(tensors), int(batch),
         Grid3(*grid), c, ORDERS[order], _at(positions), axes, hd, _dtype_code(ref),
         ctypes.byref(rot))
    return [t[1] for t in tensors]


def _vectors(what, vectors, scalars):
    """(device, n, d) of lambda's [n, d] vectors, all of one dtype, and its [n]."""
    q1 = vectors[0]
    _on(q1.get_device(), *vectors, scalars)
    for t in vectors:
        _require(t.dim() == 2 and t.shape == q1.shape and t.dtype == q1.dtype,
                 "diff_lambda: vectors of [n, d] and one dtype")
    _fp32(q1.shape[0], what, scalars)
    return q1.get_device(), q1.shape[0], q1.shape[1]


def diff_lambda(q1, k1, q2, k2, lambda_init, lam, stream=None):
    """lam [n] = exp<q1,k1> - exp<q2,k2> + lambda_init from vectors [n, d]."""
    dev, n, d = _vectors("diff_lambda lam", (q1, k1, q2, k2), lam)
    _run("atlas_diff_lambda", dev, stream, lib().atlas_diff_lambda, _at(q1), _at(k1), _at(q2),
         _at(k2), n, d, float(lambda_init), _dtype_code(q1), _at(lam))
    return lam


def diff_lambda_bwd(q1, k1, q2, k2, dlam, dq1, dk1, dq2, dk2, stream=None):
    """Gradients of ``diff_lambda``'s vectors from dlam [n]."""
    dev, n, d = _vectors("diff_lambda_bwd dlam", (q1, k1, q2, k2, dq1, dk1, dq2, dk2), dlam)
    _run("atlas_diff_lambda_bwd", dev, stream, lib().atlas_diff_lambda_bwd, _at(q1), _at(k1), _at(q2),
         _at(k2), n, d, _at(dlam), _dtype_code(q1), _at(dq1), _at(dk1), _at(dq2), _at(dk2))
    return dq1, dk1, dq2, dk2


def _diff_sides(batch, detail, glob, window_offsets, global_window_offsets, window_len, lam):
    """Shapes shared by diff_attn and its backward: (reference tensor, detail
    rows and global rows of one problem, addresses of both sides, layout). None
    stands for no rows."""
    import torch
    batch = int(batch)
    ref = next((t for t in (*detail, *glob) if t is not None and t.shape[0] > 0), None)
    _require(ref is not None and ref.dim() == 3 and batch >= 1,
             "diff_attn: [rows, heads, head_dim] tensors and batch >= 1")
    for side in (detail, glob):   # what such a side holds would be neither read nor written
        _require(side[0] is not None and side[0].shape[0] > 0 or
                 all(t is None or t.shape[0] == 0 for t in side),
                 "diff_attn: rows for a side without queries")
    dev, dtype, tail = ref.get_device(), ref.dtype, ref.shape[1:]
    counts, sides = [], []
    for side in (detail, glob):
        n = side[0].shape[0] if side[0] is not None else 0
        _require(n % batch == 0, "diff_attn: rows are not a multiple of batch")
        if n == 0:
            sides.append([None] * len(side))
        else:
            _on(dev, *side)
            for t in side:
                _require(t is None or (t.shape[0] == n and t.shape[1:] == tail and t.dtype == dtype),
                         "diff_attn: tensors of one side have one shape and dtype")
            sides.append([_at(t) for t in side])
        counts.append(n // batch)
    _on(dev, lam, window_offsets, global_window_offsets)
    _require(lam.numel() in (1, ref.shape[1]), "diff_attn: lam has one entry or one per head")
    _fp32(lam.numel(), "diff_attn lam", lam)
    for off in (window_offsets, global_window_offsets):
        _require(off is None or (off.dtype == torch.int32 and off.numel() >= 2),
                 "diff_attn: offsets are int32 [n_windows + 1]")
    if window_offsets is not None and global_window_offsets is not None:
        _require(window_offsets.numel() == global_window_offsets.numel(),
                 "diff_attn: one global range per window")
    first = window_offsets if window_offsets is not None else global_window_offsets
    ly = AttnLayout(batch, int(window_len), _at(window_offsets),
                    first.numel() - 1 if first is not None else 0, _at(global_window_offsets))
    return ref, counts[0], counts[1], sides[0], sides[1], ly


def diff_attn(q_d, k_d, v_d, q_g, k_g, v_g, lam, o_d, o_g, s_d=None, s_g=None, lse=None, *,
              batch=1, window_len=0, window_offsets=None, global_window_offsets=None,
              softmax_scale: float = 0.0, stream=None):
    """Differential attention o = (softmax(q1 k1) - lam softmax(q2 k2)) v over
    the layouts of ``local_global_attn_ex``; the halves of a head are the two
    maps. lam: fp32, one entry or one per head. For ``diff_attn_bwd`` pass s_d
    and s_g (the second map's output) and lse (fp32 [batch, heads, 2, N+G])."""
    ref, n_d, n_g, d, g, ly = _diff_sides(
        batch, (q_d, k_d, v_d, o_d, s_d), (q_g, k_g, v_g, o_g, s_g), window_offsets,
        global_window_offsets, window_len, lam)
    heads, hd = ref.shape[1], ref.shape[2]
    _on(ref.get_device(), lse)
    _fp32(2 * ly.batch * heads * (n_d + n_g), "diff_attn lse", lse)
    _run("atlas_diff_attn", ref.get_device(), stream, lib().atlas_diff_attn, d[0], d[1], d[2], n_d,
         g[0], g[1], g[2], n_g, ctypes.byref(ly), heads, hd, float(softmax_scale), _dtype_code(ref),
         _at(lam), lam.numel(), d[3], g[3], d[4], g[4], _at(lse))
    return o_d, o_g


def diff_attn_bwd(q_d, k_d, v_d, o_d, s_d, do_d, q_g, k_g, v_g, o_g, s_g, do_g, lam, lse,
                  dq_d, dk_d, dv_d, dq_g, dk_g, dv_g, dlam, workspace=None, *, batch=1,
                  window_len=0, window_offsets=None, global_window_offsets=None,
                  softmax_scale: float = 0.0, stream=None):
    """Gradients of ``diff_attn`` (same layout arguments): dq_*, dk_*, dv_* and
    dlam (as lam). workspace: any dtype, of at least
    ``diff_attn_bwd_workspace`` bytes; allocated here when not given."""
    ref, n_d, n_g, d, g, ly = _diff_sides(
        batch, (q_d, k_d, v_d, o_d, s_d, do_d, dq_d, dk_d, dv_d),
        (q_g, k_g, v_g, o_g, s_g, do_g, dq_g, dk_g, dv_g), window_offsets, global_window_offsets,
        window_len, lam)
    dev, heads, hd = ref.get_device(), ref.shape[1], ref.shape[2]
    _on(dev, lse, dlam)
    _fp32(2 * ly.batch * heads * (n_d + n_g), "diff_attn_bwd lse", lse)
    _fp32(lam.numel(), "diff_attn_bwd dlam", dlam)
    code = _dtype_code(ref)
    work = _work(workspace, ref, stream,
                 lib().atlas_diff_attn_bwd_workspace(ly.batch, n_d, n_g, heads, hd, code))
    _run("atlas_diff_attn_bwd", dev, stream, lib().atlas_diff_attn_bwd, *d[:6], n_d, *g[:6], n_g,
         ctypes.byref(ly), heads, hd, float(softmax_scale), code, _at(lam), lam.numel(), _at(lse),
         _at(work), *d[6:], *g[6:], _at(dlam))
    return dq_d, dk_d, dv_d, dq_g, dk_g, dv_g, dlam


def diff_attn_bwd_workspace(batch, n_detail, n_global, heads, head_dim, dtype) -> int:
    """Bytes of ``diff_attn_bwd``'s workspace (rows of one problem; dtype BF16
    or FP32)."""
    return int(lib().atlas_diff_attn_bwd_workspace(int(batch), int(n_detail), int(n_global),
                                                   int(heads), int(head_dim), int(dtype)))


def _norm_sizes(x, rows, groups, tensors, vectors, stats):
    rows = int(rows)
    _require(x.dim() == 2 and rows >= 1 and x.shape[0] % rows == 0,
             "group_norm: x is [samples*rows, channels]")
    _on(x.get_device(), x, *tensors, *vectors, stats)
    for t in tensors:
        _require(t.shape == x.shape and t.dtype == x.dtype,
                 "group_norm: tensors of x's shape and dtype")
    _fp32(x.shape[1], "group_norm gamma and beta", *vectors)
    samples = x.shape[0] // rows
    _fp32(2 * samples * int(groups), "group_norm stats", stats)
    return samples, rows, x.shape[1], int(groups)


def group_norm(x, gamma, beta, y, rows, groups, *, eps=1e-5, activation="none", stats=None,
               workspace=None, stream=None):
    """y = act(group norm of x [samples*rows, channels]); a sample is ``rows``
    consecutive rows (rows 1, groups = heads: each head of a token by itself).
    gamma, beta: fp32 [channels] or None. stats: fp32 [samples, groups, 2],
    needed by ``group_norm_bwd``. activation "none" or "silu"."""
    sizes, code = _norm_sizes(x, rows, groups, (y,), (gamma, beta), stats), _dtype_code(x)
    work = _work(workspace, x, stream, lib().atlas_group_norm_workspace(*sizes, code, 0))
    _run("atlas_group_norm", x.get_device(), stream, lib().atlas_group_norm, _at(x), _at(gamma),
         _at(beta), _at(y), *sizes, float(eps), ACTIVATIONS[activation], code, _at(stats), _at(work))
    return y


def group_norm_bwd(dy, x, gamma, beta, stats, dx, dgamma, dbeta, rows, groups, *,
                   activation="none", workspace=None, stream=None):
    """dx, and dgamma and dbeta (fp32 [channels], or None), of ``group_norm``
    from dy and the forward's x and stats."""
    _require(stats is not None, "group_norm_bwd: the forward's stats")
    sizes = _norm_sizes(x, rows, groups, (dy, dx), (gamma, beta, dgamma, dbeta), stats)
    code = _dtype_code(x)
    work = _work(workspace, x, stream, lib().atlas_group_norm_workspace(*sizes, code, 1))
    _run("atlas_group_norm_bwd", x.get_device(), stream, lib().atlas_group_norm_bwd, _at(dy), _at(x),
         _at(gamma), _at(beta), _at(stats), _at(dx), _at(dgamma), _at(dbeta), *sizes,
         ACTIVATIONS[activation], code, _at(work))
    return dx, dgamma, dbeta


def group_norm_workspace(x, rows, groups, backward) -> int:
    """Bytes of the workspace of ``group_norm`` or ``group_norm_bwd``."""
    return int(lib().atlas_group_norm_workspace(x.shape[0] // int(rows), int(rows), x.shape[1],
                                                int(groups), _dtype_code(x), int(bool(backward))))


def last_device_error(stream=None) -> int:
    """Synchronise and read/clear the device error word (0 = clean)."""
    import torch
    s = ctypes.c_void_p(stream.cuda_stream if stream is not None
                        else torch.cuda.current_stream().cuda_stream)
    code = ctypes.c_uint32(0)
    st = lib().atlas_last_device_error(s, ctypes.byref(code))
    if st not in (OK, ERR_TIMEOUT):
        raise AtlasError(st, "atlas_last_device_error")
    return int(code.value)


def debug_stall_next_attention():
    """Test hook: the next bf16 attention launch leaves one K tile unloaded,
    so its bounded waits expire and it reports ATLAS_ERR_TIMEOUT."""
    _check(lib().atlas_debug_stall_next_attention(), "atlas_debug_stall_next_attention")


def cached_rope_tables() -> int:
    """RoPE tables the library holds in device memory it allocated."""
    return int(lib().atlas_cached_rope_tables())


def release_caches():
    _check(lib().atlas_release_caches(), "atlas_release_caches")


def version() -> int:
    return int(lib().atlas_version())
