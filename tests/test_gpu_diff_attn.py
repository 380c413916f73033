"""Differential attention, its lambda and their gradients against a 64-bit
reference, value by value within bounds derived in diff_ref.py."""
import math

import pytest
import torch

import diff_ref
from helpers import check_no_device_error
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
GRADS = ("dq", "dk", "dv")


def rnd(*shape, seed=0, dtype=torch.float32, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def make(B, N, G, H, hd, dtype, seed=0):
    t = {}
    for i, n in enumerate(("q", "k", "v", "do")):
        t[n + "_d"] = rnd(B * N, H, hd, seed=seed + i, dtype=DT[dtype])
        t[n + "_g"] = rnd(B * G, H, hd, seed=seed + 10 + i, dtype=DT[dtype])
    return t


def run(t, lam, B, N, G, H, train=True, guard=False, **layout):
    """Forward (and backward) through the binding; a dict of outputs."""
    out = {}
    like = t["q_d"] if N else t["q_g"]
    for n in ("o", "s") + GRADS:
        for p, rows in (("d", B * N), ("g", B * G)):
            out[f"{n}_{p}"] = torch.full((rows, *like.shape[1:]), 7.0, dtype=like.dtype, device=DEV)
    lse = torch.full((B, H, 2, N + G), 7.0, device=DEV)
    o = out
    atlas.diff_attn(t["q_d"], t["k_d"], t["v_d"], t["q_g"], t["k_g"], t["v_g"], lam, o["o_d"], o["o_g"],
                    o["s_d"] if train else None, o["s_g"] if train else None, lse if train else None,
                    batch=B, **layout)
    if train:
        out["lse"], out["dlam"] = lse, torch.full_like(lam, 7.0)
        atlas.diff_attn_bwd(t["q_d"], t["k_d"], t["v_d"], o["o_d"], o["s_d"], t["do_d"], t["q_g"],
                            t["k_g"], t["v_g"], o["o_g"], o["s_g"], t["do_g"], lam, lse, o["dq_d"],
                            o["dk_d"], o["dv_d"], o["dq_g"], o["dk_g"], o["dv_g"], out["dlam"],
                            batch=B, **layout)
    torch.cuda.synchronize()
    check_no_device_error()
    return out


def against_reference(t, out, lam, B, N, G, H, hd, dtype, windows, shares=None, scale=None):
    mask = diff_ref.mask_of(N, G, windows, shares).to(DEV)
    scale = scale or (hd // 2) ** -0.5
    dlam, dlam_bound = torch.zeros(2, H, dtype=torch.float64, device=DEV)
    for b in range(B):
        for h in range(H):
            part = lambda n: torch.cat([t[n + "_d"][b * N:(b + 1) * N, h],  # noqa: E731
                                        t[n + "_g"][b * G:(b + 1) * G, h]]).double()
            r = diff_ref.Diff(part("q"), part("k"), part("v"), float(lam[h % lam.numel()]), mask, scale,
                              DT[dtype], part("do"))
            for n in ("o", "s") + GRADS:
                got = torch.cat([out[n + "_d"][b * N:(b + 1) * N, h], out[n + "_g"][b * G:(b + 1) * G, h]])
                diff_ref.check(f"{n} b{b} h{h}", got.double(), getattr(r, n), getattr(r, n + "_bound"))
            for m in range(2):
                diff_ref.check(f"lse{m} b{b} h{h}", out["lse"][b, h, m].double(), r.lse[m],
                               torch.full_like(r.lse[m], r.lse_bound) + 2.0 ** -22 * r.lse[m].abs())
            dlam[h] += r.dlam
            dlam_bound[h] += r.dlam_bound
    if lam.numel() == 1:
        dlam, dlam_bound = dlam.sum().reshape(1), dlam_bound.sum().reshape(1)
    diff_ref.check("dlam", out["dlam"].double(), dlam, dlam_bound)


FIXED = [
    # batch, n_detail, window, n_global, heads
    (1, 256, 32, 32, 2),
    (1, 0, 1, 1, 1),          # one global token alone
    (1, 1, 1, 0, 1),          # one detail token alone
    (1, 1, 1, 1, 3),
    (1, 130, 1, 5, 1),        # windows of one row
    (2, 387, 129, 1, 2),      # one row over a tile, twice
    (1, 512, 256, 0, 1),      # no global tokens
    (1, 0, 1, 129, 2),        # no detail rows
    (3, 0, 1, 333, 1),
    (1, 640, 160, 77, 1),
    (2, 768, 768, 300, 1),
    (1, 127 * 3, 127, 63, 1), # one row short of a tile
    (1, 1000, 500, 515, 2),
    (2, 96, 24, 640, 1),
    (1, 2304, 768, 260, 1),   # few long units over global keys: cut into parts
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("case", FIXED, ids=str)
def test_fixed_windows(case, hd, dtype):
    B, N, L, G, H = case
    t = make(B, N, G, H, hd, dtype)
    lam = 0.3 + 0.2 * rnd(H, seed=5).abs()
    out = run(t, lam, B, N, G, H, window_len=L)
    against_reference(t, out, lam, B, N, G, H, hd, dtype, list(range(0, N + 1, L)))
    plain = run(t, lam, B, N, G, H, train=False, window_len=L)
    assert torch.equal(plain["o_d"], out["o_d"]) and torch.equal(plain["o_g"], out["o_g"])


OFFSETS = [
    # window offsets, global ranges (None: all), n_global
    ([0, 1, 5, 40, 41, 170, 300], None, 77),
    ([0, 200, 456, 457, 600], None, 130),              # windows of over a tile, and of one row
    ([0, 200, 456, 457, 600], [0, 0, 64, 64, 130], 130),   # some windows see no global token
    ([0, 30, 60, 90], [0, 10, 10, 33], 33),
    ([0, 300], [0, 257], 257),
    ([0, 128, 256, 384], [0, 128, 131, 260], 260),
    ([0, 7], None, 0),
    # parts of units whose queries run out: some see no window
    ([0, 700, 1400, 2100], [0, 140, 140, 300], 300),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("case", OFFSETS, ids=lambda c: f"{c[0]}-{c[2]}")
def test_offsets_and_aligned(case, hd, dtype):
    windows, shares, G = case
    B, N, H = 2, windows[-1], 2
    t = make(B, N, G, H, hd, dtype)
    lam = torch.tensor([-0.4], device=DEV)             # shared by the heads, and negative
    as_dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = run(t, lam, B, N, G, H, window_offsets=as_dev(windows), global_window_offsets=as_dev(shares))
    against_reference(t, out, lam, B, N, G, H, hd, dtype, windows, shares)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_aligned_fixed_windows_and_scale(hd, dtype):
    B, N, L, G, H = 1, 384, 128, 100, 2
    t = make(B, N, G, H, hd, dtype)
    lam = torch.tensor([0.7, 0.0], device=DEV)         # lambda 0: the first map alone
    shares = [0, 50, 50, 100]
    out = run(t, lam, B, N, G, H, window_len=L, softmax_scale=0.31,
              global_window_offsets=torch.tensor(shares, dtype=torch.int32, device=DEV))
    against_reference(t, out, lam, B, N, G, H, hd, dtype, [0, 128, 256, 384], shares, scale=0.31)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sharp_logits(dtype):
    """Logits of +-200 and of -3e4: one key takes a row, or none stands out; the
    running maximum jumps late."""
    B, N, L, G, H, hd = 1, 256, 256, 300, 1, 64
    t = make(B, N, G, H, hd, dtype)
    for n in ("q_d", "q_g"):
        t[n] = (t[n].float() * 12).to(DT[dtype])
    t["k_g"][299] *= 6
    t["k_d"][:128, :, 32:] = 0
    t["q_d"][:, :, 32:] = 0
    t["q_d"][:, :, 32] = 64.0
    t["k_d"][:, :, 32] = -2600.0                        # second map: -3e4 for every window key
    t["k_d"][7, :, 32] = 0.0
    lam = torch.tensor([0.5], device=DEV)
    out = run(t, lam, B, N, G, H, window_len=L)
    for n in ("o_d", "o_g", "dq_d", "dk_d", "dv_d", "dq_g", "dk_g", "dv_g"):
        assert bool(torch.isfinite(out[n]).all()), n
    mask = diff_ref.mask_of(N, G, [0, 256]).to(DEV)
    cat = lambda n: torch.cat([t[n + "_d"][:, 0], t[n + "_g"][:, 0]]).double()  # noqa: E731
    r = diff_ref.Diff(cat("q"), cat("k"), cat("v"), 0.5, mask, 32 ** -0.5, DT[dtype], None)
    # a logit of magnitude M carries 2^-24 M: eps of the reference grows to it
    got = torch.cat([out["o_d"], out["o_g"]])[:, 0].double()
    diff_ref.check("o", got, r.o, r.o_bound)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_masked_garbage_changes_nothing(hd, dtype):
    """NaN and infinities in another problem and in other windows (of at least
    128 rows), their tiles' tails included, reach no row that must not see them."""
    B, N, G, H = 2, 600, 150, 2
    windows, shares = [0, 200, 456, 600], [0, 40, 90, 150]
    off = torch.tensor(windows, dtype=torch.int32, device=DEV)
    sh = torch.tensor(shares, dtype=torch.int32, device=DEV)
    lam = torch.tensor([0.6, 0.3], device=DEV)
    t = make(B, N, G, H, hd, dtype)
    clean = run(t, lam, B, N, G, H, window_offsets=off, global_window_offsets=sh)
    bad = {n: x.clone() for n, x in t.items()}
    for n in ("q", "k", "v", "do"):
        bad[n + "_d"][N:] = float("nan")                # problem 1
        bad[n + "_g"][G:] = float("inf")
        bad[n + "_d"][200:456] = float("inf")           # window 1 of problem 0
    bad["k_d"][300] = float("nan")
    out = run(bad, lam, B, N, G, H, window_offsets=off, global_window_offsets=sh)
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[200:456] = False
    for n in ("o", "s") + GRADS:
        assert torch.equal(out[n + "_d"][:N][keep], clean[n + "_d"][:N][keep]), n
    for n in ("o", "s", "dq"):
        assert torch.equal(out[n + "_g"][:G], clean[n + "_g"][:G]), n
    # global keys seen by windows 0 and 2 only get clean gradients
    seen = torch.ones(G, dtype=torch.bool, device=DEV)
    seen[40:90] = False
    for n in ("dk", "dv"):
        assert torch.equal(out[n + "_g"][:G][seen], clean[n + "_g"][:G][seen]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("aligned", [False, True])
def test_masked_garbage_in_short_windows(hd, dtype, aligned):
    """The same for windows that share a 128-row tile: only the rows of the window
    that holds the garbage, and the global keys it meets, are touched; those are."""
    B, N, L, G, H = 1, 200, 20, 60, 1
    shares = [0, 10, 10, 16, 22, 28, 34, 40, 46, 52, 60]
    kw = {"window_len": L}
    if aligned:
        kw["global_window_offsets"] = torch.tensor(shares, dtype=torch.int32, device=DEV)
    lam = torch.tensor([0.6], device=DEV)
    t = make(B, N, G, H, hd, dtype)
    clean = run(t, lam, B, N, G, H, **kw)
    for name, row, value in (("v_d", 45, float("inf")), ("k_d", 59, float("nan")), ("q_d", 40, float("inf")),
                             ("do_d", 51, float("nan")), ("v_d", 199, float("nan"))):
        w = row // L
        mine = slice(w * L, (w + 1) * L)
        bad = {n: x.clone() for n, x in t.items()}
        bad[name][row, 0, 3] = value
        out = run(bad, lam, B, N, G, H, **kw)
        rest = torch.ones(N, dtype=torch.bool, device=DEV)
        rest[mine] = False
        for n in ("o", "s") + GRADS:
            assert torch.equal(out[n + "_d"][rest], clean[n + "_d"][rest]), (name, n)
        for n in ("o", "s", "dq"):
            assert torch.equal(out[n + "_g"], clean[n + "_g"]), (name, n)
        if aligned:
            unseen = torch.ones(G, dtype=torch.bool, device=DEV)
            unseen[shares[w]:shares[w + 1]] = False
            for n in ("dk", "dv"):
                assert torch.equal(out[n + "_g"][unseen], clean[n + "_g"][unseen]), (name, n)
        # and the rows that do see it show it
        if name in ("v_d", "k_d"):
            assert not bool(torch.isfinite(out["o_d"][mine, 0, 3]).any()), name
        if name == "q_d":
            assert not bool(torch.isfinite(out["o_d"][row]).any())
        if name == "do_d":
            assert not bool(torch.isfinite(out["dv_d"][mine, 0, 3]).any())
            assert not bool(torch.isfinite(out["dk_d"][mine]).any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bits_streams_and_graph(dtype):
    """The same call gives the same bits: eager twice, on a side stream, and
    replayed from a graph that two captures share the inputs of."""
    B, N, L, G, H, hd = 2, 320, 160, 90, 2, 128
    t = make(B, N, G, H, hd, dtype)
    lam = torch.tensor([0.5, 0.2], device=DEV)
    first = run(t, lam, B, N, G, H, window_len=L)
    second = run(t, lam, B, N, G, H, window_len=L)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        third = run(t, lam, B, N, G, H, window_len=L)
    for n in first:
        assert torch.equal(first[n], second[n]) and torch.equal(first[n], third[n]), n
    graphs, outs = [], []
    for _ in range(2):
        o = {n: torch.empty_like(x) for n, x in first.items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            atlas.diff_attn(t["q_d"], t["k_d"], t["v_d"], t["q_g"], t["k_g"], t["v_g"], lam, o["o_d"],
                            o["o_g"], o["s_d"], o["s_g"], o["lse"], batch=B, window_len=L)
            atlas.diff_attn_bwd(t["q_d"], t["k_d"], t["v_d"], o["o_d"], o["s_d"], t["do_d"], t["q_g"],
                                t["k_g"], t["v_g"], o["o_g"], o["s_g"], t["do_g"], lam, o["lse"],
                                o["dq_d"], o["dk_d"], o["dv_d"], o["dq_g"], o["dk_g"], o["dv_g"],
                                o["dlam"], batch=B, window_len=L)
        graphs.append(g)
        outs.append(o)
    # two graphs side by side: each has its own workspace
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        for g, st in zip(graphs, (a, b)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    check_no_device_error()
    for o in outs:
        for n in first:
            assert torch.equal(first[n], o[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d", [(1, 32), (40, 64), (3, 1), (9, 257)])
def test_lambda(n, d, dtype):
    v = [rnd(n, d, seed=i, dtype=DT[dtype], std=0.3 / math.sqrt(d)) for i in range(4)]
    lam, dlam = torch.empty(n, device=DEV), rnd(n, seed=9)
    atlas.diff_lambda(*v, 0.8, lam)
    x = [a.double() for a in v]
    e = [(x[0] * x[1]).sum(1).exp(), (x[2] * x[3]).sum(1).exp()]
    tol = 2.0 ** -22 * (d + 8) * (e[0] + e[1] + 0.8)
    diff_ref.check("lam", lam.double(), e[0] - e[1] + 0.8, tol)
    dv = [torch.empty_like(a) for a in v]
    atlas.diff_lambda_bwd(*v, dlam, *dv)
    g = [dlam.double() * e[0], -dlam.double() * e[1]]
    for i in range(4):
        want = g[i // 2][:, None] * x[i ^ 1]
        diff_ref.check(f"dv{i}", dv[i].double(), want,
                       (diff_ref.unit(DT[dtype]) + 2.0 ** -22 * (d + 8)) * want.abs())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("N,G,L", [(512, 100, 256), (300, 60, 30), (640, 0, 640), (0, 332, 1)])
def test_dlambda_has_no_rounding_of_the_stored_output(N, G, L, hd, dtype):
    """Zero keys weigh all alike, and a quarter of the values are one bf16 step above
    1: every s is 1 + 2^-9, which bf16 stores as 1. With do = 1, dlambda = -(rows) D
    (1 + 2^-9). Relative errors: of a weight 2^-22 (n + 16) (diff_ref.py), of sums of
    terms of one sign over the n keys or over channels and rows below 2^-24 (n + 64)
    each; the stored s would be off by 2^-9."""
    B, H = 2, 2
    lam = torch.tensor([0.4, 0.7], device=DEV)
    t = make(B, N, G, H, hd, dtype)
    for p in "dg":
        t["k_" + p].zero_()
        t["do_" + p].fill_(1.0)
        t["v_" + p].fill_(1.0)
        t["v_" + p][::4] = 1.0 + 2.0 ** -7
    # windows, global rows and problems hold a multiple of four rows, or a share
    # of the raised values that the reference counts
    out = run(t, lam, B, N, G, H, window_len=L)
    mask = diff_ref.mask_of(N, G, list(range(0, N + 1, L)) if N else [0]).to(DEV).double()
    want = 0.0
    for b in range(B):
        v = torch.cat([t["v_d"][b * N:(b + 1) * N, 0, 0], t["v_g"][b * G:(b + 1) * G, 0, 0]]).double()
        want -= float((mask @ v / mask.sum(1)).sum()) * hd
    n = int(mask.sum(1).max())
    err = (out["dlam"].double() - want).abs() / abs(want)
    assert float(err.max()) <= 2.0 ** -22 * (n + 16) + 2 * 2.0 ** -24 * (n + 64), err


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("N,G,L", [(0, 1, 1), (0, 2, 1), (0, 3, 1), (60, 0, 2), (40, 0, 1), (90, 2, 3), (256, 1, 128)])
def test_few_keys_keep_their_accuracy(N, G, L, hd):
    """bf16 rows of one to five keys, as a whole: weights that are divided by their
    own sum, and dP - D without the stored outputs' rounding. Each element then
    carries independent roundings, of P (or W, or dS) and of the result, each at most
    U of its term: 2 U sum|terms|, not U |o| / (P - D)-fold. Rounding errors of
    independent sign add like their squares, a third of a bound on average, so the
    norms stay below 2 U |terms|."""
    B, H = 3, 2
    lam = torch.tensor([0.62, 0.7], device=DEV)
    t = make(B, N, G, H, hd, "bf16", seed=3 * N + G)
    out = run(t, lam, B, N, G, H, window_len=L)
    mask = diff_ref.mask_of(N, G, list(range(0, N + 1, L)) if N else [0]).to(DEV)
    U, few = diff_ref.unit(torch.bfloat16), mask.sum(1) <= 8
    sums = {}
    for b in range(B):
        for h in range(H):
            part = lambda n: torch.cat([t[n + "_d"][b * N:(b + 1) * N, h],  # noqa: E731
                                        t[n + "_g"][b * G:(b + 1) * G, h]]).double()
            q, k, v, do = (part(n) for n in ("q", "k", "v", "do"))
            r = diff_ref.Diff(q, k, v, float(lam[h]), mask, (hd // 2) ** -0.5, torch.bfloat16, do)
            half = hd // 2
            P = [torch.softmax((q[:, m * half:(m + 1) * half] @ k[:, m * half:(m + 1) * half].T * half ** -0.5)
                               .masked_fill(~mask, -math.inf), 1) for m in range(2)]
            dp = do @ v.T
            ds = [c * p * (dp - (p * dp).sum(1, keepdim=True)) for c, p in zip((1.0, -float(lam[h])), P)]
            # of weights that add up to one, a common relative error drops out: P (1 - P)
            spread = sum(c * (p * (1 - p)) @ v.abs() for c, p in zip((1.0, float(lam[h])), P))
            terms = {"o": spread + r.o.abs(),
                     "dq": torch.cat([d.abs() @ k[:, m * half:(m + 1) * half].abs() * half ** -0.5
                                      for m, d in enumerate(ds)], 1)}
            for name, size in terms.items():
                got = torch.cat([out[name + "_d"][b * N:(b + 1) * N, h], out[name + "_g"][b * G:(b + 1) * G, h]])
                e = sums.setdefault(name, [0.0, 0.0])
                e[0] += float((got.double() - getattr(r, name))[few].square().sum())
                # (fp32 part: eps of the logits' terms on every weight and on dP)
                e[1] += float((2 * U * size + r.eps * (P[0] + P[1]) @ v.abs() * (1 if name == "o" else 0))
                              [few].square().sum())
    for name, (e, bound) in sums.items():
        assert e <= bound or e == 0.0, (name, e ** 0.5, bound ** 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("case", ["one global row", "windows of one row", "one row in a long list"])
def test_the_one_key_of_a_row_has_no_gradient(case, hd, dtype):
    """A softmax over one key is 1 whatever the key: dq of the row and dk from it
    are 0, not a rounding; dv is the row's (1 - lambda) do."""
    B, H = 2, 2
    lam = torch.tensor([0.3, 0.6], device=DEV)
    if case == "one global row":
        N, G, lone, off = 130, 1, [130], None
    elif case == "windows of one row":
        N, G, lone, off = 150, 0, list(range(150)), None
    else:                          # window form: windows of 200, 1 and 150 rows
        N, G, lone, off = 351, 0, [200], [0, 200, 201, 351]
    t = make(B, N, G, H, hd, dtype, seed=5)
    layout = {"window_offsets": torch.tensor(off, dtype=torch.int32, device=DEV)} if off else \
        {"window_len": 130 if G else 1}
    out = run(t, lam, B, N, G, H, **layout)
    cat = lambda src, name: torch.cat([src[name + "_" + p].view(B, -1, H, hd) for p in "dg"], 1)  # noqa: E731
    dq = cat(out, "dq")[:, lone]
    assert not dq.any(), float(dq.abs().max())
    if not G:                      # (the key of a global row is seen by detail rows too)
        assert not cat(out, "dk")[:, lone].any()
        want = cat(t, "do")[:, lone].double() * (1 - lam.double())[:, None]
        err = (cat(out, "dv")[:, lone].double() - want).abs()
        # W = 1 - lambda: each weight's logit and sum 2^-22 (hd/2 |s| + 17), W rounded (bf16), dv rounded
        u = diff_ref.unit(DT[dtype])
        assert bool((err <= want.abs() * (2 * u if dtype == "bf16" else u) + 2.0 ** -22 * (8 * hd + 17) *
                     cat(t, "do")[:, lone].double().abs()).all())


def test_gradients_against_differences():
    """Central differences of the fp32 forward along random directions, every
    input and lambda: truncation h^2 / 6 of the third derivative (bounded by 60
    |do| |dir|^3 terms at unit inputs) and rounding 2^-20 sum|do o| / h."""
    B, N, L, G, H, hd = 1, 24, 8, 5, 1, 64
    t = make(B, N, G, H, hd, "fp32")
    lam = torch.tensor([0.4], device=DEV)
    out = run(t, lam, B, N, G, H, window_len=L)

    def loss(x, l):
        o = run(x, l, B, N, G, H, window_len=L)
        return float((o["o_d"].double() * t["do_d"].double()).sum() +
                     (o["o_g"].double() * t["do_g"].double()).sum())

    h = 2.0 ** -7
    scale = float(t["do_d"].abs().sum() + t["do_g"].abs().sum())
    for n in ("q_d", "k_d", "v_d", "q_g", "k_g", "v_g"):
        dirn = rnd(*t[n].shape, seed=77)
        dirn /= dirn.norm()
        ends = [loss({**t, n: t[n] + sg * h * dirn}, lam) for sg in (1, -1)]
        want = float((out["d" + n].double() * dirn.double()).sum())
        assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 10 * h * h + 2.0 ** -20 * scale / h * 0.1, n
    ends = [loss(t, lam + sg * h) for sg in (1, -1)]     # linear in lambda
    assert abs((ends[0] - ends[1]) / (2 * h) - float(out["dlam"])) <= 2.0 ** -20 * scale / h * 0.1


def test_an_expired_wait_is_reported():
    """The forward kernel's first K tile left unloaded: its waits run out, the
    error word says so, and the context stays usable."""
    t = make(1, 256, 100, 1, 64, "bf16")
    lam = torch.tensor([0.5], device=DEV)
    o = {n: torch.empty_like(t["q_" + n]) for n in "dg"}
    args = [t[n] for n in ("q_d", "k_d", "v_d", "q_g", "k_g", "v_g")]
    atlas.debug_stall_next_attention()
    atlas.diff_attn(*args, lam, o["d"], o["g"], window_len=128)
    assert atlas.last_device_error() != 0
    assert atlas.last_device_error() == 0
    out = run(t, lam, 1, 256, 100, 1, window_len=128)
    against_reference(t, out, lam, 1, 256, 100, 1, 64, "bf16", [0, 128, 256])
