"""Cases of the differential-attention layer's operators, and their plain forms.

Three operators that stand in a row in such a layer: rotary positions (`rotary`), differential
attention over the framework's windows and global tokens (`diff`), and group norm, channels last,
with an activation (`norm`), which also normalises the heads of the attention's output.
`own` false: elementary torch operations in 32 bits (64 for angles); `own` true: the framework's calls.
"""
import itertools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rotary_case(name, grid, cube, order, tensors, head_dim, split, layout, dtype, fused=False,
                positions=0, scaling="none", factor=1.0, original=1.0, transpose=False,
                scales=(1.0, 1.0, 1.0), batch=1):
    """tensors: heads of every tensor of the call, as text, with a "v" before one that moves without rotating."""
    return {"name": name, "op": "rotary", "dtype": dtype, "batch": batch, "T": grid[0], "H": grid[1],
            "W": grid[2], "ct": cube[0], "ch": cube[1], "cw": cube[2], "order": order, "tensors": tensors,
            "head_dim": head_dim, "d_t": split[0], "d_h": split[1], "d_w": split[2], "layout": layout,
            "fused": fused, "positions": positions, "scaling": scaling, "factor": factor,
            "original": original, "transpose": transpose, "s_t": scales[0], "s_h": scales[1],
            "s_w": scales[2]}


def diff_case(name, train, dtype, batch, heads, head_dim, global_rows, window_len=0, windows=0,
              grid=(0, 0, 0), cube=(1, 1, 1), aligned=False, shared_lambda=False):
    """windows > 0: that many windows of window_len rows; else the windows of `grid` cut into `cube`
    (partial cubes at its edges), or no detail rows at all. aligned: a window's queries see a
    share of the global rows of its own instead of all."""
    return {"name": name, "op": "diff", "train": train, "dtype": dtype, "batch": batch, "heads": heads,
            "head_dim": head_dim, "global_rows": global_rows, "window_len": window_len,
            "windows": windows, "T": grid[0], "H": grid[1], "W": grid[2], "ct": cube[0], "ch": cube[1],
            "cw": cube[2], "aligned": aligned, "shared_lambda": shared_lambda}


def norm_case(name, train, dtype, samples, rows, channels, groups, silu):
    return {"name": name, "op": "norm", "train": train, "dtype": dtype, "samples": samples, "rows": rows,
            "channels": channels, "groups": groups, "silu": silu}


def listed():
    return [
        # 256 tokens of two heads in fp32: the path's smallest call, where the launch is what it costs
        rotary_case("rotary_tiny", (4, 8, 8), (2, 4, 4), "reorder", "2,2,v2", 64, (16, 24, 24),
                    "interleaved", "fp32"),
        # one 720p layer: Q, K (rotated) and V (moved only) out of one fused projection into cube order
        rotary_case("rotary_720p", (21, 48, 80), (3, 16, 16), "reorder", "40,40,v40", 128, (44, 42, 42),
                    "half", "bf16", fused=True),
        # packed sequences with a position per token, half of the head rotated, fewer K than Q heads,
        # frequencies interpolated by parts for a context sixteen times the trained one
        rotary_case("rotary_positions", (1, 1, 65537), (1, 1, 1), "raster", "40,8", 128, (64, 0, 0),
                    "half", "bf16", positions=131072, scaling="by_parts", factor=16.0, original=8192.0),
        # the gradient's way back from partial cubes of the 8K grid: rotation undone, raster order,
        # the temporal axis stretched by a larger base
        rotary_case("rotary_grad", (8, 270, 480), (3, 16, 16), "unorder", "2,2", 128, (44, 42, 42),
                    "interleaved", "bf16", scaling="ntk", factor=4.0, transpose=True),
        # a training step on 256 tokens in fp32: eight launches' latency
        diff_case("diff_tiny", True, "fp32", 1, 2, 64, 32, window_len=32, windows=8),
        # 720p inference, one tenth of the heads: windows of 768 rows and 5,040 global tokens
        diff_case("diff_720p", False, "bf16", 1, 4, 128, 5040, window_len=768, windows=105),
        # the proxy alone: full attention over 32,760 global tokens, heads of 64
        diff_case("diff_global", False, "bf16", 1, 1, 64, 32760),
        # training on two small clips whose cubes do not divide the grid, aligned global tokens
        diff_case("diff_partial", True, "bf16", 2, 4, 64, 301, grid=(5, 18, 26), cube=(3, 8, 8),
                  aligned=True, shared_lambda=True),
        # 720p training, one head: forward and gradients
        diff_case("diff_720p_train", True, "bf16", 1, 1, 128, 5040, window_len=768, windows=105),
        # the heads of a 720p layer's attention output, each token's head normalised by itself
        norm_case("norm_heads", False, "bf16", 80640, 1, 5120, 40, False),
        # a hidden layer of a video decoder: 21 frames of 96 x 160, SiLU, forward and gradients
        norm_case("norm_latent", True, "bf16", 2, 322560, 128, 32, True),
        # three short odd clips in fp32: groups of five channels
        norm_case("norm_small", True, "fp32", 3, 1001, 60, 12, True),
    ]


def spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "diff", "diff", "diff", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "rotary":
        head_dim = rng.choice([32, 64, 80, 96, 128])
        half = head_dim // 2
        d_t = 2 * rng.randint(1, half // 3)
        d_h = 2 * rng.randint(0, half // 3)
        d_w = 2 * rng.randint(0, half // 3)
        T, H, W = spread(rng, 1, 42), spread(rng, 1, 144), spread(rng, 1, 240)
        heads = [rng.randint(1, 16) for _ in range(rng.randint(1, 3))]
        batch = rng.randint(1, 2)
        limit = (1 << 29) // (batch * T * H * W * head_dim)
        heads = [max(1, min(h, limit // len(heads))) for h in heads]
        positions = rng.choice([0, 0, spread(rng, 100, 1 << 20)])
        order = "raster" if positions else rng.choice(["raster", "reorder", "unorder"])
        return rotary_case(
            "", (T, H, W), (rng.randint(1, 4), rng.randint(1, 16), rng.randint(1, 16)), order,
            ",".join(str(h) for h in heads), head_dim, (d_t, d_h, d_w),
            rng.choice(["half", "interleaved"]), dtype, fused=rng.random() < 0.5, positions=positions,
            scaling=rng.choice(["none", "ntk", "by_parts"]), factor=rng.uniform(1.0, 32.0),
            original=float(spread(rng, 16, 8192)), transpose=rng.random() < 0.3,
            scales=(rng.choice([1.0, 2.0, 4.0]), rng.choice([1.0, 8.0]), 1.0), batch=batch)
    if op == "diff":
        train = rng.random() < 0.5
        head_dim = rng.choice([64, 128])
        shared = rng.random() < 0.3
        if rng.random() < 0.5:
            window_len = spread(rng, 1, 1536)
            windows = spread(rng, 1, max(1, 20000 // window_len))
            most = 6_000_000 if dtype == "fp32" else 60_000_000
            global_rows = spread(rng, 1, 4096)
            while global_rows > 1 and (windows * (window_len + global_rows) > 500_000 or window_len * windows * (
                    window_len + global_rows) + global_rows ** 2 > most):
                global_rows, windows = global_rows // 2, max(1, windows // 2)
            return diff_case("", train, dtype, rng.randint(1, 2), rng.randint(1, 3), head_dim, global_rows,
                             window_len=window_len, windows=windows, shared_lambda=shared)
        side = 3 if dtype == "bf16" else 1
        grid = (rng.randint(1, 5), rng.randint(1, 8 * side), rng.randint(1, 8 * side))
        cube = (rng.randint(1, 3), rng.randint(1, 12), rng.randint(1, 12))
        return diff_case("", train, dtype, rng.randint(1, 2), rng.randint(1, 3), head_dim,
                         spread(rng, 1, 700), grid=grid, cube=cube, aligned=rng.random() < 0.5,
                         shared_lambda=shared)
    groups = rng.choice([1, 4, 8, 12, 32, 40])
    channels = groups * rng.choice([16, 20, 32, 64, 128])
    if rng.random() < 0.4:
        samples, rows = spread(rng, 1, 80640), spread(rng, 1, 8)
    elif rng.random() < 0.3:
        channels, samples, rows = groups * rng.choice([1, 2, 5, 8]), rng.randint(1, 4), spread(rng, 50, 300000)
    else:
        samples, rows = rng.randint(1, 4), spread(rng, 1, 300000)
    rows = max(1, min(rows, (1 << 26) // channels // samples))
    return norm_case("", rng.random() < 0.6, dtype, min(samples, (1 << 26) // channels), rows, channels, groups,
                     rng.random() < 0.6)


def heads_of(case):
    return [(int(h.lstrip("v")), not h.startswith("v")) for h in case["tensors"].split(",")]


def windows_of(case):
    """Detail rows and global rows of each window, as boundaries."""
    if case["windows"]:
        offsets = [w * case["window_len"] for w in range(case["windows"] + 1)]
    else:
        t, h, w = ([min(c, n - s) for s in range(0, n, c)] for n, c in
                   ((case["T"], case["ct"]), (case["H"], case["ch"]), (case["W"], case["cw"])))
        offsets = list(itertools.accumulate((a * b * c for a in t for b in h for c in w), initial=0))
    n, g = len(offsets) - 1, case["global_rows"]
    return offsets, [w * g // max(n, 1) for w in range(n + 1)]


def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, kind=dtype):
        return torch.randn(shape, generator=gen, device=device, dtype=torch.float32).mul_(std).to(kind)

    state = {"case": case}
    if case["op"] == "rotary":
        heads, hd = heads_of(case), case["head_dim"]
        rows = case["batch"] * case["T"] * case["H"] * case["W"]
        if case["fused"]:
            # one buffer [rows, all heads], as a projection leaves it: each tensor is a slice of its columns
            whole = normal(rows, sum(h for h, _ in heads), hd)
            starts = [sum(h for h, _ in heads[:i]) for i in range(len(heads))]
            state["src"] = [whole[:, s:s + h] for s, (h, _) in zip(starts, heads)]
        else:
            state["src"] = [normal(rows, h, hd) for h, _ in heads]
        state["dst"] = [torch.empty(rows, h, hd, dtype=dtype, device=device) for h, _ in heads]
        state["positions"] = None
        if case["positions"]:
            axes = 1 if case["d_h"] + case["d_w"] == 0 else 3
            state["positions"] = torch.randint(0, case["positions"], (rows, axes), generator=gen,
                                               device=device, dtype=torch.int32)
        return state
    if case["op"] == "diff":
        offsets, shares = windows_of(case)
        B, H, D, N, G = case["batch"], case["heads"], case["head_dim"], offsets[-1], case["global_rows"]
        for part, n in (("d", B * N), ("g", B * G)):
            for name in ("q", "k", "v", "do"):
                state[name + "_" + part] = normal(n, H, D)
            for name in ("o", "s", "dq", "dk", "dv"):
                state[name + "_" + part] = torch.empty(n, H, D, dtype=dtype, device=device)
        n = 1 if case["shared_lambda"] else H
        state["vectors"] = [normal(n, D // 2, std=0.1) for _ in range(4)]
        state["dvectors"] = [torch.empty_like(v) for v in state["vectors"]]
        state["lam"], state["dlam"] = (torch.empty(n, dtype=torch.float32, device=device) for _ in range(2))
        state["lambda_init"] = 0.8 - 0.6 * math.exp(-0.3 * 4)
        state["lse"] = torch.empty(B, H, 2, N + G, dtype=torch.float32, device=device)
        state["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=device)
        state["shares"] = torch.tensor(shares, dtype=torch.int32, device=device)
        state["work"] = torch.empty(B * H * 2 * (N + G) + 4096 * H, dtype=torch.float32, device=device)
        return state
    M, C = case["samples"] * case["rows"], case["channels"]
    state["x"] = normal(M, C) + normal(1, C)
    state["dy"] = normal(M, C)
    state["gamma"] = normal(C, std=0.2, kind=torch.float32) + 1
    state["beta"] = normal(C, std=0.2, kind=torch.float32)
    state["y"], state["dx"] = torch.empty_like(state["x"]), torch.empty_like(state["x"])
    state["dgamma"], state["dbeta"] = torch.empty_like(state["gamma"]), torch.empty_like(state["beta"])
    state["stats"] = torch.empty(case["samples"], case["groups"], 2, dtype=torch.float32, device=device)
    return state


# ---- plain forms -------------------------------------------------------------------------------


def frequencies(case, width, kind=torch.float64):
    """Angle per position of each of the width / 2 pairs of one axis (scaled for a longer context)."""
    k = torch.arange(width // 2, dtype=kind, device="cuda")
    theta, s = 10000.0, case["factor"]
    if case["scaling"] == "ntk" and width > 2:
        theta = theta * s ** (width / (width - 2))
    omega = theta ** (-2.0 * k / width) if width else k
    if case["scaling"] == "by_parts":
        turns = case["original"] * omega / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        omega = omega * (keep + (1 - keep) / s)
    return omega


def magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0


def grid_index(case):
    """Index along each axis of the tokens of one problem, in raster order."""
    axes = [torch.arange(case[a], device="cuda") for a in "THW"]
    return [x.reshape(-1) for x in torch.meshgrid(*axes, indexing="ij")]


def cube_order(case):
    """Raster row of every place of the cube order (all problems)."""
    t, h, w = grid_index(case)
    n_h, n_w = -(-case["H"] // case["ch"]), -(-case["W"] // case["cw"])
    cube = (t // case["ct"] * n_h + h // case["ch"]) * n_w + w // case["cw"]
    order = torch.argsort(cube, stable=True)
    first = torch.arange(case["batch"], device="cuda")[:, None] * order.numel()
    return (first + order).reshape(-1)


def pair_channels(case):
    """First and second channel of every rotated pair, and the axis it turns with."""
    widths = [case["d_t"], case["d_h"], case["d_w"]]
    k = [torch.arange(d // 2, device="cuda") for d in widths]
    start = [0, widths[0], widths[0] + widths[1]]
    if case["layout"] == "half":
        first = torch.cat([s + x for s, x in zip(start, k)])
        second = torch.cat([s + x + d // 2 for s, x, d in zip(start, k, widths)])
    else:
        first = torch.cat([s + 2 * x for s, x in zip(start, k)])
        second = first + 1
    axis = torch.cat([torch.full_like(x, a) for a, x in enumerate(k)])
    return first, second, axis


def positions_of(state):
    """[rows, axes] positions in raster order, scaled, in 64 bits."""
    case = state["case"]
    scale = torch.tensor([case["s_t"], case["s_h"], case["s_w"]], dtype=torch.float64, device="cuda")
    if state["positions"] is not None:
        return state["positions"].double() * scale[:state["positions"].shape[1]]
    return (torch.stack(grid_index(case), dim=1).double() * scale).repeat(case["batch"], 1)


def plain_rotary(state):
    case = state["case"]
    first, second, axis = pair_channels(case)
    omega = torch.cat([frequencies(case, case[d]) for d in ("d_t", "d_h", "d_w")])
    angle = positions_of(state)[:, axis] * omega
    angle = -angle if case["transpose"] else angle
    cos = (angle.cos() * magnitude(case)).float()[:, None, :]
    sin = (angle.sin() * magnitude(case)).float()[:, None, :]
    order = cube_order(case) if case["order"] != "raster" else None

    def turn(x, rotated):
        if case["order"] == "unorder":
            y = torch.empty_like(x, memory_format=torch.contiguous_format)
            y[order] = x
        else:
            y = x.clone(memory_format=torch.contiguous_format)
        if rotated:
            a, b = y[..., first].float(), y[..., second].float()
            y[..., first] = (a * cos - b * sin).to(y.dtype)
            y[..., second] = (a * sin + b * cos).to(y.dtype)
        return y[order] if case["order"] == "reorder" else y

    return [turn(x, rotated) for x, (_, rotated) in zip(state["src"], heads_of(case))]


def attend(q, k, v, lam, scale, mask, do):
    """Differential attention of [X, H, rows, 2, d] queries over keys of the same layout and
    [X, H, keys, D] values; with `do` also its gradients."""
    s = torch.matmul(q.transpose(2, 3), k.permute(0, 1, 3, 4, 2)) * scale  # [X, H, 2, rows, keys]
    if mask is not None:
        s = s.masked_fill(~mask, -math.inf)
    s = s - s.amax(dim=-1, keepdim=True)
    p = s.exp_()
    p = p / p.sum(dim=-1, keepdim=True)
    both = p[:, :, 0] - lam[:, None, None] * p[:, :, 1]
    o = torch.matmul(both, v)
    if do is None:
        return o, None
    dp = torch.matmul(do, v.transpose(-1, -2))
    mean = (p * dp[:, :, None]).sum(dim=-1, keepdim=True)  # [X, H, 2, rows, 1]
    weight = torch.stack([torch.ones_like(lam), -lam], dim=1)[:, :, None, None]
    ds = p * (dp[:, :, None] - mean) * weight * scale
    dq = torch.matmul(ds, k.transpose(2, 3)).transpose(2, 3)
    dk = torch.matmul(ds.transpose(-1, -2), q.transpose(2, 3)).transpose(2, 3)
    dv = torch.matmul(both.transpose(-1, -2), do)
    return o, (dq, dk, dv, -mean[:, :, 1].sum(dim=(0, 2, 3)))


def dense_mask(offsets, shares, N, G):
    """Which of the N + G keys each of the N + G rows sees."""
    row = torch.arange(N + G, device="cuda")
    window = torch.searchsorted(offsets, row, right=True) - 1
    share = torch.searchsorted(shares, row - N, right=True) - 1
    detail = row < N
    own_window = detail[None, :] & (window[:, None] == window[None, :])
    own_share = ~detail[None, :] & (window[:, None] == share[None, :])
    return torch.where(detail[:, None], own_window | own_share, ~detail[None, :])


def plain_diff(state):
    case = state["case"]
    B, H, D, G = case["batch"], case["heads"], case["head_dim"], case["global_rows"]
    N, L, W = state["q_d"].shape[0] // B, case["window_len"], case["windows"]
    scale, train = (D // 2) ** -0.5, case["train"]
    vec = [x.float() for x in state["vectors"]]
    e1, e2 = (vec[0] * vec[1]).sum(-1).exp(), (vec[2] * vec[3]).sum(-1).exp()
    lam = (e1 - e2 + state["lambda_init"]).expand(H)

    def split(name, part, rows, last):
        x = state[name + "_" + part].float().reshape(-1, rows, H, *last).transpose(1, 2)
        return x

    maps = (2, D // 2)
    if W or not N:
        # every detail row of a window sees the same keys: the window's, then the global ones
        kg, vg = split("k", "g", G, maps), split("v", "g", G, (D,))
        dog = split("do", "g", G, (D,)) if train else None
        og, gg = attend(split("q", "g", G, maps), kg, vg, lam, scale, None, dog)
        if N:
            kd = torch.cat([split("k", "d", L, maps), kg.repeat_interleave(W, dim=0)], dim=2)
            vd = torch.cat([split("v", "d", L, (D,)), vg.repeat_interleave(W, dim=0)], dim=2)
            dod = split("do", "d", L, (D,)) if train else None
            od, gd = attend(split("q", "d", L, maps), kd, vd, lam, scale, None, dod)
        out_d = [od] if N else []
        if train:
            dq, dk, dv, dlam = gg
            if N:
                out_d += [gd[0], gd[1][:, :, :L], gd[2][:, :, :L]]
                dk = dk + gd[1][:, :, L:].unflatten(0, (B, W)).sum(dim=1)
                dv = dv + gd[2][:, :, L:].unflatten(0, (B, W)).sum(dim=1)
                dlam = dlam + gd[3]
            out_g = [og, dq, dk, dv]
        else:
            out_g = [og]
    else:
        kinds = (("q", maps), ("k", maps), ("v", (D,)), ("do", (D,)))
        q, k, v, do = (torch.cat([split(n, "d", N, last), split(n, "g", G, last)], dim=2) for n, last in kinds)
        mask = dense_mask(state["offsets"], state["shares"], N, G)
        if not case["aligned"]:
            row = torch.arange(N + G, device="cuda")
            mask = mask | ((row >= N)[None, :] & (row < N)[:, None])
        o, g = attend(q, k, v, lam, scale, mask, do if train else None)
        whole = [o, *g[:3]] if train else [o]
        out_d, out_g = [x[:, :, :N] for x in whole], [x[:, :, N:] for x in whole]
        dlam = g[3] if train else None

    dtype = DTYPES[case["dtype"]]
    names = ("o", "dq", "dk", "dv")
    out = {n + "_d": x.transpose(1, 2).reshape(B * N, H, D).to(dtype) for n, x in zip(names, out_d)}
    out |= {n + "_g": x.transpose(1, 2).reshape(B * G, H, D).to(dtype) for n, x in zip(names, out_g)}
    if train:
        dlam = dlam.sum(dim=0, keepdim=True) if case["shared_lambda"] else dlam
        a, b = (dlam * e1)[:, None], (-dlam * e2)[:, None]
        out["dvectors"] = [x.to(dtype) for x in (a * vec[1], a * vec[0], b * vec[3], b * vec[2])]
    return out


def plain_norm(state):
    case = state["case"]
    shape = (case["samples"], case["rows"], case["groups"], case["channels"] // case["groups"])
    gamma, beta = (state[n].reshape(shape[2:]) for n in ("gamma", "beta"))
    x = state["x"].float().reshape(shape)
    mean = x.mean(dim=(1, 3), keepdim=True)
    rstd = ((x - mean).square().mean(dim=(1, 3), keepdim=True) + 1e-5).rsqrt()
    hat = (x - mean) * rstd
    z = hat * gamma + beta
    gate = 1 / (1 + (-z).exp()) if case["silu"] else None
    y = z * gate if case["silu"] else z
    back = lambda a: a.reshape(-1, case["channels"]).to(state["x"].dtype)  # noqa: E731
    if not case["train"]:
        return back(y)
    dz = state["dy"].float().reshape(shape)
    dz = dz * (gate * (1 + z * (1 - gate))) if case["silu"] else dz
    dgamma, dbeta = (dz * hat).sum(dim=(0, 1)).reshape(-1), dz.sum(dim=(0, 1)).reshape(-1)
    dh = dz * gamma
    dx = rstd * (dh - dh.mean(dim=(1, 3), keepdim=True) - hat * (dh * hat).mean(dim=(1, 3), keepdim=True))
    return back(y), back(dx), dgamma, dbeta


# ---- the framework's calls ---------------------------------------------------------------------


def own_rotary(state):
    from video_dit_windowed_b200 import atlas
    case = state["case"]
    rot = atlas.make_rotary(10000.0, (case["d_t"], case["d_h"], case["d_w"]),
                            (case["s_t"], case["s_h"], case["s_w"]), layout=case["layout"],
                            scaling=case["scaling"], factor=(case["factor"],) * 3,
                            original=(case["original"],) * 3, beta_fast=32.0, beta_slow=1.0,
                            magnitude=magnitude(case))
    atlas.rotary([(s, d, r) for s, d, (_, r) in zip(state["src"], state["dst"], heads_of(case))],
                 (case["T"], case["H"], case["W"]), rot, cube=(case["ct"], case["ch"], case["cw"]),
                 order=case["order"], positions=state["positions"], transpose=case["transpose"],
                 batch=case["batch"])
    return state["dst"]


def own_diff(state):
    from video_dit_windowed_b200 import atlas
    case, t = state["case"], state
    layout = {"batch": case["batch"]}
    if case["windows"]:
        layout["window_len"] = case["window_len"]
    elif t["q_d"].shape[0]:
        layout["window_offsets"] = t["offsets"]
    if case["aligned"]:
        layout["global_window_offsets"] = t["shares"]
    atlas.diff_lambda(*t["vectors"], t["lambda_init"], t["lam"])
    ins = (t["q_d"], t["k_d"], t["v_d"], t["q_g"], t["k_g"], t["v_g"])
    parts = ("d", "g") if t["q_d"].shape[0] else ("g",)
    if not case["train"]:
        atlas.diff_attn(*ins, t["lam"], t["o_d"], t["o_g"], **layout)
        return {"o_" + p: t["o_" + p] for p in parts}
    atlas.diff_attn(*ins, t["lam"], t["o_d"], t["o_g"], t["s_d"], t["s_g"], t["lse"], **layout)
    atlas.diff_attn_bwd(t["q_d"], t["k_d"], t["v_d"], t["o_d"], t["s_d"], t["do_d"], t["q_g"], t["k_g"],
                        t["v_g"], t["o_g"], t["s_g"], t["do_g"], t["lam"], t["lse"], t["dq_d"], t["dk_d"],
                        t["dv_d"], t["dq_g"], t["dk_g"], t["dv_g"], t["dlam"], **layout)
    atlas.diff_lambda_bwd(*t["vectors"], t["dlam"], *t["dvectors"])
    out = {n + "_" + p: t[n + "_" + p] for p in parts for n in ("o", "dq", "dk", "dv")}
    out["dvectors"] = t["dvectors"]
    return out


def own_norm(state):
    from video_dit_windowed_b200 import atlas
    case = state["case"]
    act = "silu" if case["silu"] else "none"
    atlas.group_norm(state["x"], state["gamma"], state["beta"], state["y"], case["rows"], case["groups"],
                     eps=1e-5, activation=act, stats=state["stats"] if case["train"] else None)
    if not case["train"]:
        return state["y"]
    atlas.group_norm_bwd(state["dy"], state["x"], state["gamma"], state["beta"], state["stats"], state["dx"],
                         state["dgamma"], state["dbeta"], case["rows"], case["groups"], activation=act)
    return state["y"], state["dx"], state["dgamma"], state["dbeta"]


def run(state):
    op = state["case"]["op"]
    if own:
        return own_rotary(state) if op == "rotary" else own_diff(state) if op == "diff" else own_norm(state)
    return plain_rotary(state) if op == "rotary" else plain_diff(state) if op == "diff" else plain_norm(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        rows = case["batch"] * case["T"] * case["H"] * case["W"]
        heads, turned = sum(h for h, _ in heads_of(case)), sum(h for h, r in heads_of(case) if r)
        rot = case["d_t"] + case["d_h"] + case["d_w"]
        axes = (1 if case["d_h"] + case["d_w"] == 0 else 3) if case["positions"] else 0
        return {"bytes": rows * (2 * heads * case["head_dim"] * size + 4 * axes), "flops": 3 * rows * turned * rot}
    if case["op"] == "diff":
        offsets, shares = windows_of(case)
        N, G, D = offsets[-1], case["global_rows"], case["head_dim"]
        seen = [(b - a, (d - c) if case["aligned"] else G) for a, b, c, d in
                zip(offsets, offsets[1:], shares, shares[1:])]
        pairs = sum(l * (l + g) for l, g in seen) + G * G
        rows, cells = N + G, case["batch"] * case["heads"]
        # two maps' logits (D) and their two products with V (2 D), a multiply and an add each
        flops, tensors = 6 * D, 4
        if case["train"]:
            # logits again, dO V^T, dV, dQ, dK: five products of width D
            flops, tensors = flops + 10 * D, 4 + 4
        return {"bytes": cells * rows * D * size * tensors, "flops": cells * pairs * flops}
    n = case["samples"] * case["rows"] * case["channels"]
    return {"bytes": n * size * (4 if case["train"] else 2), "flops": n * (24 if case["train"] else 8)}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)

    def frequency(d, k):
        theta = 10000.0
        if case["scaling"] == "ntk" and d > 2:
            theta *= case["factor"] ** (d / (d - 2))
        omega = theta ** (-2 * k / d)
        if case["scaling"] == "by_parts":
            share = min(1.0, max(0.0, (case["original"] * omega / (2 * math.pi) - 1) / 31))
            omega = share * omega + (1 - share) * omega / case["factor"]
        return omega

    def rotary():
        widths, scales = (case["d_t"], case["d_h"], case["d_w"]), (case["s_t"], case["s_h"], case["s_w"])
        rows = case["T"] * case["H"] * case["W"]
        index = torch.arange(rows, device="cuda")
        where = [index // (case["H"] * case["W"]), index // case["W"] % case["H"], index % case["W"]]
        rank = torch.zeros_like(index)
        for axis, cube, extent in zip(where, ("ct", "ch", "cw"), "THW"):
            rank = rank * -(-case[extent] // case[cube]) + axis // case[cube]
        place = torch.empty_like(index)
        place[torch.sort(rank, stable=True).indices] = index  # cube-order place of each raster row
        outs = []
        for x, (_, rotated) in zip(state["src"], heads_of(case)):
            x = x.unflatten(0, (case["batch"], rows))
            y = (x[:, place] if case["order"] == "unorder" else x).double()
            if rotated:
                base = 0
                for a, d in enumerate(widths):
                    if d == 0:
                        continue
                    seg = y[..., base:base + d]
                    pair = seg.unflatten(-1, (2, d // 2)).transpose(-1, -2) if case["layout"] == "half" \
                        else seg.unflatten(-1, (d // 2, 2))
                    z = torch.view_as_complex(pair.contiguous())
                    p = where[a].double().expand(case["batch"], rows) if state["positions"] is None \
                        else state["positions"][:, a].double().unflatten(0, (case["batch"], rows))
                    freq = torch.tensor([frequency(d, k) for k in range(d // 2)], device="cuda",
                                        dtype=torch.float64)
                    phi = (p * scales[a])[..., None, None] * freq * (-1 if case["transpose"] else 1)
                    z = torch.view_as_real(z * torch.polar(torch.full_like(phi, magnitude(case)), phi))
                    y[..., base:base + d] = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" \
                        else z.flatten(-2)
                    base += d
            if case["order"] == "reorder":
                moved = torch.empty_like(y)
                moved[:, place] = y
                y = moved
            outs.append(y.flatten(0, 1))
        return outs

    def diff():
        offsets, shares = windows_of(case)
        B, H, D, N, G = case["batch"], case["heads"], case["head_dim"], offsets[-1], case["global_rows"]
        train, scale, half = case["train"], (D // 2) ** -0.5, D // 2
        a1, b1, a2, b2 = (x.double() for x in state["vectors"])
        e1, e2 = torch.exp((a1 * b1).sum(1)), torch.exp((a2 * b2).sum(1))
        lam = (e1 - e2 + state["lambda_init"]).expand(H)
        out = {n + "_" + p: torch.zeros(B * r, H, D, dtype=torch.float64, device="cuda")
               for p, r in (("d", N), ("g", G)) if r for n in (("o", "dq", "dk", "dv") if train else ("o",))}
        dlam = torch.zeros(H, dtype=torch.float64, device="cuda")
        jobs = [("d", offsets[w], offsets[w + 1], shares[w] if case["aligned"] else 0,
                 shares[w + 1] if case["aligned"] else G) for w in range(len(offsets) - 1)]
        jobs += [("g", s, min(s + 1024, G), 0, G) for s in range(0, G, 1024)]
        if len(jobs) * B * H > 20000:
            return None
        for b in range(B):
            for h in range(H):
                for part, r0, r1, g0, g1 in jobs:
                    if part == "d" and r0 == r1:
                        continue
                    rows = slice(b * (N if part == "d" else G) + r0, b * (N if part == "d" else G) + r1)
                    near = [("d", rows)] if part == "d" else []
                    keys = near + [("g", slice(b * G + g0, b * G + g1))]
                    q = state["q_" + part][rows, h].double()
                    k = torch.cat([state["k_" + p][r, h] for p, r in keys]).double()
                    v = torch.cat([state["v_" + p][r, h] for p, r in keys]).double()
                    p1 = torch.softmax(q[:, :half] @ k[:, :half].T * scale, dim=1)
                    p2 = torch.softmax(q[:, half:] @ k[:, half:].T * scale, dim=1)
                    out["o_" + part][rows, h] = p1 @ v - lam[h] * (p2 @ v)
                    if not train:
                        continue
                    do = state["do_" + part][rows, h].double()
                    dp = do @ v.T
                    d1, d2 = (p1 * dp).sum(1, keepdim=True), (p2 * dp).sum(1, keepdim=True)
                    s1, s2 = p1 * (dp - d1) * scale, -lam[h] * p2 * (dp - d2) * scale
                    dlam[h] -= d2.sum()
                    out["dq_" + part][rows, h] = torch.cat([s1 @ k[:, :half], s2 @ k[:, half:]], dim=1)
                    dk = torch.cat([s1.T @ q[:, :half], s2.T @ q[:, half:]], dim=1)
                    dv = (p1 - lam[h] * p2).T @ do
                    at = 0
                    for p, r in keys:
                        n = r.stop - r.start
                        out["dk_" + p][r, h] += dk[at:at + n]
                        out["dv_" + p][r, h] += dv[at:at + n]
                        at += n
        if train:
            dlam = dlam.sum().reshape(1) if case["shared_lambda"] else dlam
            x, y = (dlam * e1)[:, None], (dlam * e2)[:, None]
            out["dvectors"] = [x * b1, x * a1, -y * b2, -y * a2]
        return out

    def norm():
        S, R, C, K = case["samples"], case["rows"], case["channels"], case["groups"]
        x = state["x"].double().view(S, R, K, C // K).transpose(1, 2).flatten(2)  # [S, K, R * C / K]
        var, mean = torch.var_mean(x, dim=2, correction=0, keepdim=True)
        hat = ((x - mean) / torch.sqrt(var + 1e-5)).unflatten(2, (R, C // K))
        gamma, beta = (state[n].double().view(1, K, 1, C // K) for n in ("gamma", "beta"))
        z = gamma * hat + beta
        gate = torch.sigmoid(z) if case["silu"] else torch.ones_like(z)
        flat = lambda a: a.transpose(1, 2).reshape(S * R, C)  # noqa: E731
        y = flat(z * gate)
        if not case["train"]:
            return y
        dz = state["dy"].double().view(S, R, K, C // K).transpose(1, 2)
        if case["silu"]:
            dz = dz * (gate + z * gate * (1 - gate))
        dgamma, dbeta = (dz * hat).sum((0, 2)).reshape(C), dz.sum((0, 2)).reshape(C)
        dh = dz * gamma
        m1, m2 = dh.mean((2, 3), keepdim=True), (dh * hat).mean((2, 3), keepdim=True)
        dx = (dh - m1 - hat * m2) / torch.sqrt(var + 1e-5).unsqueeze(3)
        return y, flat(dx), dgamma, dbeta

    return {"rotary": rotary, "diff": diff, "norm": norm}[case["op"]]()
