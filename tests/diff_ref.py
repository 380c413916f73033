"""Plain 64-bit forms of the differential-attention layer's operators, with the
error bounds of the library's arithmetic beside every value.

Bounds (U: half a step of the I/O type, torch.finfo(t).eps / 2):
  * an output is rounded once: U |y|;
  * bf16 attention also rounds each map's weights (forward) and the two maps'
    joint weights and dS (backward) to bf16 before their products: U times the sum
    of the products' magnitudes;
  * a weight P = exp(s - lse) carries the fp32 error of its logit (a sum of d
    products, twice: numerator and denominator), of exp and of the sum over n
    keys: eps(n) = 2^-22 (d max sum|q||k| scale + n + 16) relative;
  * D = <do, o> carries the error of the stored o.
"""
import math

import numpy as np
import torch


def unit(dtype):
    return torch.finfo(dtype).eps / 2


# ---- rotary ----------------------------------------------------------------

def rotary_omega(theta, d, k, scaling, factor, original, fast=32.0, slow=1.0):
    if scaling == "ntk" and d > 2:
        theta = theta * factor ** (d / (d - 2))
    omega = theta ** (-2.0 * k / d)
    if scaling == "by_parts":
        g = min(1.0, max(0.0, (original * omega / (2 * math.pi) - slow) / (fast - slow)))
        omega = omega * (g + (1 - g) / factor)
    return omega


def rotary(x, pos, theta, split, scales, layout, scaling="none", factor=(1, 1, 1),
           original=(0, 0, 0), magnitude=1.0, transpose=False):
    """x [rows, heads, hd] float64 numpy, pos [rows, 3] -> (y, bound without the output
    rounding). Angles in extended precision. cos and sin come from an angle in
    turns of pi held in fp32 (pi 2^-24), sincospif (2 ulp) and the magnitude's
    product, the rotation from two more roundings: below 2^-20 (|x1| + |x2|) m in all; the fp64
    angle adds 2^-50 |phi|."""
    y, err = x.copy(), np.zeros_like(x)
    base = 0
    for a, d in enumerate(split):
        for k in range(d // 2):
            c1, c2 = (base + 2 * k, base + 2 * k + 1) if layout == "interleaved" else \
                (base + k, base + k + d // 2)
            w = rotary_omega(theta, d, k, scaling, factor[a], original[a])
            phi = pos[:, a].astype(np.longdouble) * np.longdouble(scales[a]) * np.longdouble(w)
            phi = -phi if transpose else phi
            c = np.cos(phi).astype(np.float64)[:, None] * magnitude
            s = np.sin(phi).astype(np.float64)[:, None] * magnitude
            x1, x2 = x[..., c1], x[..., c2]
            y[..., c1], y[..., c2] = x1 * c - x2 * s, x1 * s + x2 * c
            e = (np.abs(x1) + np.abs(x2)) * abs(magnitude) * (
                2.0 ** -20 + 2.0 ** -50 * np.abs(phi).astype(np.float64)[:, None])
            err[..., c1] = err[..., c2] = e
        base += d
    return y, err


def cube_rows(grid, cube):
    """Raster row of every place of the cube order."""
    T, H, W = grid
    out = []
    for bt in range(0, T, cube[0]):
        for bh in range(0, H, cube[1]):
            for bw in range(0, W, cube[2]):
                for t in range(bt, min(bt + cube[0], T)):
                    for h in range(bh, min(bh + cube[1], H)):
                        for w in range(bw, min(bw + cube[2], W)):
                            out.append((t * H + h) * W + w)
    return np.array(out, dtype=np.int64)


# ---- differential attention ------------------------------------------------

def mask_of(N, G, windows, shares=None):
    """[N+G, N+G]: which keys (columns) a row sees. windows: offsets over the
    detail rows; shares: global ranges per window, None for all."""
    m = torch.zeros(N + G, N + G, dtype=torch.bool)
    for w in range(len(windows) - 1):
        a, b = windows[w], windows[w + 1]
        m[a:b, a:b] = True
        g0, g1 = (shares[w], shares[w + 1]) if shares is not None else (0, G)
        m[a:b, N + g0:N + g1] = True
    m[N:, N:] = True
    return m


class Diff:
    """One problem and head: outputs, gradients and their bounds. All inputs are
    float64 tensors [rows, D] on one device (detail rows, then global rows)."""

    def __init__(self, q, k, v, lam, mask, scale, dtype, do=None):
        h = q.shape[1] // 2
        U = unit(dtype)
        up = U if dtype == torch.bfloat16 else 0.0    # weights and dS rounded to bf16
        qs, ks = (q[:, :h], q[:, h:]), (k[:, :h], k[:, h:])
        P, A, eps, self.lse = [], [], 0.0, []
        for qm, km in zip(qs, ks):
            s = (qm @ km.T * scale).masked_fill(~mask, -math.inf)
            big = float((qm.abs() @ km.abs().T * scale).max())
            eps = max(eps, 2.0 ** -22 * (h * big + mask.shape[1] + 16))
            self.lse.append(torch.logsumexp(s, 1))
            P.append(torch.softmax(s, 1))
            A.append(P[-1] @ v.abs())
        self.eps, al = eps, abs(lam)
        o = [p @ v for p in P]
        self.s, self.o = o[1], o[0] - lam * o[1]
        err = [(up + eps) * a for a in A]
        self.s_bound = err[1] + U * o[1].abs()
        self.o_bound = err[0] + al * err[1] + U * self.o.abs()
        # an absolute error of the logit's terms
        self.lse_bound = eps
        if do is None:
            return
        dp = do @ v.T
        dp_err = eps * (do.abs() @ v.abs().T)
        D = [(do * x).sum(1, keepdim=True) for x in o]
        e2 = (do.abs() * (self.s_bound + eps * o[1].abs())).sum(1, keepdim=True)
        e1 = (do.abs() * (self.o_bound + eps * self.o.abs())).sum(1, keepdim=True) + al * e2
        dq, dk, dqb, dkb = [], [], [], []
        for c, p, d, e, qm, km in zip((1.0, -lam), P, D, (e1, e2), qs, ks):
            ds = c * p * (dp - d)
            # dS's own rounding, P's and dP's errors, D's
            de = (up + 4 * eps) * ds.abs() + abs(c) * p * (dp_err + e + 2.0 ** -23 * (dp.abs() + d.abs()))
            dq.append(ds @ km * scale)
            dk.append(ds.T @ qm * scale)
            dqb.append((de + eps * ds.abs()) @ km.abs() * scale)
            dkb.append((de + eps * ds.abs()).T @ qm.abs() * scale)
        W = P[0] - lam * P[1]
        wide = P[0] + al * P[1]
        self.dq, self.dk = torch.cat(dq, 1), torch.cat(dk, 1)
        self.dq_bound = torch.cat(dqb, 1) + U * self.dq.abs()
        self.dk_bound = torch.cat(dkb, 1) + U * self.dk.abs()
        self.dv = W.T @ do
        self.dv_bound = (up * W.abs() + 4 * eps * wide).T @ do.abs() + U * self.dv.abs()
        self.dlam = -D[1].sum()
        self.dlam_bound = e2.sum() + 2.0 ** -20 * D[1].abs().sum()


# ---- group norm --------------------------------------------------------------

def group_norm(x, gamma, beta, rows, groups, eps, silu, dtype, dy=None):
    """x [samples*rows, C] float64. Returns dict of values and "<name>_bound".
    fp32 statistics: a mean of n values by partial sums of at most n/64 + 512
    terms carries e = 2^-24 (n/64 + 512) of the mean magnitude; exp and the
    division in sigmoid 2^-20."""
    U = unit(dtype)
    M, C = x.shape
    S, cg = M // rows, C // groups
    shape = (S, rows, groups, cg)
    n = rows * cg
    e = 2.0 ** -24 * (n / 64 + 512)
    X = x.reshape(shape)
    ga = gamma.reshape(groups, cg) if gamma is not None else torch.ones(groups, cg, dtype=x.dtype, device=x.device)
    be = beta.reshape(groups, cg) if beta is not None else torch.zeros(groups, cg, dtype=x.dtype, device=x.device)
    mean = X.mean((1, 3), keepdim=True)
    var = ((X - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = (var + eps).rsqrt()
    hat = (X - mean) * rstd
    mag = X.abs().mean((1, 3), keepdim=True)
    # mean off by e mag; the variance's relative error follows from the centred sum
    hat_err = (e * mag + 2.0 ** -23 * (X.abs() + mean.abs())) * rstd + hat.abs() * (
        4 * e + 2 * (e * mag * rstd) ** 2 + 2.0 ** -22)
    z = hat * ga + be
    z_err = hat_err * ga.abs() + 2.0 ** -23 * z.abs()
    g = torch.sigmoid(z) if silu else torch.ones_like(z)
    y = z * g
    y_err = z_err * (1.1 if silu else 1.0) + (2.0 ** -20 * y.abs() if silu else 0.0)
    out = {"y": y, "y_bound": y_err + U * y.abs(), "mean": mean.reshape(S, groups),
           "mean_bound": (e * mag + 2.0 ** -23 * mean.abs()).reshape(S, groups),
           "rstd": rstd.reshape(S, groups),
           "rstd_bound": (rstd * (4 * e + 2 * (e * mag * rstd) ** 2 + 2.0 ** -22)).reshape(S, groups)}
    if dy is not None:
        DY = dy.reshape(shape)
        slope = g + z * g * (1 - g) if silu else torch.ones_like(z)
        dz = DY * slope
        # |act''| <= 1/2; the stored statistics are the library's own
        dz_err = DY.abs() * (0.5 * z_err * silu + 2.0 ** -20 * slope.abs() + 2.0 ** -20 * silu)
        dh, dh_err = dz * ga, dz_err * ga.abs() + 2.0 ** -24 * (dz * ga).abs()
        m1, m2 = dh.mean((1, 3), keepdim=True), (dh * hat).mean((1, 3), keepdim=True)
        m1_err = dh_err.mean((1, 3), keepdim=True) + e * dh.abs().mean((1, 3), keepdim=True)
        m2_err = (dh_err * hat.abs() + dh.abs() * hat_err).mean((1, 3), keepdim=True) + \
            e * (dh * hat).abs().mean((1, 3), keepdim=True)
        core = dh - m1 - hat * m2
        dx = rstd * core
        rel = 4 * e + 2 * (e * mag * rstd) ** 2 + 2.0 ** -22
        dx_err = rstd * (dh_err + m1_err + hat.abs() * m2_err + hat_err * m2.abs() +
                         2.0 ** -22 * (dh.abs() + m1.abs() + (hat * m2).abs())) + rel * dx.abs()
        big = 2.0 ** -24 * (M / 64 + 512)
        out |= {"dx": dx, "dx_bound": dx_err + U * dx.abs(),
                "dgamma": (dz * hat).sum((0, 1)).reshape(C),
                "dgamma_bound": (dz_err * hat.abs() + dz.abs() * hat_err + big * (dz * hat).abs()).sum((0, 1)).reshape(C),
                "dbeta": dz.sum((0, 1)).reshape(C),
                "dbeta_bound": (dz_err + big * dz.abs()).sum((0, 1)).reshape(C)}
    return {k: (v.reshape(M, C) if v.dim() == 4 else v) for k, v in out.items()}


def check(name, got, want, bound):
    got = torch.as_tensor(got, dtype=torch.float64, device=want.device)
    assert got.shape == want.shape, f"{name}: shape {tuple(got.shape)} for {tuple(want.shape)}"
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    over = (got - want).abs() - bound - 2.0 ** -133
    assert float(over.max()) <= 0.0, (
        f"{name}: error {float((got - want).abs().max()):.3e}, {int((over > 0).sum())} of "
        f"{over.numel()} out of bound (bound there {float(bound.reshape(-1)[over.argmax()]):.3e})")
