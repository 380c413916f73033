"""Group norm: addresses, lengths and values at the edges of what the call allows."""
import pytest
import torch

from test_gpu_group_norm import DEV, DT, rnd
from video_dit_windowed_b200 import atlas

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", [(301, 1, 1280, 10), (5, 9, 24, 3), (2, 9000, 64, 4)], ids=str)
def test_fp32_arrays_on_a_4_byte_boundary(case, dtype):
    """stats, gamma, beta, dgamma and dbeta one float behind a 16-byte boundary: the
    same bits as on one, in each of the three forms."""
    S, R, C, K = case
    x, dy = rnd(S * R, C, dtype=DT[dtype]), rnd(S * R, C, seed=1, dtype=DT[dtype])

    def run(shift):
        at = lambda n: torch.full((n + shift,), 9.0, device=DEV)[shift:]  # noqa: E731
        gamma, beta = at(C).copy_(1 + 0.2 * rnd(C, seed=2)), at(C).copy_(0.2 * rnd(C, seed=3))
        stats, dg, db = at(2 * S * K), at(C), at(C)
        assert all(t.data_ptr() % 16 == 4 * shift for t in (gamma, beta, stats, dg, db))
        y, dx = torch.empty_like(x), torch.empty_like(x)
        atlas.group_norm(x, gamma, beta, y, R, K, activation="silu", stats=stats)
        atlas.group_norm_bwd(dy, x, gamma, beta, stats, dx, dg, db, R, K, activation="silu")
        return y, stats, dx, dg, db

    for a, b in zip(run(0), run(1)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", [(400, 20000, 32, 8, 1), (400, 20000, 32, 8, 9000), (200, 1500, 1024, 64, 1),
                                  (2, 60000, 64, 4, 1), (30, 5000, 60, 12, 700)], ids=str)
def test_variance_after_unlike_first_rows(case, dtype):
    """The first rows of every sample are zeros (padding), the others lie around 1000
    with deviation 1. A thread sums at most 1,024 rows, of squares below four times
    what stays when it re-centres (2^-24 of each, 4 + 16 + .. rows): 8 * 1024 * 2^-24
    of the variance; half of it in rstd. The mean: 2^-23 of its magnitude a step."""
    S, R, C, K, zeros = case
    x = (1000 + rnd(S * R, C)).to(DT[dtype])
    x.view(S, R, C)[:, :zeros] = 0
    y, stats = torch.empty_like(x), torch.empty(S, K, 2, device=DEV)
    atlas.group_norm(x, None, None, y, R, K, stats=stats)
    for s in range(0, S, 50):
        part = x.view(S, R, K, C // K)[s:s + 50].double()
        mean = part.mean((1, 3))
        rstd = ((part - mean[:, None, :, None]).square().mean((1, 3)) + 1e-5).rsqrt()
        got = stats[s:s + 50].double()
        assert float((got[..., 1] / rstd - 1).abs().max()) <= 4 * 1024 * 2.0 ** -24
        assert float((got[..., 0] / mean - 1).abs().max()) <= 2.0 ** -21


def test_samples_longer_than_a_chunk():
    """Many samples, each in chunks of 1,024 rows and a rest: statistics and all
    gradients. fp32 sums of at most 1,024 terms a thread and a few hundred parts:
    2^-24 * 1,536 of the terms' magnitudes, as test_variance_after_unlike_first_rows."""
    S, R, C, K = 40, 1100, 8192, 64
    x, dy = rnd(S * R, C) + 3, rnd(S * R, C, seed=1)
    gamma = 1 + 0.2 * rnd(C, seed=2)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(S, K, 2, device=DEV)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    atlas.group_norm(x, gamma, None, y, R, K, stats=stats)
    atlas.group_norm_bwd(dy, x, gamma, None, stats, dx, dg, db, R, K)
    tol = 1536 * 2.0 ** -24
    want_g, size_g, want_b, size_b = torch.zeros(4, C, dtype=torch.float64, device=DEV)
    for s in range(S):
        rows = slice(s * R, (s + 1) * R)
        a, g = x[rows].double().view(R, K, -1), dy[rows].double()
        mean, var = a.mean((0, 2), keepdim=True), a.var((0, 2), unbiased=False, keepdim=True)
        rstd = (var + 1e-5).rsqrt()
        assert float((stats[s, :, 1].double() / rstd.flatten() - 1).abs().max()) <= tol / 2
        hat = ((a - mean) * rstd).view(R, C)
        # y: xhat's own roundings and the statistics' errors (of means of order 3)
        assert float((y[rows].double() - hat * gamma.double()).abs().max()) <= 10 * tol
        want_g += (g * hat).sum(0)
        size_g += (g * hat).abs().sum(0)
        want_b += g.sum(0)
        size_b += g.abs().sum(0)
        dh = (g * gamma.double()).view(R, K, -1)
        h = hat.view(R, K, -1)
        want = rstd * (dh - dh.mean((0, 2), keepdim=True) - h * (dh * h).mean((0, 2), keepdim=True))
        assert float((dx[rows].double() - want.view(R, C)).abs().max()) <= 20 * tol
    # (dgamma also carries xhat's error, 4 tol of dy at most)
    assert bool(((dg.double() - want_g).abs() <= tol * size_g + 4 * tol * size_b).all())
    assert bool(((db.double() - want_b).abs() <= tol * size_b).all())


@pytest.mark.parametrize("case", [(2, 1, 64, 8), (3, 16, 60, 12), (2, 9000, 64, 16)], ids=str)
def test_fp32_silu_far_from_zero(case):
    """x = +-1 (mean 0, variance 1, eps 0: xhat = x exactly), gamma and beta whole, so
    z is exact down to -80. y = z / (1 + exp(-z)), in units of 2^-24: the power of two
    4 (2 ulp), its correction and their product 2, the sum 1, the reciprocal 2, y's
    product 1: 10. The slope s (1 + z (1 - s)) takes 6 more roundings: 2^-20."""
    S, R, C, K = case
    x = torch.ones(S * R, C, device=DEV)
    x.view(S * R, C)[:, ::2] = -1
    if C // K % 2:
        x.view(S, R, C)[:, 1::2] *= -1
    gamma = torch.ones(C, device=DEV)
    beta = -(torch.arange(C, device=DEV) % 80).float()
    y, stats = torch.empty_like(x), torch.empty(S, K, 2, device=DEV)
    atlas.group_norm(x, gamma, beta, y, R, K, eps=0.0, activation="silu", stats=stats)
    assert torch.equal(stats, torch.tensor([0.0, 1.0], device=DEV).expand(S, K, 2))
    z = (x * gamma + beta).double()
    want = z / (1 + torch.exp(-z))
    assert float(((y.double() - want).abs() / want.abs().clamp_min(1e-40)).max()) <= 10 * 2.0 ** -24
    # dbeta of one row with dy = 1 at a time: the slope itself
    dy = torch.zeros_like(x)
    dy[S * R // 2] = 1
    dx, db = torch.empty_like(x), torch.empty(C, device=DEV)
    atlas.group_norm_bwd(dy, x, gamma, beta, stats, dx, None, db, R, K, activation="silu")
    zr = z[S * R // 2]
    s = 1 / (1 + torch.exp(-zr))
    slope = s * (1 + zr * (1 - s))
    terms = s * (1 + zr.abs() * (1 - s))
    assert bool(((db.double() - slope).abs() <= 2.0 ** -20 * terms).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", [(40, 1, 128, 2), (4, 50, 64, 4), (1, 20011, 128, 32), (300, 3000, 32, 8),
                                  (20, 4, 32800, 1)], ids=str)
def test_deviations_whose_squares_overflow(case, dtype):
    """Deviations of 1e25: their squares pass the range of the fp32 statistics. The
    variance is infinite and rstd 0 in every form, so y is beta: never a small
    variance and large values."""
    S, R, C, K = case
    x = (rnd(S * R, C).sign() * 1e25).to(DT[dtype])
    if R == 4:   # the same mean in every channel, far from the first row
        x.view(S, R, C)[:] = torch.tensor([1.0, -1, -1, -1], device=DEV)[:, None] * 1e25
    beta = rnd(C, seed=1)
    y, stats = torch.empty_like(x), torch.empty(S, K, 2, device=DEV)
    atlas.group_norm(x, None, beta, y, R, K, stats=stats)
    assert not stats[..., 1].any()
    assert torch.equal(y, beta.to(DT[dtype]).expand(S * R, C))
