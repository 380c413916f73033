"""Differential attention where values are not finite or units are many: what a row
that sees such a value gets, and that no other row's bits change."""
import pytest
import torch

from test_gpu_diff_attn import DEV, make, rnd, run
from video_dit_windowed_b200 import atlas  # noqa: F401

pytestmark = pytest.mark.gpu


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("steep", [0, 1], ids=["steep first map", "steep second map"])
def test_non_finite_value_reaches_every_channel_of_its_rows(hd, steep):
    """bf16, windows below 128 rows: a row that sees a key whose v holds one value
    that is not finite is NaN in all channels of o and s, whichever map's warps are
    ahead. One map's logits grow along the keys, so that it keeps moving its
    reference and falls behind the other's; several launches, since a warp's lead
    is a matter of timing."""
    B, L, W, H, share = 1, 20, 32, 4, 100
    N, G = L * W, W * share
    shares = [w * share for w in range(W + 1)]
    lam = torch.tensor([0.6, 0.2, -0.3, 0.9], device=DEV)
    half = hd // 2
    for seed in range(3):
        t = make(B, N, G, H, hd, "bf16", seed=seed)
        t["q_d"][..., steep * half:(steep + 1) * half] = 4.0
        ramp = torch.linspace(0.0, 40.0, share, device=DEV).repeat(W)[:, None, None] / half
        t["k_g"][..., steep * half:(steep + 1) * half] = ramp.to(torch.bfloat16)
        hit = torch.zeros(W, dtype=torch.bool, device=DEV)
        for w, ch, value in ((3, 3, "nan"), (9, hd - 1, "inf"), (17, half, "-inf"), (31, 0, "nan")):
            t["v_g"][w * share + 37 + w, :, ch] = float(value)
            hit[w] = True
        for w, ch in ((5, hd - 2), (20, 1)):
            t["v_d"][w * L + 7, :, ch] = float("inf")
            hit[w] = True
        rows = hit.repeat_interleave(L)
        first = None
        for _ in range(8):
            out = run(t, lam, B, N, G, H, window_len=L, global_window_offsets=int32(shares))
            for n in ("o_d", "s_d"):
                assert bool(torch.isnan(out[n][rows]).all()), n
                assert bool(torch.isfinite(out[n][~rows]).all()), n
            first = first or out
            for n in ("o_d", "s_d"):
                assert torch.equal(first[n][~rows], out[n][~rows]), n


def rest_of(N, w, L):
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[w * L:(w + 1) * L] = False
    return keep


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("L", [20, 160])
def test_rows_whose_logits_are_all_minus_infinity(L, hd, dtype):
    """0 / 0 in the softmax's definition: NaN in o (and in s for the second map),
    in the gradients that the row reaches, and lse -inf, in both types."""
    B, N, G, H = 1, 320, 0, 1
    lam = torch.tensor([0.6], device=DEV)
    for ch, both in ((3, False), (hd // 2 + 3, True)):
        t = make(B, N, G, H, hd, dtype)
        mine = slice(L, 2 * L)
        t["k_d"][mine, 0, ch] = float("-inf")
        t["q_d"][mine, 0, ch] = 1.0
        t["q_d"][L + 7, 0, ch] = 2.0
        out = run(t, lam, B, N, G, H, window_len=L)
        m = 1 if both else 0
        assert bool((out["lse"][0, 0, m, mine] == float("-inf")).all())
        assert bool(torch.isfinite(out["lse"][0, 0, 1 - m]).all())
        assert bool(torch.isnan(out["o_d"][mine]).all())
        assert bool(torch.isnan(out["s_d"][mine]).all()) == both
        assert bool(torch.isnan(out["dq_d"][mine]).all())
        keep = rest_of(N, 1, L)
        for n in ("o_d", "s_d", "dq_d", "dk_d", "dv_d"):
            assert bool(torch.isfinite(out[n][keep]).all()), n


SHORT = {
    # what changes in the rows of one window: tensor, row in it, channel, value
    "nan key": lambda t, a, b: t["k_d"][a + 3, 0].__setitem__(3, float("nan")),
    "inf query": lambda t, a, b: t["q_d"][a + 5, 0].__setitem__(40, float("inf")),
    "large keys": lambda t, a, b: t["k_d"][a:b].mul_(12.0),
    "large queries": lambda t, a, b: t["q_d"][a:b].mul_(16.0),
    "nan queries": lambda t, a, b: t["q_d"][a:b].fill_(float("nan")),
    # logits of -inf for all of the window's own keys, in the first map
    "own keys at -inf": lambda t, a, b: (t["q_d"][a:b, 0, 3].fill_(1.0),
                                         t["k_d"][a:b, 0, 3].fill_(float("-inf"))),
}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("grow", [1.0, 9.0], ids=["level", "growing"])
@pytest.mark.parametrize("change", SHORT, ids=str)
def test_rows_keep_their_bits_beside_a_changed_window(hd, change, grow):
    """bf16, windows that share a 128-row tile and see 300 global keys, whose whole
    tiles take no mask: whatever one window's rows hold, the others' bits stay."""
    B, N, L, G, H, w = 1, 200, 20, 300, 1, 4
    lam = torch.tensor([0.6], device=DEV)
    t = make(B, N, G, H, hd, "bf16")
    # level global keys: no other row moves its reference; growing ones: each does now and then
    t["k_g"] = (t["k_g"].float() * torch.linspace(0.5, grow, G, device=DEV)[:, None, None]).to(torch.bfloat16)
    clean = run(t, lam, B, N, G, H, window_len=L)
    bad = {n: x.clone() for n, x in t.items()}
    SHORT[change](bad, w * L, (w + 1) * L)
    out = run(bad, lam, B, N, G, H, window_len=L)
    keep = rest_of(N, w, L)
    for n in ("o", "s", "dq", "dk", "dv"):
        assert torch.equal(out[n + "_d"][keep], clean[n + "_d"][keep]), n
    for n in ("o", "s", "dq"):
        assert torch.equal(out[n + "_g"], clean[n + "_g"]), n
    every = torch.cat([keep, torch.ones(G, dtype=torch.bool, device=DEV)])
    assert torch.equal(out["lse"][..., every], clean["lse"][..., every])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("L", [20, 160])
def test_key_at_minus_infinity_reaches_dq(L, hd, dtype):
    """A key with -inf in a channel where its queries are positive has weight 0, so
    o is finite, but dq = sum dS k holds 0 * -inf: NaN, as the formula gives it.
    Queries of other windows keep finite gradients."""
    B, N, G, H = 1, 320, 30, 2
    lam = torch.tensor([0.6, 0.3], device=DEV)
    t = make(B, N, G, H, hd, dtype)
    t["q_d"][L:2 * L, :, 3] = 1.0
    t["k_d"][L + 7, :, 3] = float("-inf")
    out = run(t, lam, B, N, G, H, window_len=L)
    for n in ("o", "s", "dv"):
        for p in "dg":
            assert bool(torch.isfinite(out[f"{n}_{p}"]).all()), (n, p)
    assert bool(torch.isnan(out["dq_d"][L:2 * L, :, 3]).all())
    keep = rest_of(N, 1, L)
    assert bool(torch.isfinite(out["dq_d"][keep]).all()) and bool(torch.isfinite(out["dq_g"]).all())
    assert bool(torch.isfinite(out["dk_d"]).all()) and bool(torch.isfinite(out["dlam"]).all())
