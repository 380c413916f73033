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
