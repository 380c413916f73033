"""The differential-attention layer's host side: sizes that the library plans and
calls that the binding refuses (no GPU needed)."""
import pytest
import torch

from video_dit_windowed_b200 import atlas, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return atlas.lib()


@pytest.mark.parametrize("samples,rows,channels,row_threads", [(300, 200000, 1024, 1), (592, 50000, 2048, 1),
                                                               (400, 300000, 32, 32), (1, 400000000, 4, 256)])
def test_norm_chunks_stay_short(lib, samples, rows, channels, row_threads):
    """fp32 sums of up to 1,024 rows a thread, however many samples fill the GPU by
    themselves: the workspace holds 8 bytes a (sample, chunk, channel)."""
    groups = 4
    for backward in (0, 1):
        size = lib.atlas_group_norm_workspace(samples, rows, channels, groups, atlas.FP32, backward)
        chunks = (size - samples * groups * 8) // (samples * channels * 8)
        assert chunks * row_threads * 1024 >= rows


def test_a_side_without_queries_has_nothing_else(lib):
    """q None stands for no rows: outputs or keys given for that side would never be
    written or read, so they are refused."""
    x, lam = torch.zeros(4, 2, 64), torch.ones(2)
    none = torch.zeros(0, 2, 64)
    for detail in ((None, x, x, x), (None, None, None, x), (none, x, x, x), (None, None, x, None)):
        with pytest.raises(ValueError, match="without queries"):
            atlas.diff_attn(*detail[:3], x, x, x, lam, detail[3], x)
        with pytest.raises(ValueError, match="without queries"):
            atlas.diff_attn(x, x, x, *detail[:3], lam, x, detail[3])
    with pytest.raises(ValueError, match="without queries"):
        atlas.diff_attn_bwd(None, None, None, None, None, None, x, x, x, x, x, x, lam, lam, x, None, None,
                            x, x, x, lam)
