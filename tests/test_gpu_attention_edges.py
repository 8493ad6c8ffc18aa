"""cached_attention at the edges of what a row sees: windows, pages behind them, extreme sizes,
streams.  References and tolerances as in test_gpu_attention."""
import math

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import layer_ref as ref
from test_gpu_attention import BF16, D, FP8, NAN8, SCALE, check, launch, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def test_nan_at_both_ends_of_a_window_over_three_tiles():
    """Values that only some of a sequence's queries see are NaN, at the window's edge and at the
    causal end, in the channels of one warp; sequences enough that a CTA takes an item's
    three tiles in turn.  Each NaN reaches the rows that see it and no others, whatever the
    order in which the warps run."""
    N, H, hk, page, window, t = 56, 8, 8, 16, 200, 4
    kv = [250 + 5 * n for n in range(N)]
    d = make([t] * N, kv, H, hk, page, seed=31)
    clean, clean_lse, status = launch(d, window=window)
    assert status == kda.OK
    bad = dict(d, v=d["v"].clone())
    want = torch.zeros(N * t, H, D, dtype=torch.bool)
    for n in range(N):
        p = kv[n] - t + torch.arange(t)
        some = [j for j in range(kv[n]) if 0 < int(((j <= p) & (j > p - window)).sum()) < t]
        for i, j in enumerate(some):
            h = (n + i) % hk
            bad["v"][int(d["table"][n, j // page]), h, j % page, 32:64] = NAN8
            sees = (j <= p) & (j > p - window)
            want[n * t:(n + 1) * t, h, 32:64] |= sees[:, None]
    assert bool(want.any())
    for _ in range(20):
        out, lse, status = launch(bad, window=window)
        assert status == kda.OK
        assert torch.equal(out.isnan().cpu(), want)
        assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse, clean_lse)
