"""The hybrid-layer example: decoding token by token gives the rows that one prefill gives.

Both runs round the same quantities to bf16 (projections, layer outputs) and to e4m3 (keys and
values, at the same scales but for pages still being filled), with sums in another order: a few
bf16 roundings, 2^-8 each, and e4m3 neighbours of keys and values averaged over the context.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_matches_one_prefill():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    got, want = ex.run([65, 1, 130], 5, hidden=512)
    assert bool(torch.isfinite(got).all())
    assert float((got - want).norm() / want.norm()) < 0.02
