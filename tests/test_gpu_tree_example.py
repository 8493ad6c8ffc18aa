"""The operators on trees and pages run together as a speculative decode loop does: the rows of the kept
branches against one prefill of the kept tokens.

Both runs round to bf16 at the same places (norms, projections, outputs) and keep keys and values in e4m3 with
power-of-two scales; they differ in how tokens fall into pages' scales (a rejected draft may raise a page's
scale) and in the order of sums.  A cache entry is within 2^-4 of itself in either; its error enters a row through the
attention layer's output alone, averaged over the keys, so that rows agree to a few 2^-8 of their norm: 0.02.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()
    sys.path.insert(0, ROOT)


@pytest.mark.parametrize("prompts,samples,steps,nodes,page", [
    ([100, 37, 256], 2, 4, 12, 16), ([5], 1, 6, 64, 16), ([64, 33], 3, 3, 8, 64), ([300] * 8, 2, 3, 40, 32)])
def test_tree_verify(prompts, samples, steps, nodes, page):
    from examples import tree_verify
    got, want = tree_verify.run(prompts, samples, steps, nodes, hidden=512, page=page)
    assert got.shape == want.shape and got.shape[0] > 0
    off = float((got - want).norm() / want.norm())
    print(f"relative difference {off:.2e}")
    assert off < 0.02
