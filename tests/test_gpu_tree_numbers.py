"""tree_recurrent_fwd with a node that is no number late in a tree: the nodes before it, whose outputs are made while
the later ones' u are under way, keep every bit."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from test_gpu_tree_attention import trees_of
from test_gpu_tree_recurrent import D, forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


@pytest.mark.parametrize("lens,most", [([64] * 4, 64), ([31, 32] * 20, 32), ([16] * 30, 16)])
@pytest.mark.parametrize("node", [-1, 9])
def test_the_nodes_before_one_that_is_no_number(lens, most, node):
    """Every second sequence has a bad value row (in one channel) at one of its nodes."""
    H = 8
    d = make(lens, H, seed=21)
    trees = trees_of(lens, 22, "chain")
    parents = [p for t in trees for p in t]
    out, u, status = forward(d, lens, parents, most)
    assert status == kda.OK
    bad = dict(d, v=d["v"].clone())
    want = torch.zeros(sum(lens), H, D, dtype=torch.bool)
    at = 0
    for n, t in enumerate(lens):
        if n % 2 == 0:
            i = node % t
            bad["v"][at + i, n % H, 5 + n % 100] = float("nan")
            want[at + i:at + t, n % H, 5 + n % 100] = True       # (a chain: all that follow)
        at += t
    want = want.cuda()
    for _ in range(20):
        o, x, status = forward(bad, lens, parents, most)
        assert status == kda.OK
        assert torch.equal(o.isnan(), want) and torch.equal(x.isnan(), want)
        assert torch.equal(o[~want], out[~want]) and torch.equal(x[~want], u[~want])
