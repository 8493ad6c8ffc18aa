"""tree_recurrent_fwd with a node that is no number late in a tree (the nodes before it, whose outputs are made while
the later ones' u are under way, keep every bit), and with channels far below the largest."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import kda_workloads as W
import tree_ref as ref
from test_gpu_tree_attention import trees_of
from test_gpu_tree_recurrent import D, f64, forward, make, within

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


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_channels_far_below_the_largest(state):
    """A chain whose channels lose e^-5 a node but for one, which the keys and the state do not use and the queries
    do: what is left of an output comes from entries of c qh far below its largest.  The product with the state takes
    two f16 terms a factor, the largest brought to 2^13 or more: an entry is off by 2^-22 of itself (the recurrence's
    other tests count that) or f16's half step of 2^-25, 2^-38 of the largest.  That adds, a channel, at most
    2^-38 (max|S| |c qh| + |S| max|c qh|), so 2^-30 max|S| max|c qh| over 128 channels.  The vectors of the keys
    shrink as a whole and lose nothing."""
    lens, H = [8], 2
    d = make(lens, H, state, seed=23)
    d["k"][:, :, 0] = 0
    d["v"][:] = 0
    d["state"][:, :, 0] = 0
    d["A_log"][:] = 0
    d["dt_bias"][:] = 40
    d["dt_bias"][:, 0] = -80
    tree = list(range(-1, 7))
    out, u, status = forward(d, lens, tree, 8)
    assert status == kda.OK
    a = [f64(d[x]) for x in "qkvg"] + [f64(d["beta"])]
    o, uu, after, bo, bu, ba = ref.recurrence(*a, f64(d["A_log"]), f64(d["dt_bias"]), -5.0, W.SCALE, f64(d["state"][0]), tree)
    within(u, uu, bu, 8, False)
    q = f64(d["q"])
    most = (q / (q * q).sum(-1, keepdim=True).sqrt() * W.SCALE).abs().amax(-1, keepdim=True)
    step = 2.0 ** -30 * f64(d["state"][0]).abs().amax((-2, -1))[None, :, None] * most
    tol = bo * (2.0 ** -15 + 8 * 2.0 ** -19) + 2.0 ** -8 * o.abs() + step
    assert float(((f64(out) - o).abs() / tol).max()) <= 1.0
