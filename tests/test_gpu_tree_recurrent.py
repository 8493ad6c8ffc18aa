"""tree_recurrent_fwd and tree_commit on the GPU against the recurrence node by node in 64 bits.

Tolerances.  Let m be a result's magnitude: the same sums over absolute values, along the node's branch
(tree_ref.recurrence).  Every sum of 128 products in fp32 is off by at most 2^-17 m (the state's products by
2^-21 m more: two f16 terms a factor), norms and gates by 2^-20 of what they multiply, and a branch of
d nodes multiplies d decays and adds d terms, 2^-20 m each.  u, out and the state each meet three
such sums (u's own, those of the u before it, which m counts already, and their own): 2^-15 m + d 2^-19 m.
Results in bf16 are rounded once more: 2^-8 of themselves.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import kda_workloads as W
import tree_ref as ref
from test_gpu_tree_attention import cu_of, i32, trees_of

pytestmark = pytest.mark.gpu

BF16, D = torch.bfloat16, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def status_words():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def make(lens, H, state="f32", seed=0, std=0.1, pad=0, strided=False):
    g = torch.Generator().manual_seed(seed + 7 * len(lens) + H)
    T, N = sum(lens) + pad, len(lens)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = rnd(T, 4 * H * D + 8 * -(-H // 8)).to(BF16).cuda()
    d = {x: p[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i, x in enumerate("qkvg")}
    d["beta"] = p[:, 4 * H * D:][:, :H]
    if not strided:
        d = {x: y.contiguous() for x, y in d.items()}
    d["A_log"] = torch.log(1 + 15 * torch.rand(H, generator=g)).cuda()
    d["dt_bias"] = (0.1 * rnd(H, D)).cuda()
    s = std * rnd(N, H, D, D)
    d["state"] = s.to(BF16 if state == "bf16" else torch.float32).cuda()
    return d


def forward(d, lens, parents, most=64, state="own", **kw):
    ws = status_words()
    s0 = d["state"] if isinstance(state, str) else state
    out, u = kda.tree_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["dt_bias"], -5.0,
                                    W.SCALE, s0, cu_of(lens), i32(parents), most, workspace=ws, **kw)
    return out, u, kda.last_device_status(ws)


def commit(d, lens, parents, u, nodes, most=64, state="own", **kw):
    ws = status_words()
    s0 = d["state"] if isinstance(state, str) else state
    fin = kda.tree_commit(d["k"], d["g"], d["A_log"], d["dt_bias"], -5.0, s0, cu_of(lens), i32(parents), u,
                          i32(nodes), most, workspace=ws, **kw)
    return fin, kda.last_device_status(ws)


def f64(t):
    return t.float().double().cpu()


def within(got, want, big, depth, bf16):
    tol = big * (2.0 ** -15 + depth * 2.0 ** -19) + (2.0 ** -8 * want.abs() if bf16 else 0.0)
    worst = float(((f64(got) - want).abs() / tol.clamp(min=1e-30)).max())
    assert worst <= 1.0, worst


def check(d, lens, trees, nodes, out, u, fin, zero=False):
    """Outputs, u and the accepted states of every sequence."""
    at = 0
    for n, (t, tree) in enumerate(zip(lens, trees)):
        s0 = f64(d["state"][n]) * (0.0 if zero else 1.0)
        end = nodes[n] if t else -1
        if t:
            a = [f64(d[x][at:at + t]) for x in "qkvg"] + [f64(d["beta"][at:at + t])]
            o, uu, after, bo, bu, ba = ref.recurrence(*a, f64(d["A_log"]), f64(d["dt_bias"]), -5.0, W.SCALE, s0, tree)
            deep = max(len(ref.branch(tree, i)) for i in range(t))
            within(out[at:at + t], o, bo, deep, True)
            within(u[at:at + t], uu, bu, deep, False)
        if end < 0:
            assert torch.equal(f64(fin[n]), s0)
        else:
            within(fin[n], after[end], ba[end], deep, fin.dtype is BF16)
        at += t


CASES = [
    # nodes, heads
    ([1], 1),
    ([8], 16),
    ([9, 16, 1], 3),
    ([0, 5, 0, 32, 17, 1], 4),
    ([33, 64, 2], 2),
    ([64] * 3, 5),
    ([3] * 70, 2),
]


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["any", "chain", "roots"])
@pytest.mark.parametrize("lens,H", CASES)
def test_trees(lens, H, kind, state):
    d = make(lens, H, state, seed=1, strided=kind == "any")
    trees = trees_of(lens, 31, kind)
    parents = [p for t in trees for p in t]
    g = torch.Generator().manual_seed(5)
    nodes = [int(torch.randint(-1, n, (1,), generator=g)) if n else -1 for n in lens]
    for most in {max(lens), 64}:
        out, u, status = forward(d, lens, parents, most)
        assert status == kda.OK
        for ends in (nodes, [n - 1 for n in lens]):
            fin, status = commit(d, lens, parents, u, ends, most)
            assert status == kda.OK
            check(d, lens, trees, ends, out, u, fin)


@pytest.mark.parametrize("std", [0.0, 1e-30, 30.0, 1e30])
def test_states_of_any_size(std):
    """Zeros, values below f16's range by far, and above it; rows of very unequal size."""
    lens, H = [12, 5], 2
    d = make(lens, H, seed=2, std=std)
    d["state"][:, :, 5] *= 1e-4
    d["state"][:, :, 77] = 0
    d["state"][:, :, :, 9] *= 1e-3
    trees = trees_of(lens, 32)
    parents = [p for t in trees for p in t]
    out, u, status = forward(d, lens, parents)
    assert status == kda.OK
    fin, status = commit(d, lens, parents, u, [11, 2])
    assert status == kda.OK
    check(d, lens, trees, [11, 2], out, u, fin)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_no_state(dtype):
    lens, H = [7, 20], 2
    d = make(lens, H, seed=3)
    trees = trees_of(lens, 33)
    parents = [p for t in trees for p in t]
    out, u, status = forward(d, lens, parents, state=None, state_dtype=dtype)
    assert status == kda.OK
    fin, status = commit(d, lens, parents, u, [-1, 19], state=None, state_dtype=dtype)
    assert status == kda.OK and fin.dtype is dtype
    check(d, lens, trees, [-1, 19], out, u, fin, zero=True)


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_a_chain_is_the_recurrence(state):
    """recurrent_fwd on the same tokens: both within the tolerance of the definition, so within twice it
    of each other; its per-token states are the commits of every node."""
    lens, H = [6, 1, 11], 3
    d = make(lens, H, state, seed=4)
    trees = trees_of(lens, 0, "chain")
    parents = [p for t in trees for p in t]
    out, u, _ = forward(d, lens, parents)
    _, fin, states = kda.recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["dt_bias"], -5.0,
                                       W.SCALE, d["state"], cu_of(lens), token_states=True)
    for back in range(3):
        ends = [max(-1, n - 1 - back) for n in lens]
        got, _ = commit(d, lens, parents, u, ends)
        check(d, lens, trees, ends, out, u, got)
        for n, e in enumerate(ends):
            if e >= 0:
                near = f64(states[sum(lens[:n]) + e])
                assert float((f64(got[n]) - near).abs().max()) <= (2e-3 if state == "f32" else 2e-2)


def test_commit_in_place_and_outputs_given():
    lens, H = [10, 0, 31], 2
    d = make(lens, H, seed=5, pad=4)
    trees = trees_of(lens, 35)
    parents = [p for t in trees for p in t] + [9] * 4
    out = torch.full((45, H, D), 3.0, dtype=BF16, device="cuda")
    u = torch.full((45, H, D), 3.0, device="cuda")
    got = forward(d, lens, parents, 31, out=out, u=u)
    assert got[0] is out and got[1] is u and got[2] == kda.OK
    assert bool((out[41:] == 3.0).all()) and bool((u[41:] == 3.0).all())
    want, _ = commit(d, lens, parents, u, [9, -1, -1], 31)
    check(d, lens, trees, [9, -1, -1], out, u, want)
    before = d["state"].clone()
    fin, status = commit(d, lens, parents, u, [9, -1, -1], 31, final_state=d["state"])
    assert fin is d["state"] and status == kda.OK and torch.equal(fin, want)
    assert torch.equal(fin[1:], before[1:])


def test_device_errors():
    """A malformed sequence's rows and state stay, the one beside it is done; a bad parent counts as none."""
    lens, H = [4, 6], 2
    d = make(lens, H, seed=6)
    trees = trees_of(lens, 36)
    parents = [p for t in trees for p in t]
    out = torch.full((10, H, D), 3.0, dtype=BF16, device="cuda")
    u = torch.zeros((10, H, D), device="cuda")
    got = forward(d, lens, parents, 5, out=out, u=u)
    assert got[2] == kda.ERR_INVALID_ARG and bool((out[4:] == 3.0).all())
    fin, status = commit(d, lens, parents, u, [3, 5], 5)
    assert status == kda.ERR_INVALID_ARG and torch.equal(fin[1], d["state"][1])
    check(d, lens[:1], trees[:1], [3], out[:4], u[:4], fin[:1])
    for bad in (4, -2):
        fin, status = commit(d, lens, parents, u, [bad, -1])
        assert status == kda.ERR_BAD_TREE and torch.equal(fin, d["state"])
    odd = [-1, 3, -7, 0] + parents[4:]
    out, u, status = forward(d, lens, odd)
    assert status == kda.ERR_BAD_TREE
    fixed = [[-1, -1, -1, 0], trees[1]]
    fin, status = commit(d, lens, odd, u, [3, 5])
    assert status == kda.ERR_BAD_TREE
    check(d, lens, fixed, [3, 5], out, u, fin)


def test_nan_stays_on_its_branches():
    """A node without numbers takes its descendants with it, and nothing else; a state's infinity its column."""
    lens, H = [20], 2
    d = make(lens, H, seed=7)
    trees = trees_of(lens, 37)
    clean, clean_u, _ = forward(d, lens, trees[0])
    d["k"][3, 1] = float("nan")
    out, u, status = forward(d, lens, trees[0])
    assert status == kda.OK
    want = torch.zeros(20, H, D, dtype=torch.bool)
    for i in range(20):
        if 3 in ref.branch(trees[0], i):
            want[i, 1] = True
    assert torch.equal(out.isnan().cpu(), want) and torch.equal(u.isnan().cpu(), want)
    assert torch.equal(out.cpu()[~want], clean.cpu()[~want])
    d = make(lens, H, seed=7)
    d["state"][0, 1, 50, 60] = float("inf")
    out, u, status = forward(d, lens, trees[0])
    other = torch.ones(D, dtype=torch.bool)
    other[60] = False
    assert torch.equal(out[:, 0], clean[:, 0]) and torch.equal(out[:, 1][:, other], clean[:, 1][:, other])
    assert not bool(out[:, 1, 60].isfinite().any())


def test_graph_and_stream():
    lens, H = [8, 30], 2
    d = make(lens, H, seed=8)
    trees = [trees_of(lens, s) for s in (38, 39)]
    parents, nodes, cu = i32([p for t in trees[0] for p in t]), i32([7, 20]), cu_of(lens)
    ws = status_words()

    def step(stream=None):
        out, u = kda.tree_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["dt_bias"], -5.0,
                                        W.SCALE, d["state"], cu, parents, 30, workspace=ws, stream=stream)
        return out, u, kda.tree_commit(d["k"], d["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], cu, parents, u,
                                       nodes, 30, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, u, fin = step()
    for t, ends in zip(trees, ([3, -1], [0, 29])):
        parents.copy_(i32([p for x in t for p in x]))
        nodes.copy_(i32(ends))
        graph.replay()
        check(d, lens, t, ends, out, u, fin)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    again = step(other)
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(x, y) for x, y in zip(again, (out, u, fin)))
    assert kda.last_device_status(ws) == kda.OK


def test_states_at_the_end_of_fp32():
    """Values whose column's largest is near fp32's: still within f16 once scaled."""
    lens, H = [9], 1
    d = make(lens, H, seed=9, std=1.0)
    d["state"].clamp_(-2, 2)
    d["state"][:, :, :, 7] *= 2.0 ** 120
    d["state"][:, :, 3, 8] = 2.0 ** 122
    trees = trees_of(lens, 40)
    out, u, status = forward(d, lens, trees[0])
    assert status == kda.OK and bool(torch.isfinite(out.float()).all())
    fin, status = commit(d, lens, trees[0], u, [8])
    assert status == kda.OK
    check(d, lens, trees, [8], out, u, fin)


def test_calls_without_tokens_or_sequences():
    d = make([1], 2, seed=10)
    none = {x: d[x][:0] for x in ("q", "k", "v", "g", "beta")}
    empty = i32([])
    out, u = kda.tree_recurrent_fwd(*none.values(), d["A_log"], d["dt_bias"], -5.0, W.SCALE, d["state"], i32([0, 0]),
                                    empty, 4)
    assert out.shape == (0, 2, D) and u.shape == (0, 2, D)
    fin = kda.tree_commit(none["k"], none["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], i32([0, 0]), empty, u,
                          i32([-1]), 4)
    assert torch.equal(fin, d["state"])
    out, u = kda.tree_recurrent_fwd(*none.values(), d["A_log"], d["dt_bias"], -5.0, W.SCALE, d["state"][:0], i32([0]),
                                    empty, 4)
    assert out.shape == (0, 2, D)
    mask, pos = kda.tree_plan(empty, i32([0, 0]), i32([5]), 4)
    assert mask.shape == pos.shape == (0,)


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("most", [8, 16, 32])
def test_more_sequences_than_run_at_once(most, state):
    """Several (sequence, head) pairs a multiprocessor, one after the other; a sequence's results do not depend on
    the batch that it is in."""
    H = 8
    lens = [(5 * n + 3) % (most + 1) for n in range(41)] + [most]
    d = make(lens, H, state, seed=11, strided=True)
    trees = trees_of(lens, 41)
    parents = [p for t in trees for p in t]
    ends = [n - 1 for n in lens]
    out, u, status = forward(d, lens, parents, most)
    assert status == kda.OK
    fin, status = commit(d, lens, parents, u, ends, most)
    assert status == kda.OK
    check(d, lens, trees, ends, out, u, fin)
    some = {x: d[x] for x in ("A_log", "dt_bias")}
    n, T = 7, sum(lens[:7])
    some.update({x: d[x][:T] for x in ("q", "k", "v", "g", "beta")}, state=d["state"][:n])
    few = forward(some, lens[:n], parents[:T], most)
    assert few[2] == kda.OK and torch.equal(few[0], out[:T]) and torch.equal(few[1], u[:T])
