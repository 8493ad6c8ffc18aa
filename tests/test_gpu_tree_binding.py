"""The two ways a call on trees or pages can be marshalled give the same bytes: the usual call goes through
C++, one that names a stream through the Python checks."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from kda_gated_delta_chunk_gb300 import layer
from test_gpu_pages import cache_of, on_gpu, pool_of, status_words, table_of
from test_gpu_tree_attention import cu_of, i32, trees_of
from test_gpu_tree_recurrent import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def same(a, b):
    for x, y in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and y.is_contiguous()
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


LENS, KV = [8, 1, 20], [50, 9, 300]


def test_plan_attention_and_accept():
    trees = trees_of(LENS, 1)
    parents, cu, kv, ws = i32([p for t in trees for p in t]), cu_of(LENS), i32(KV), status_words()
    here = torch.cuda.current_stream()
    usual = layer.native().tree_plan(parents, cu, kv, 20, ws)
    assert type(usual) is tuple
    same(usual, kda.tree_plan(parents, cu, kv, 20, workspace=ws))
    same(usual, kda.tree_plan(parents, cu, kv, 20, workspace=ws, stream=here))
    table, pages = table_of(KV, 16, 2)
    table = table.clamp(max=pages - 1).cuda()
    cache = cache_of(pages, 2, 16, 3)
    q = torch.randn(sum(LENS), 4, 128, device="cuda").to(torch.bfloat16)
    wsa = kda.alloc_attention_workspace(3, 4, 2, 20)
    for lse in (False, True):
        args = (q, *cache, table, kv, cu)
        usual = layer.native().tree_attention(*args, 0.1, 20, 5.0, 64, lse, wsa, usual[0] if lse is None else kda.tree_plan(
            parents, cu, kv, 20, workspace=ws)[0])
        assert type(usual) is tuple
        mask = kda.tree_plan(parents, cu, kv, 20, workspace=ws)[0]
        for s in (None, here):
            same(usual, kda.tree_attention(*args, mask, 0.1, 20, 5.0, 64, lse=lse, workspace=wsa, stream=s))
    ends, got = i32([7, 0, 11]), []
    for s in (None, here):
        c = [x.clone() for x in cache]
        got.append((kda.cache_accept(*c, table, kv, cu, parents, ends, 20, workspace=ws, stream=s), *c))
    same(*got)
    assert isinstance(layer.native().cache_accept(*cache, table, kv, cu, parents, ends, 20, ws), torch.Tensor)
    with pytest.raises(kda.KDAError, match="invalid argument"):
        kda.tree_plan(parents, cu, kv, 65, workspace=ws)
    with pytest.raises(kda.KDAError, match="invalid argument"):
        kda.tree_attention(*args, mask, 0.1, 20, window=19, workspace=wsa)


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_recurrence(state):
    d, trees = make(LENS, 3, state, strided=True), trees_of(LENS, 4)
    parents, cu, ws, ends = i32([p for t in trees for p in t]), cu_of(LENS), status_words(), i32([3, -1, 19])
    args = [d[x] for x in ("q", "k", "v", "g", "beta", "A_log", "dt_bias")] + [-5.0, 0.1, d["state"], cu, parents, 20]
    usual = layer.native().tree_recurrent_fwd(*args, ws)
    assert type(usual) is tuple
    fin = layer.native().tree_commit(d["k"], d["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], cu, parents, usual[1],
                                     ends, 20, None, ws)
    assert isinstance(fin, torch.Tensor)
    for s in (None, torch.cuda.current_stream()):
        got = kda.tree_recurrent_fwd(*args, workspace=ws, stream=s)
        same(usual, got)
        end = (d["k"], d["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], cu, parents, got[1], ends, 20)
        same(fin, kda.tree_commit(*end, workspace=ws, stream=s))
        into = torch.empty_like(d["state"])
        assert kda.tree_commit(*end, final_state=into, workspace=ws, stream=s) is into
        same(fin, into)
    with pytest.raises(kda.KDAError, match="lower_bound"):
        kda.tree_commit(*end[:4], -6.0, *end[5:], workspace=ws)


def test_pages():
    state, ws = pool_of([100, 37, 0, 0], 16, 12, 60, 5), status_words()
    got = []
    for s in (None, torch.cuda.current_stream()):
        pool = [x.contiguous() for x in on_gpu(*state)]
        cache = cache_of(60, 2, 16, 6)
        fro, to = kda.fork_pages(*pool, i32([0, 1]), i32([2, 3]), 16, workspace=ws, stream=s)
        kda.copy_pages(*cache, fro, to, workspace=ws, stream=s)
        kda.reserve_pages(*pool, i32([9, 9, 9, 30]), 16, workspace=ws, stream=s)
        kda.free_pages(*pool, 16, rows=i32([0]), workspace=ws, stream=s)
        kda.free_pages(*pool, 16, workspace=ws, stream=s)
        got.append((fro, to, *pool, *cache))
    same(*got)
    n = layer.native()
    assert n.free_pages(*pool, 16, None, ws) is True and n.free_pages(*pool, 16, i32([1]), ws) is True
    assert n.reserve_pages(*pool, i32([0] * 4), 16, ws) is True
    assert type(n.fork_pages(*pool, i32([0]), i32([2]), 16, ws)) is tuple
    assert n.copy_pages(*cache, i32([-1]), i32([-1]), ws) is True
    assert kda.last_device_status(ws) == kda.OK
    with pytest.raises(kda.KDAError, match="invalid argument"):
        kda.free_pages(*pool, 0, workspace=ws)
