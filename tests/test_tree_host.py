"""The C entry points and the binding of the operators on drafted trees on a host without a GPU:
refusals come before any device is touched."""
import ctypes

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from test_layer_host import A, L, cache  # noqa: F401  (L: the library, a fixture)

INVALID, MISALIGNED = kda.ERR_INVALID_ARG, kda.ERR_MISALIGNED


def plan(L, **over):
    a = dict(parents=A, cu=A, kv=A, mask=A, pos=A, ws=A, stream=None, T=4, N=1, most=4, wsb=256)
    a.update(over)
    return L.kda_tree_plan(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(T=2 ** 31), INVALID), (dict(N=-1), INVALID), (dict(most=65), INVALID), (dict(most=0), INVALID),
    (dict(most=-1), INVALID), (dict(parents=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
    (dict(mask=None), INVALID), (dict(pos=None), INVALID), (dict(ws=None), INVALID), (dict(parents=A + 2), MISALIGNED),
    (dict(mask=A + 4), MISALIGNED), (dict(pos=A + 1), MISALIGNED), (dict(kv=A + 2), MISALIGNED),
    (dict(ws=A + 8), MISALIGNED), (dict(wsb=255), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_plan_refuses(L, over, code):
    assert plan(L, **over) == code


def attend(L, c=None, **over):
    a = dict(q=A, qs=512, c=ctypes.byref(c if c is not None else cache()), cu=A, mask=A, scale=0.1, cap=0.0,
             window=0, out=A, os=512, lse=A, ws=A, stream=None, T=4, N=1, H=4, most=4, wsb=1 << 30)
    a.update(over)
    return L.kda_tree_attention(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(most=65), INVALID), (dict(mask=None), INVALID), (dict(window=3), INVALID), (dict(window=-1), INVALID),
    (dict(mask=A + 4), MISALIGNED), (dict(H=3), INVALID), (dict(scale=float("nan")), INVALID), (dict(cap=-1.0), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(most=0), INVALID), (dict(qs=500), INVALID),
    (dict(qs=516), MISALIGNED), (dict(wsb=300), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_attention_refuses(L, over, code):
    assert attend(L, **over) == code


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.tree_plan(i, i, i[:1], 2)
    q = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.tree_attention(q, q, q, q, q, i, i, i, i, 1.0, 2)


def test_new_codes_have_texts(L):
    assert "tree" in kda.status_string(kda.ERR_BAD_TREE)
    assert "pages" in kda.status_string(kda.ERR_OUT_OF_PAGES)


def accept(L, c=None, **over):
    a = dict(c=ctypes.byref(c if c is not None else cache()), cu=A, parents=A, node=A, lens=2 * A, ws=A, stream=None,
             T=4, N=1, most=4, wsb=256)
    a.update(over)
    return L.kda_cache_accept(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(most=65), INVALID), (dict(parents=None), INVALID), (dict(node=None), INVALID), (dict(lens=None), INVALID),
    (dict(lens=A), INVALID), (dict(N=2 ** 30), INVALID), (dict(node=A + 2), MISALIGNED), (dict(lens=A + 1), MISALIGNED),
    (dict(wsb=0), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_accept_refuses(L, over, code):
    assert accept(L, **over) == code


def test_accept_refuses_lengths_over_its_inputs(L):
    assert accept(L, node=3 * A, lens=3 * A) == INVALID
    assert accept(L, node=3 * A, lens=A) == INVALID


POOL = dict(refs=A, pages=10, table=A, stride=4, rows=3, blocks=4, lens=A, page=16)


def pool(L, call, **over):
    tail = dict(free=dict(list=A, num=2), reserve=dict(new=A), fork=dict(src=A, dst=A, num=2, fro=A, to=A))[call]
    a = dict(POOL, **tail, ws=A, wsb=256, stream=None)
    a.update(over)
    return getattr(L, "kda_pages_" + call)(*a.values())


@pytest.mark.parametrize("call", ["free", "reserve", "fork"])
@pytest.mark.parametrize("over,code", [
    (dict(refs=None), INVALID), (dict(pages=0), INVALID), (dict(table=None), INVALID), (dict(stride=3), INVALID),
    (dict(rows=-1), INVALID), (dict(blocks=-1), INVALID), (dict(lens=None), INVALID), (dict(page=0), INVALID),
    (dict(page=2 ** 30), INVALID), (dict(ws=None), INVALID), (dict(refs=A + 4), MISALIGNED), (dict(table=A + 2), MISALIGNED),
    (dict(lens=A + 2), MISALIGNED), (dict(ws=A + 4), MISALIGNED), (dict(wsb=16), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_pool_refuses(L, call, over, code):
    assert pool(L, call, **over) == code


@pytest.mark.parametrize("call,over", [
    ("free", dict(num=-1)), ("reserve", dict(new=None)), ("reserve", dict(rows=16385)), ("fork", dict(num=16385)),
    ("fork", dict(num=-1)), ("fork", dict(rows=16385)), ("fork", dict(src=None)), ("fork", dict(dst=None)),
    ("fork", dict(fro=None)), ("fork", dict(to=None))])
def test_pool_calls_refuse(L, call, over):
    assert pool(L, call, **over) == INVALID


def test_reserve_refuses_tables_whose_requests_may_pass_32_bits(L):
    assert pool(L, "reserve", rows=16384, blocks=2 ** 17, stride=2 ** 17) == INVALID
    assert pool(L, "reserve", rows=2, blocks=2 ** 30, stride=2 ** 30, page=1) == INVALID
    assert pool(L, "reserve", rows=16384, blocks=2 ** 17 - 1, stride=2 ** 17, new=A + 1) == MISALIGNED


@pytest.mark.parametrize("over,code", [
    (dict(fro=None), INVALID), (dict(to=None), INVALID), (dict(num=-1), INVALID), (dict(num=2 ** 30), INVALID),
    (dict(ws=None), INVALID), (dict(c=None), INVALID), (dict(fro=A + 2), MISALIGNED),
    (dict(wsb=0), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_copy_refuses(L, over, code):
    a = dict(c=ctypes.byref(cache()), fro=A, to=A, num=2, ws=A, wsb=256, stream=None)
    a.update(over)
    assert L.kda_pages_copy(*a.values()) == code


def recur(L, **over):
    a = dict(q=A, qs=512, k=A, ks=512, v=A, vs=512, g=A, gs=512, beta=A, bs=4, A_log=A, dt=A, lb=-5.0, scale=0.1, s0=A,
             sd=0, cu=A, parents=A, out=A, u=A, ws=A, stream=None, T=4, N=1, H=4, most=4, wsb=256)
    a.update(over)
    return L.kda_tree_recurrent_fwd(*a.values())


def commit(L, **over):
    a = dict(k=A, ks=512, g=A, gs=512, A_log=A, dt=A, lb=-5.0, s0=A, s1=A, sd=0, cu=A, parents=A, u=A, node=A, ws=A,
             stream=None, T=4, N=1, H=4, most=4, wsb=256)
    a.update(over)
    return L.kda_tree_commit(*a.values())


@pytest.mark.parametrize("call", [recur, commit])
@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(N=2 ** 20, H=2 ** 12, ks=2 ** 19, gs=2 ** 19), INVALID),
    (dict(most=65), INVALID), (dict(most=0), INVALID), (dict(sd=2), INVALID), (dict(k=None), INVALID), (dict(g=None), INVALID),
    (dict(A_log=None), INVALID), (dict(dt=None), INVALID), (dict(u=None), INVALID), (dict(parents=None), INVALID),
    (dict(ks=500), INVALID), (dict(gs=511), INVALID), (dict(lb=-5.1), kda.ERR_UNSAFE_LOWER_BOUND),
    (dict(lb=0.1), kda.ERR_UNSAFE_LOWER_BOUND), (dict(lb=float("nan")), kda.ERR_UNSAFE_LOWER_BOUND),
    (dict(ks=516), MISALIGNED), (dict(k=A + 8), MISALIGNED), (dict(dt=A + 4), MISALIGNED), (dict(s0=A + 8), MISALIGNED),
    (dict(u=A + 4), MISALIGNED), (dict(wsb=255), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_recurrence_refuses(L, call, over, code):
    assert call(L, **over) == code


@pytest.mark.parametrize("call,over,code", [
    (recur, dict(q=None), INVALID), (recur, dict(v=None), INVALID), (recur, dict(beta=None), INVALID), (recur, dict(bs=3), INVALID),
    (recur, dict(out=None), INVALID), (recur, dict(scale=float("inf")), INVALID), (recur, dict(beta=A + 1), MISALIGNED),
    (recur, dict(out=A + 2), MISALIGNED), (commit, dict(s1=None), INVALID), (commit, dict(node=None), INVALID),
    (commit, dict(s1=A + 8), MISALIGNED), (commit, dict(node=A + 1), MISALIGNED)])
def test_recurrence_and_commit_refuse(L, call, over, code):
    assert call(L, **over) == code


@pytest.mark.parametrize("call", [recur, commit])
def test_recurrence_refuses_rows_past_32_bits(L, call):
    wide = dict(ks=2 ** 28, gs=2 ** 28, qs=2 ** 28, vs=2 ** 28, bs=2 ** 21)
    wide = {k: v for k, v in wide.items() if call is recur or k in ("ks", "gs")}
    assert call(L, H=2 ** 20 + 1, **wide) == INVALID
    assert call(L, H=2 ** 20, **dict(wide, ks=2 ** 28 + 4)) == MISALIGNED
