"""The full-attention layer's C entry points and binding on a host without a GPU: refusals come
before any device is touched, and the rotation table is the definition's."""
import ctypes
import math

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from kda_gated_delta_chunk_gb300 import build as kbuild

A = 1 << 20        # a 16-byte aligned stand-in for a device pointer: never dereferenced here


class Cache(ctypes.Structure):      # kda_kv_cache of kda.h
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("kv_lens", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def norm(L, **over):
    a = dict(x=A, ldx=64, r=A, ldr=64, rdt=1, w=A, wdt=1, eps=1e-6, ro=A, lds=64, y=A, ldy=64, y8=A,
             ldy8=64, ys=A, group=128, rows=4, cols=64)
    a.update(over)
    return L.kda_add_rms_norm(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(cols=0), dict(cols=32769, ldx=1 << 20), dict(group=64), dict(wdt=2),
    dict(rdt=5), dict(eps=float("inf")), dict(w=None), dict(y=None, y8=None, ys=None), dict(ys=None),
    dict(ro=None), dict(x=None), dict(ldx=63), dict(ldr=63), dict(lds=63), dict(ldy=63), dict(ldy8=63)])
def test_norm_refuses(L, over):
    assert norm(L, **over) == kda.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(x=A + 1), dict(r=A + 2, rdt=0), dict(w=A + 1), dict(ys=A + 2)])
def test_norm_refuses_misaligned_elements(L, over):
    assert norm(L, **over) == kda.ERR_MISALIGNED


def cache(**over):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, page_stride=4096, head_stride=2048, token_stride=128,
             scale_stride=2, num_pages=3, page_size=16, kv_heads=2, max_blocks=4, block_table=A,
             table_stride=4, kv_lens=A)
    a.update(over)
    return Cache(*a.values())


def append(L, c=None, **over):
    a = dict(q=A, qs=512, k=A, ks=256, v=A, vs=256, rope=A, rows=9, rot=32, inter=0, pos=None, qo=A,
             qos=512, c=ctypes.byref(c if c is not None else cache()), cu=A, ws=A, stream=None, T=4,
             N=1, H=4, wsb=256)
    a.update(over)
    return L.kda_rope_append(*a.values())


@pytest.mark.parametrize("over", [
    dict(page_size=24), dict(page_size=256), dict(num_pages=0), dict(kv_heads=0), dict(max_blocks=-1),
    dict(table_stride=3), dict(scale_stride=1), dict(token_stride=112), dict(head_stride=64),
    dict(page_stride=0), dict(page_stride=1 << 40), dict(k=None), dict(v_scale=None),
    dict(block_table=None), dict(kv_lens=None), dict(max_blocks=1 << 28, table_stride=1 << 28)])
def test_cache_refusals(L, over):
    assert append(L, cache(**over)) == kda.ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(k=A + 8), dict(token_stride=136), dict(page_stride=4104),
                                  dict(k_scale=A + 2), dict(kv_lens=A + 1)])
def test_cache_alignment(L, over):
    assert append(L, cache(**over)) == kda.ERR_MISALIGNED


@pytest.mark.parametrize("over,code", [
    (dict(rot=24), kda.ERR_INVALID_ARG), (dict(rot=144), kda.ERR_INVALID_ARG),
    (dict(rot=-16), kda.ERR_INVALID_ARG), (dict(rope=None), kda.ERR_INVALID_ARG),
    (dict(rows=0), kda.ERR_INVALID_ARG), (dict(inter=2), kda.ERR_INVALID_ARG),
    (dict(T=-1), kda.ERR_INVALID_ARG), (dict(N=-1), kda.ERR_INVALID_ARG), (dict(H=0), kda.ERR_INVALID_ARG),
    (dict(cu=None), kda.ERR_INVALID_ARG), (dict(ws=None), kda.ERR_INVALID_ARG), (dict(k=None), kda.ERR_INVALID_ARG),
    (dict(qo=None), kda.ERR_INVALID_ARG), (dict(ks=248), kda.ERR_INVALID_ARG), (dict(qos=500), kda.ERR_INVALID_ARG),
    (dict(ks=260), kda.ERR_MISALIGNED), (dict(rope=A + 4), kda.ERR_MISALIGNED), (dict(v=A + 2), kda.ERR_MISALIGNED),
    (dict(wsb=128), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_append_refuses(L, over, code):
    assert append(L, **over) == code


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.add_rms_norm(x, x, x[0])
    k = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.rope_append(None, k, k, None, k, k, k, k, k, k, torch.zeros(2))


def test_rope_table():
    t = kda.rope_table(50, 32, base=500.0, device="cpu").double()
    for p in (0, 1, 49):
        for j in (0, 7, 15):
            a = p * 500.0 ** (-2 * j / 32)
            assert abs(t[p, j] - math.cos(a)) < 1e-7 and abs(t[p, 16 + j] - math.sin(a)) < 1e-7
    lin = kda.rope_table(50, 32, base=500.0, scaling="linear", factor=2.0, device="cpu").double()
    assert torch.equal(lin[40], t[20])
    up = kda.rope_table(50, 32, base=500.0, scaling="base", factor=2.0, device="cpu").double()
    assert torch.equal(up[:, 0], t[:, 0])                       # the highest frequency stays
    a = 40 * 500.0 ** (-30 / 32) / 2.0                          # the lowest is divided by the factor
    assert abs(up[40, 15] - math.cos(a)) < 1e-7
    ramp = kda.rope_table(4096, 128, scaling="ramp", factor=4.0, original_positions=1024,
                          device="cpu").double()
    m = 0.1 * math.log(4.0) + 1.0
    assert abs(ramp[1000, 0] - m * math.cos(1000.0)) < 1e-6     # turns often: as it was
    a = 1000 * 10000.0 ** (-126 / 128) / 4.0                    # turns less than once: divided
    assert abs(ramp[1000, 63] - m * math.cos(a)) < 1e-6
    for bad in (dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=160), dict(rot_dim=32, scaling="x"),
                dict(rot_dim=32, scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            kda.rope_table(8, device="cpu", **bad)


def attend(L, c=None, **over):
    a = dict(q=A, qs=512, c=ctypes.byref(c if c is not None else cache()), cu=A, scale=0.1, cap=0.0,
             window=0, o=A, os=512, lse=A, ws=A, stream=None, T=4, N=1, H=4, mq=4, wsb=1 << 30)
    a.update(over)
    return L.kda_cached_attention(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(H=3, qs=512), kda.ERR_INVALID_ARG), (dict(mq=0), kda.ERR_INVALID_ARG),
    (dict(mq=-1), kda.ERR_INVALID_ARG), (dict(window=-1), kda.ERR_INVALID_ARG),
    (dict(scale=float("nan")), kda.ERR_INVALID_ARG), (dict(cap=-0.5), kda.ERR_INVALID_ARG),
    (dict(q=None), kda.ERR_INVALID_ARG), (dict(o=None), kda.ERR_INVALID_ARG), (dict(qs=504), kda.ERR_INVALID_ARG),
    (dict(os=516), kda.ERR_MISALIGNED), (dict(q=A + 8), kda.ERR_MISALIGNED), (dict(lse=A + 2), kda.ERR_MISALIGNED),
    (dict(wsb=0), kda.ERR_WORKSPACE_TOO_SMALL)])
def test_attention_refuses(L, over, code):
    assert attend(L, **over) == code


def test_attention_workspace_size(L):
    assert kda.attention_workspace_size(-1, 8, 2, 1) == 0
    assert kda.attention_workspace_size(1, 8, 3, 1) == 0
    a = kda.attention_workspace_size(4, 8, 2, 1)
    assert a >= 256 and a % 16 == 0
    assert L.kda_cached_attention is not None


def test_binding_packs_the_cache_as_the_header_lays_it_out():
    from kda_gated_delta_chunk_gb300 import layer
    names = [n for n, _ in Cache._fields_]
    raw = layer._CACHE.pack(*range(1, len(names) + 1))
    got = Cache.from_buffer_copy(raw)
    assert layer._CACHE.size == ctypes.sizeof(Cache)
    assert [getattr(got, n) for n in names] == list(range(1, len(names) + 1))


@pytest.mark.parametrize("original,rot,base", [(131072, 128, 10000.0), (65536, 64, 10000.0), (1024, 128, 10000.0),
                                               (4096, 32, 500000.0)])
def test_ramp_divides_in_full_only_what_turns_slowly(original, rot, base):
    """A pair keeps its frequency when it turns beta_fast times or more within the original context,
    is divided in full when it turns beta_slow times or less, and between the two first pairs
    of either kind (wherever they lie) the share grows linearly with the pair's index."""
    factor, fast, slow = 8.0, 32.0, 1.0
    t = kda.rope_table(2, rot, base=base, scaling="ramp", factor=factor, original_positions=original,
                       device="cpu").double()
    amp = 0.1 * math.log(factor) + 1.0
    turns = lambda j: original * base ** (-2 * j / rot) / (2 * math.pi)  # noqa: E731
    last_kept = max(j for j in range(1000) if turns(j) >= fast)
    first_cut = min(j for j in range(1000) if turns(j) <= slow)
    for j in range(rot // 2):
        share = min(max((j - last_kept) / (first_cut - last_kept), 0.0), 1.0)
        want = base ** (-2 * j / rot) * (1 - share + share / factor)
        assert abs(t[1, j] - amp * math.cos(want)) < 2e-7 and abs(t[1, rot // 2 + j] - amp * math.sin(want)) < 2e-7, j


@pytest.mark.parametrize("args", [(2 ** 32 + 1, 8, 2, 1), (1, 2 ** 32 + 8, 2, 1), (1, 8, 2, 2 ** 32), (1, 8, 2, -2 ** 31 - 1)])
def test_sizes_past_32_bits_are_refused(args):
    with pytest.raises(kda.KDAError) as e:
        kda.attention_workspace_size(*args)
    assert e.value.code == kda.ERR_INVALID_ARG


def test_without_the_marshalling_module_the_python_code_takes_the_calls(monkeypatch, tmp_path):
    """... with one warning; it is built per torch version, and a call does not need it."""
    from kda_gated_delta_chunk_gb300 import layer
    monkeypatch.setattr(kbuild, "binding_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(layer, "_native", None)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="none.so is missing"):
        with pytest.raises(ValueError, match="CUDA tensor"):
            kda.add_rms_norm(x, x, x[0])
    import warnings
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="CUDA tensor"):
            kda.add_rms_norm(x, x, x[0])


SIZES = [(h, kv, q) for h in (1, 2, 8, 32, 33, 64, 96, 256) for kv in (1, 2, 4, 8, 32, 64)
         if h % kv == 0 for q in (0, 1, 2, 4, 8, 33, 300)]


def test_attention_workspace_grows_with_every_size(L):
    """A workspace sized for larger heads, kv heads, sequences or query lengths (each on its own)
    serves the smaller call: the size does not fall, and the call does not refuse it."""
    size = {a: kda.attention_workspace_size(3, *a) for a in SIZES}
    for (h, kv, q), n in size.items():
        assert n > 0 and kda.attention_workspace_size(7, h, kv, q) >= n
        for (h2, kv2, q2), m in size.items():
            if h2 <= h and kv2 <= kv and q2 <= q:
                assert m <= n, ((h2, kv2, q2), (h, kv, q))
                if q2:
                    c = cache(kv_heads=kv2, scale_stride=kv2)
                    rc = attend(L, c, T=0, N=0, H=h2, qs=h2 * 128, os=h2 * 128, mq=q2, wsb=n)   # launches nothing
                    assert rc in (kda.OK, kda.ERR_CUDA, kda.ERR_UNSUPPORTED_DEVICE), (rc, h2, kv2, q2)
