"""The two ways a call of the full-attention layer can be marshalled give the same bytes.

The usual call is checked and given its outputs in C++; one that names a stream goes through the
Python checks.  The same kernels run on the same inputs, so the results are equal bit for bit.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from kda_gated_delta_chunk_gb300 import layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def same(a, b):
    if a is None or b is None:
        assert a is None and b is None
        return
    assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and b.is_contiguous()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def cache(g, seqs=3, heads=2, page=16, blocks=4, dtype=torch.float8_e4m3fn):
    pages = seqs * blocks
    k, v = (torch.zeros(pages, heads, page, 128, dtype=torch.uint8, device="cuda").view(dtype) for _ in "kv")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(seqs, blocks)
    return [k, v, torch.ones(pages, heads, device="cuda"), torch.ones(pages, heads, device="cuda"), table]


@pytest.mark.parametrize("want,group", [("bf16", 128), ("fp8", 128), ("fp8", 0), ("both", 128)])
@pytest.mark.parametrize("residual", [None, BF16, torch.float32])
def test_norm(want, group, residual):
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(9, 400, generator=g, device="cuda").to(BF16)
    for x in (wide, wide[:, 8:208], wide[:1, :200], wide[:0]):
        r = None if residual is None else torch.randn(x.shape, generator=g, device="cuda").to(residual)
        w = torch.randn(x.shape[1], generator=g, device="cuda").to(residual or BF16)
        usual = layer._load_native().add_rms_norm(x, r, w, 1e-5, want, group)
        assert type(usual) is tuple
        for a, b, c in zip(usual, kda.add_rms_norm(x, r, w, 1e-5, want, group),
                           kda.add_rms_norm(x, r, w, 1e-5, want, group, stream=torch.cuda.current_stream())):
            same(a, b)
            same(a, c)


@pytest.mark.parametrize("rot,positions,dtype", [(0, False, torch.uint8), (64, False, torch.float8_e4m3fn),
                                                 (128, True, torch.float8_e4m3fn)])
def test_append_and_attention(rot, positions, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    T, cu = 12, torch.tensor([0, 1, 9, 12], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 40, 3], dtype=torch.int32, device="cuda")
    q, k, v = torch.randn(T, 8, 128, generator=g, device="cuda").to(BF16).split((4, 2, 2), 1)
    rope = kda.rope_table(64, rot) if rot else None
    pos = torch.randint(0, 64, (T,), generator=g, device="cuda", dtype=torch.int32) if positions else None
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    a, b = cache(g, dtype=dtype), cache(g, dtype=dtype)
    first = layer._load_native().rope_append(q, k, v, rope, *a, lens, cu, False, pos, status)
    assert isinstance(first, torch.Tensor)
    same(first, kda.rope_append(q, k, v, rope, *b, lens, cu, positions=pos, workspace=status,
                                stream=torch.cuda.current_stream()))
    for x, y in zip(a, b):
        same(x, y)
    ws = kda.alloc_attention_workspace(3, 4, 2, 8)
    for lse in (True, False):
        usual = layer._load_native().cached_attention(first, *a, lens, cu, 0.1, 8, 20.0, 16, lse, ws)
        assert type(usual) is tuple
        other = kda.cached_attention(first, *a, lens, cu, 0.1, 8, 20.0, 16, lse=lse, workspace=ws,
                                     stream=torch.cuda.current_stream())
        same(usual[0], other[0])
        same(usual[1], other[1])
    assert kda.last_device_status(ws) == kda.OK and kda.last_device_status(status) == kda.OK


def test_what_is_not_usual_is_left_alone():
    g = torch.Generator(device="cuda").manual_seed(3)
    native = layer._load_native()
    x, w = torch.randn(4, 64, device="cuda").to(BF16), torch.ones(64, dtype=BF16, device="cuda")
    for args in ((x.cpu(), None, w, 1e-6, "bf16", 128), (x.float(), None, w, 1e-6, "bf16", 128),
                 (x, None, w[:32], 1e-6, "bf16", 128), (x, x[:2], w, 1e-6, "bf16", 128),
                 (x, None, w, "1", "bf16", 128), (x, None, w, 1e-6, "fp4", 128), (x, None, w, 1e-6, "fp8", 2 ** 40),
                 (x.t(), None, w[:4], 1e-6, "bf16", 128), (None, None, w, 1e-6, "bf16", 128), (x,)):
        assert native.add_rms_norm(*args) is None
    c = cache(g)
    lens, cu = torch.full((3,), 4, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    q, ws = torch.randn(3, 4, 128, device="cuda").to(BF16), kda.alloc_attention_workspace(3, 4, 2, 1)
    good = [q, *c, lens, cu, 0.1, 1, 0.0, 0, True, ws]
    assert type(native.cached_attention(*good)) is tuple
    for i, bad in ((0, q.float()), (0, q[..., :64]), (1, c[0].cpu()), (1, c[0].transpose(1, 2)), (2, c[1][:3]),
                   (3, c[2].double()), (4, c[3][:, :1]), (5, c[4][0]), (5, c[4].long()), (6, lens[:2]),
                   (7, cu.long()), (7, cu[::2]), (8, None), (9, 2 ** 31), (12, q), (13, None), (13, q)):
        args = list(good)
        args[i] = bad
        assert native.cached_attention(*args) is None, i
    assert type(native.cached_attention(*good[:9], 0, *good[10:])) is int      # refused by the entry point
    with pytest.raises(kda.KDAError):
        kda.cached_attention(*good[:9], 0, workspace=ws)


def test_without_the_module_the_results_are_the_same(monkeypatch, tmp_path):
    from kda_gated_delta_chunk_gb300 import build as kbuild
    x, w = torch.randn(4, 64, device="cuda").to(BF16), torch.ones(64, dtype=BF16, device="cuda")
    want = kda.add_rms_norm(x, x, w, 1e-6, "both", 128)
    monkeypatch.setattr(kbuild, "binding_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(layer, "_native", None)
    with pytest.warns(RuntimeWarning):
        got = kda.add_rms_norm(x, x, w, 1e-6, "both", 128)
    for a, b in zip(got, want):
        same(a, b)
