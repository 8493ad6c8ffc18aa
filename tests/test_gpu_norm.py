"""add_rms_norm on the GPU against the definition in 64 bits.

Tolerances: a bf16 result is within half an ulp, at most 2^-8 of the value, of the fp32 one;
the fp32 chain (a sum of at most 32768 squares added pairwise across threads and in at most 32
steps within one, a reciprocal root, two products) is within 2^-17 of the exact value.  An e4m3
result is within half a step: 2^-4 of the value, or 2^-10 scales near zero.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
REL32 = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()
    assert kda.device_check(torch.cuda.current_device()) == kda.OK


def inputs(T, C, rdt=BF16, wdt=BF16, seed=0):
    g = torch.Generator().manual_seed(100 + seed + T + C)
    x = torch.randn(T, C, generator=g).to(BF16)
    r = None if rdt is None else (3 * torch.randn(T, C, generator=g)).to(rdt)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(wdt)
    return x, r, w


def cuda(t):
    return None if t is None else t.cuda()


def check_bf16(got, want):
    tol = (2.0 ** -8 + REL32) * want.abs()
    d = (got.cpu().double() - want).abs()
    assert bool((d <= tol).all()), float((d - tol).max())


def check_fp8(y8, scale, want, group):
    T, C = want.shape
    w = 128 if group else C
    assert scale.shape == (T, -(-C // w))
    s = scale.cpu().double().repeat_interleave(w, 1)[:, :C]
    top = torch.stack([want[:, a:a + w].abs().amax(1) for a in range(0, C, w)], 1)
    ws = (top / 448.0).clamp(min=2.0 ** -40)
    assert bool(((scale.cpu().double() - ws).abs() <= REL32 * ws).all())
    d = (y8.view(torch.float8_e4m3fn).cpu().double() * s - want).abs()
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + REL32 * want.abs()
    assert bool((d <= tol).all()), float((d - tol).max())


SHAPES = [(1, 1), (3, 7), (1, 8), (5, 127), (2, 128), (9, 129), (4, 1000), (7, 1024), (3, 1032),
          (200, 1160), (14, 7168), (160, 7168), (170, 8192), (2, 8193), (153, 32768), (1, 32767)]


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("rdt,wdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32), (None, BF16)])
def test_sum_norm_and_both_outputs(T, C, rdt, wdt):
    x, r, w = inputs(T, C, rdt, wdt)
    s64, y64 = ref.add_rms_norm(x, r, w, 1e-6)
    for group in (128, 0):
        s, y, y8, sc = kda.add_rms_norm(x.cuda(), cuda(r), w.cuda(), 1e-6, want="both", group=group)
        torch.cuda.synchronize()
        if r is None:
            assert s is None
        else:   # one fp32 addition, then one rounding to the residual's type
            assert torch.equal(s.cpu(), (x.float() + r.float()).to(rdt))
        check_bf16(y, y64)
        check_fp8(y8, sc, y64, group)


@pytest.mark.parametrize("C", [512, 1016, 7168])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strided_rows_and_in_place(C, off):
    """Rows in wider buffers (off 1: not even 16-byte aligned); the residual updated in place;
    nothing around the rows is touched."""
    T = 6
    x, r, w = inputs(T, C, seed=1)
    _, y64 = ref.add_rms_norm(x, r, w, 1e-5)
    def wide(t):
        b = torch.full((T, C + 24), 7.0, dtype=t.dtype, device="cuda")
        b[:, off:off + C] = t.cuda()
        return b
    bx, br, by = wide(x), wide(r), wide(torch.zeros_like(x))
    b8 = torch.full((T, C + 24), 9, dtype=torch.uint8, device="cuda")
    view = lambda b: b[:, off:off + C]  # noqa: E731
    s, y, y8, sc = kda.add_rms_norm(view(bx), view(br), w.cuda(), 1e-5, want="both",
                                    residual_out=view(br), y=view(by), y8=view(b8))
    torch.cuda.synchronize()
    assert torch.equal(view(br).cpu(), (x.float() + r.float()).to(BF16))
    check_bf16(view(by), y64)
    check_fp8(view(b8).contiguous(), sc, y64, 128)
    for b in (bx, br, by):
        assert bool((b[:, :off].float() == 7).all()) and bool((b[:, off + C:].float() == 7).all())
    assert bool((b8[:, :off] == 9).all()) and bool((b8[:, off + C:] == 9).all())
    assert torch.equal(view(bx).cpu(), x)


def test_zeros_tiny_and_large_values():
    C = 256
    x = torch.zeros(4, C)
    x[1] = 2.0 ** -70
    x[2] = 2.0 ** 60
    x[3, 5] = 1.0
    w = torch.ones(C)
    w[:128] = 0.0
    x, w = x.to(BF16), w.to(BF16)
    _, y64 = ref.add_rms_norm(x, None, w, 1e-6)
    _, y, y8, sc = kda.add_rms_norm(x.cuda(), None, w.cuda(), 1e-6, want="both")
    torch.cuda.synchronize()
    check_bf16(y, y64)
    check_fp8(y8, sc, y64, 128)
    assert bool((sc[:, 0] == 2.0 ** -40).all())


def test_non_finite_rows_stay_theirs():
    """A NaN or infinity makes its own row non-finite and no other."""
    x, r, w = inputs(5, 640, seed=2)
    x[1, 3] = float("nan")
    x[3, 600] = float("inf")
    _, y64 = ref.add_rms_norm(x[[0, 2, 4]], r[[0, 2, 4]], w, 1e-6)
    for group in (128, 0):
        _, y, y8, sc = kda.add_rms_norm(x.cuda(), r.cuda(), w.cuda(), 1e-6, want="both", group=group)
        torch.cuda.synchronize()
        check_bf16(y[[0, 2, 4]], y64)
        check_fp8(y8.view(torch.uint8)[[0, 2, 4]], sc[[0, 2, 4]], y64, group)
        assert bool(y[1].isnan().all()) and bool(y[3, 600].isnan())
        assert bool(y8[1].float().isnan().all())


def test_no_rows_and_other_stream():
    w = torch.ones(64, dtype=BF16, device="cuda")
    s, y, _, _ = kda.add_rms_norm(torch.empty(0, 64, dtype=BF16, device="cuda"),
                                  torch.empty(0, 64, dtype=BF16, device="cuda"), w)
    assert y.shape == (0, 64)
    x, r, w = inputs(40, 512, seed=3)
    _, y64 = ref.add_rms_norm(x, r, w, 1e-6)
    side = torch.cuda.Stream()
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    side.wait_stream(torch.cuda.current_stream())
    _, y, _, _ = kda.add_rms_norm(xd, rd, wd, stream=side)
    side.synchronize()
    check_bf16(y, y64)


def test_refusals():
    x, r, w = (t.cuda() for t in inputs(2, 64))
    with pytest.raises(TypeError):
        kda.add_rms_norm(x.float(), r, w)
    with pytest.raises(ValueError, match="shape"):
        kda.add_rms_norm(x, r[:1], w)
    with pytest.raises(ValueError, match="want"):
        kda.add_rms_norm(x, r, w, want="int8")
    with pytest.raises(ValueError, match="strided"):
        kda.add_rms_norm(x.t().contiguous().t(), r, w)
    for bad in (dict(group=64, want="fp8"), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises((kda.KDAError, ValueError)):
            kda.add_rms_norm(x, r, w, **bad)
    big = torch.zeros(1, 32776, dtype=BF16, device="cuda")
    with pytest.raises(kda.KDAError) as e:
        kda.add_rms_norm(big, None, big[0])
    assert e.value.code == kda.ERR_INVALID_ARG
