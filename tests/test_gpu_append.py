"""rope_append on the GPU against the definition in 64 bits.

Tolerances: rotated queries are one bf16 rounding (at most 2^-8 of the value) of fp32 products
and sums, each within 2^-24 of |a| + |b|.  A cached entry is within half an e4m3 step of the
value plus that; where the fp32 value and the exact one straddle the middle of a step the entry
may be the neighbour.  Scales are equal: the inputs keep the largest magnitudes off the
boundaries 448 * 2^e by more than fp32 rounding.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, D = torch.bfloat16, 128
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def make(lens, starts, H, hk, page, rot, seed=0, layout="hpd", extra=2):
    """Inputs on the host; the caches hold `starts` earlier tokens appended by the reference."""
    g = torch.Generator().manual_seed(seed + 17 * len(lens) + page)
    T, N = sum(lens), len(lens)
    kv = [a + b for a, b in zip(lens, starts)]
    blocks = [-(-b // page) for b in kv]
    width = max(blocks + [1]) + 1
    pages = sum(blocks) + extra
    perm = torch.randperm(pages, generator=g)
    table = torch.full((N, width), -5, dtype=torch.int32)     # never read past the used ones
    at = 0
    for i, b in enumerate(blocks):
        table[i, :b] = perm[at:at + b].int()
        at += b
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(q=rnd(T, H, D).to(BF16), k=rnd(T, hk, D).to(BF16), v=(2 * rnd(T, hk, D)).to(BF16))
    d["kv_lens"] = torch.tensor(kv, dtype=torch.int32)
    d["cu"] = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)) if N else [0], dtype=torch.int32)
    d["table"] = table
    d["rope"] = kda.rope_table(max(kv + [1]), rot, device="cpu") if rot else None
    for c in "kv":
        raw = torch.randint(0, 256, (pages, hk, page, D), generator=g, dtype=torch.uint8)
        raw = torch.where((raw & 0x7F) == 0x7F, torch.zeros_like(raw), raw)   # no NaN
        rc = ref.Cache(raw.view(FP8), torch.full((pages, hk), 3.0))
        for i in range(N):
            rc.append(0.5 * rnd(starts[i], hk, D).double(), table[i], starts[i])
        d[c + "_ref"] = rc
        d[c + "_raw"] = rc.q.float().to(FP8)
        d[c + "_scale"] = rc.s.float()
    return d


def on_gpu(d, layout):
    """Cache tensors on the GPU in one of the accepted layouts."""
    out = []
    pages, hk, page, _ = d["k_raw"].shape
    if layout == "hpd":
        out = [d["k_raw"].cuda(), d["v_raw"].cuda()]
    elif layout == "phd":      # [pages, page, heads, 128]
        out = [d[c].view(torch.uint8).transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in ("k_raw", "v_raw")]
    else:                      # keys and values in one pool
        pool = torch.stack([d["k_raw"].view(torch.uint8), d["v_raw"].view(torch.uint8)], 1).cuda()
        out = [pool[:, 0], pool[:, 1]]
    return out + [d["k_scale"].cuda(), d["v_scale"].cuda()]


def cu(t):
    return None if t is None else t.cuda()


def run(d, caches, interleaved=False, positions=None, **kw):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q = kda.rope_append(cu(d["q"]), d["k"].cuda(), d["v"].cuda(), cu(d["rope"]), *caches,
                        d["table"].cuda(), d["kv_lens"].cuda(), d["cu"].cuda(),
                        interleaved=interleaved, positions=cu(positions), workspace=ws, **kw)
    return q, kda.last_device_status(ws)


def expect(d, interleaved=False, positions=None):
    """The reference's rotated queries; its caches are advanced in place."""
    c = d["cu"].tolist()
    q64 = torch.zeros(d["q"].shape, dtype=torch.float64)
    size = torch.zeros(d["q"].shape, dtype=torch.float64)
    for n, kv in enumerate(d["kv_lens"].tolist()):
        t0, t1 = c[n], c[n + 1]
        k = d["k"][t0:t1].double()
        for t in range(t0, t1):
            p = kv - (t1 - t) if positions is None else int(positions[t])
            if d["rope"] is not None:
                q64[t] = ref.rotate(d["q"][t], d["rope"], p, interleaved)
                k[t - t0] = ref.rotate(d["k"][t], d["rope"], p, interleaved)
            else:
                q64[t] = d["q"][t].double()
            size[t] = d["q"][t].double().abs().amax(-1, keepdim=True) * 2
        d["k_ref"].append(k, d["table"][n], kv)
        d["v_ref"].append(d["v"][t0:t1].double(), d["table"][n], kv)
    return q64, size


def check_cache(got, scale, rc, exact):
    s = scale.cpu().double()
    assert torch.equal(s, rc.s)
    g = got.contiguous().view(FP8).cpu().double()
    if exact:
        assert torch.equal(g, rc.q)
        return
    off = g != rc.q
    # a neighbour, and only where fp32 rounding can decide: a small share of the entries
    step = torch.maximum(rc.q.abs() * 2.0 ** -3, torch.full_like(rc.q, 2.0 ** -9))
    assert bool(((g - rc.q).abs() <= step).all())
    assert float(off.double().mean()) <= 1e-4


CASES = [
    # lens, starts, H, hk, page, rot, interleaved
    ([1], [0], 2, 1, 16, 128, False),
    ([1, 1, 1, 1], [15, 16, 17, 0], 8, 2, 16, 64, True),
    ([5, 0, 33, 1], [0, 7, 30, 63], 4, 4, 32, 128, False),
    ([100, 1, 64], [0, 500, 64], 6, 3, 64, 32, False),
    ([130, 3], [127, 128], 5, 5, 128, 16, True),
    ([64, 65, 63], [1, 0, 1], 3, 1, 64, 0, False),
    ([300], [11], 7, 7, 16, 112, False),
]


@pytest.mark.parametrize("layout", ["hpd", "phd", "pool"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}p{c[4]}r{c[5]}")
def test_rotation_and_append(case, layout):
    lens, starts, H, hk, page, rot, inter = case
    d = make(lens, starts, H, hk, page, rot)
    caches = on_gpu(d, layout)
    q, status = run(d, caches, inter)
    assert status == kda.OK
    q64, size = expect(d, inter)
    tol = 2.0 ** -8 * q64.abs() + 2.0 ** -22 * size
    assert bool(((q.cpu().double() - q64).abs() <= tol).all())
    check_cache(caches[0], caches[2], d["k_ref"], rot == 0)
    check_cache(caches[1], caches[3], d["v_ref"], True)     # values are not rotated: exact
    # the same call again changes nothing
    before = [c.clone() for c in caches]
    run(d, caches, inter)
    for a, b in zip(caches, before):
        assert torch.equal(a.view(torch.uint8) if a.dtype == FP8 else a,
                           b.view(torch.uint8) if b.dtype == FP8 else b)


@pytest.mark.parametrize("page", [16, 64])
def test_the_split_into_calls_does_not_matter(page):
    """One call, or token by token with magnitudes that grow and shrink: the same bytes and
    scales.  Values stay above the smallest normal of the final scale, where requantising by a
    power of two is exact."""
    T, hk = 75, 2
    g = torch.Generator().manual_seed(5)
    x = (1 + torch.rand(T, hk, D, generator=g)) * (torch.randint(0, 2, (T, hk, D), generator=g) * 2 - 1)
    x = (x * 2.0 ** torch.randint(-3, 4, (T, hk, 1), generator=g)).to(BF16).cuda()
    pages = -(-T // page)
    table = torch.randperm(pages, generator=g).int().view(1, -1).cuda()
    def fresh():
        return [torch.zeros(pages, hk, page, D, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2)] + \
            [torch.full((pages, hk), float("nan"), device="cuda") for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    one = fresh()
    kda.rope_append(None, x, x, None, *one, table, i32(T), i32(0, T))
    for cuts in ([1] * T, [10, 1, 20, 44], [74, 1]):
        many, at = fresh(), 0
        for c in cuts:
            kda.rope_append(None, x[at:at + c], x[at:at + c], None, *many, table, i32(at + c), i32(0, c))
            at += c
        for a, b in zip(one, many):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_values_at_the_scales_boundaries():
    """Magnitudes of exactly 448 * 2^e take 2^e, the next bf16 above takes 2^(e+1); zeros and the
    tiniest values take 2^-64; infinities saturate and NaN stays, neither moves the scale."""
    tops = [448.0, 450.0, 1.75, 1.7578125, 2.0 ** -80, 0.0, 2.0 ** 100, 3.0]
    hk = len(tops)
    x = torch.zeros(1, hk, D)
    for h, t in enumerate(tops):
        x[0, h, 0], x[0, h, 1] = -t, t / 2
    x[0, 7, 2], x[0, 7, 3], x[0, 7, 4] = float("inf"), float("-inf"), float("nan")
    x = x.to(BF16)
    kc = torch.zeros(2, hk, 16, D, dtype=torch.uint8, device="cuda").view(FP8)
    vc, ks, vs = kc.clone(), torch.zeros(2, hk, device="cuda"), torch.zeros(2, hk, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kda.rope_append(None, x.cuda(), x.cuda(), None, kc, vc, ks, vs, i32(1).view(1, 1), i32(1), i32(0, 1))
    want = [1.0, 2.0, 2.0 ** -8, 2.0 ** -7, 2.0 ** -64, 2.0 ** -64, 2.0 ** 92, 2.0 ** -7]
    assert ks[1].tolist() == want and vs[1].tolist() == want
    got = vc[1, :, 0].float().cpu()
    assert got[7, 2] == 448 and got[7, 3] == -448 and bool(got[7, 4].isnan())
    for h in range(7):
        assert torch.equal(got[h].double(), ref.e4m3_grid(x[0, h].double() / want[h]))
    assert bool((kc[0].view(torch.uint8) == 0).all())


def test_strided_inputs_positions_and_in_place_queries():
    lens, H, hk = [9, 4], 4, 2
    d = make(lens, [3, 0], H, hk, 32, 64)
    T = sum(lens)
    qkv = torch.zeros(T, (H + 2 * hk) * D + 64, dtype=BF16, device="cuda")
    cols = lambda a, n: qkv[:, a:a + n * D].unflatten(1, (n, D))  # noqa: E731
    q, k, v = cols(8, H), cols(8 + H * D, hk), cols(8 + (H + hk) * D, hk)
    q.copy_(d["q"]); k.copy_(d["k"]); v.copy_(d["v"])  # noqa: E702
    caches = on_gpu(d, "hpd")
    pos = torch.tensor([0, 1, 2, 5, 5, 5, 9, 11, 0, 1, 2, 3, 4], dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = kda.rope_append(q, k, v, d["rope"].cuda(), *caches, d["table"].cuda(), d["kv_lens"].cuda(),
                          d["cu"].cuda(), positions=pos.cuda(), q_out=q, workspace=ws)
    assert out is q and kda.last_device_status(ws) == kda.OK
    q64, size = expect(d, positions=pos)
    assert bool(((q.cpu().double() - q64).abs() <= 2.0 ** -8 * q64.abs() + 2.0 ** -22 * size).all())
    check_cache(caches[0], caches[2], d["k_ref"], False)
    check_cache(caches[1], caches[3], d["v_ref"], True)
    assert torch.equal(k.cpu(), d["k"]) and bool((qkv[:, :8] == 0).all()) and bool((qkv[:, -56:] == 0).all())


@pytest.mark.parametrize("page,long,inter", [(64, 70, False), (64, 19, True), (128, 130, True), (128, 40, False)])
def test_few_new_tokens_in_large_pages(page, long, inter):
    """Pages that are taken in parts: single rows anywhere in a page, and sequences whose new rows
    lie in several parts, with older rows before them."""
    lens = [1] * 30 + [long, 2, 0, 3]
    starts = [(11 * n) % (2 * page) for n in range(30)] + [page - 9, page - 1, 5, 15]
    d = make(lens, starts, 4, 2, page, 64, seed=9)
    caches = on_gpu(d, "hpd")
    q, status = run(d, caches, inter)
    assert status == kda.OK
    q64, size = expect(d, inter)
    assert bool(((q.cpu().double() - q64).abs() <= 2.0 ** -8 * q64.abs() + 2.0 ** -22 * size).all())
    check_cache(caches[0], caches[2], d["k_ref"], False)
    check_cache(caches[1], caches[3], d["v_ref"], True)


def test_many_sequences():
    """More sequences than a CTA has threads, for the pages and for the queries' positions."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (1100,), generator=g).tolist()
    starts = torch.randint(0, 20, (1100,), generator=g).tolist()
    lens[700], starts[901] = 90, 50
    d = make(lens, starts, 2, 1, 16, 32)
    caches = on_gpu(d, "hpd")
    q, status = run(d, caches)
    assert status == kda.OK
    q64, size = expect(d)
    assert bool(((q.cpu().double() - q64).abs() <= 2.0 ** -8 * q64.abs() + 2.0 ** -22 * size).all())
    check_cache(caches[0], caches[2], d["k_ref"], False)
    check_cache(caches[1], caches[3], d["v_ref"], True)


def test_device_errors_skip_and_report():
    """A page outside the pool, a cache longer than the table, fewer cached than new tokens, a
    position outside the rotation table: recorded, and the rest of the batch is right."""
    for broken in ("page", "long", "short", "rope"):
        d = make([3, 4], [5, 20], 2, 2, 16, 32)
        caches = on_gpu(d, "hpd")
        good = make([3, 4], [5, 20], 2, 2, 16, 32)
        expect(good)
        if broken == "page":
            d["table"][0, 0] = d["k_raw"].shape[0]
        elif broken == "long":
            d["kv_lens"][0] = 16 * d["table"].shape[1] + 1
        elif broken == "short":
            d["kv_lens"][0] = 2
        else:
            d["rope"] = d["rope"][:24]      # sequence 1 sits at positions 20 to 23
            d["kv_lens"][0] = 8 + 16 * 1    # ... and sequence 0 now at 21 to 23
            d["rope"] = d["rope"][:23]
        _, status = run(d, caches)
        assert status == kda.ERR_BAD_CACHE_INDEX, broken
        if broken in ("page", "long", "short"):
            for b in range(2):
                pg = int(d["table"][1, b])
                for c, r in ((caches[1], good["v_ref"]),):
                    assert torch.equal(c[pg].cpu().double(), r.q[pg])
            for c, s, before in ((caches[0], caches[2], "k"), (caches[1], caches[3], "v")):
                pg = int(good["table"][0, 0])
                assert torch.equal(c[pg].view(torch.uint8).cpu(), d[before + "_raw"][pg].view(torch.uint8))
                assert torch.equal(s[pg].cpu(), d[before + "_scale"][pg])


def test_empty_calls_and_refusals():
    d = make([4], [0], 2, 2, 16, 32)
    caches = on_gpu(d, "hpd")
    args = lambda: [d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["rope"].cuda(), *caches,  # noqa: E731
                    d["table"].cuda(), d["kv_lens"].cuda(), d["cu"].cuda()]
    a = args()
    z = torch.zeros(0, 2, D, dtype=BF16, device="cuda")
    assert kda.rope_append(z, z, z, a[3], *caches, a[8], torch.zeros_like(a[9]), torch.zeros_like(a[10])).shape == (0, 2, D)
    with pytest.raises(ValueError, match="heads"):
        kda.rope_append(a[0], a[1][:, :1], a[2][:, :1], *a[3:])
    with pytest.raises(TypeError):
        kda.rope_append(a[0], a[1].half(), *a[2:])
    with pytest.raises(kda.KDAError) as e:     # rot_dim 24
        kda.rope_append(*a[:3], a[3][:, :24].contiguous(), *a[4:])
    assert e.value.code == kda.ERR_INVALID_ARG
    odd = [torch.zeros(2, 2, 24, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    with pytest.raises(kda.KDAError) as e:     # page size 24
        kda.rope_append(*a[:4], *odd, torch.ones(2, 2, device="cuda"), torch.ones(2, 2, device="cuda"), *a[8:])
    assert e.value.code == kda.ERR_INVALID_ARG
    wide = torch.zeros(4, 2 * D + 4, dtype=BF16, device="cuda")[:, :2 * D].unflatten(1, (2, D))
    with pytest.raises(kda.KDAError) as e:     # a token stride that is no multiple of 8
        kda.rope_append(a[0], wide, *a[2:])
    assert e.value.code == kda.ERR_MISALIGNED
    with pytest.raises(ValueError, match="strides"):
        kda.rope_append(*a[:5], caches[1].repeat(1, 2, 1, 1)[:, :2], *a[6:])
