"""cached_attention at the edges of what a row sees: windows, pages behind them, extreme sizes,
streams.  References and tolerances as in test_gpu_attention."""
import math

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import layer_ref as ref
from test_gpu_attention import BF16, D, FP8, NAN8, SCALE, check, launch, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def test_nan_at_both_ends_of_a_window_over_three_tiles():
    """Values that only some of a sequence's queries see are NaN, at the window's edge and at the
    causal end, in the channels of one warp; sequences enough that a CTA takes an item's
    three tiles in turn.  Each NaN reaches the rows that see it and no others, whatever the
    order in which the warps run."""
    N, H, hk, page, window, t = 56, 8, 8, 16, 200, 4
    kv = [250 + 5 * n for n in range(N)]
    d = make([t] * N, kv, H, hk, page, seed=31)
    clean, clean_lse, status = launch(d, window=window)
    assert status == kda.OK
    bad = dict(d, v=d["v"].clone())
    want = torch.zeros(N * t, H, D, dtype=torch.bool)
    for n in range(N):
        p = kv[n] - t + torch.arange(t)
        some = [j for j in range(kv[n]) if 0 < int(((j <= p) & (j > p - window)).sum()) < t]
        for i, j in enumerate(some):
            h = (n + i) % hk
            bad["v"][int(d["table"][n, j // page]), h, j % page, 32:64] = NAN8
            sees = (j <= p) & (j > p - window)
            want[n * t:(n + 1) * t, h, 32:64] |= sees[:, None]
    assert bool(want.any())
    for _ in range(20):
        out, lse, status = launch(bad, window=window)
        assert status == kda.OK
        assert torch.equal(out.isnan().cpu(), want)
        assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse, clean_lse)


WINDOWED = [
    # q_lens, kv_lens, heads, kv_heads, window
    ([1, 1, 1], [300, 131, 1000], 8, 2, 20),
    ([1] * 4, [260, 511, 640, 100], 16, 2, 70),
    ([4, 4, 2], [700, 333, 129], 16, 4, 33),
    ([8, 1], [900, 555], 16, 4, 150),
    ([100], [500], 16, 4, 40),
    ([150, 1, 3], [800, 400, 270], 4, 4, 64),
    ([300], [1500], 8, 1, 200),
]


@pytest.mark.parametrize("stale", ["index", "nan", "zero", "inf"])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("case", WINDOWED, ids=lambda c: f"q{c[0]}kv{c[1]}w{c[4]}")
def test_pages_given_back_behind_the_window(case, page, stale):
    """Pages wholly before the window of the sequence's first new query: their table entries point
    nowhere, or their entries are NaN and their scales NaN, zero or infinite."""
    q_lens, kv_lens, H, hk, window = case
    d = make(q_lens, kv_lens, H, hk, page, seed=33)
    for n, (a, b) in enumerate(zip(q_lens, kv_lens)):
        gone = max(0, b - a - window + 1) // page
        pg = d["table"][n, :gone].long()
        if stale == "index":
            d["table"][n, :gone] = -1
        else:
            x = {"nan": float("nan"), "zero": 0.0, "inf": math.inf}[stale]
            for c in "kv":
                d[c][pg] = NAN8
                d[c + "s"][pg] = x
    out, lse, status = launch(d, window=window)
    assert status == kda.OK
    # (the reference reads pages that are not there: give it the last one, which the window hides)
    host = dict(d, table=d["table"].clone())
    for n, b in enumerate(kv_lens):
        row = host["table"][n, :-(-b // page)]
        row[row < 0] = row[-1]
    check(host, out, lse, window=window)


@pytest.mark.parametrize("q_len,kv_len,H,hk", [(4, 308, 8, 2), (120, 400, 4, 2)])
def test_a_page_without_a_scale_stays_with_the_rows_that_see_it(q_len, kv_len, H, hk):
    """A NaN value scale of a page that only the first queries' windows reach: those rows are NaN,
    the others as without it."""
    page, window = 16, 50
    d = make([q_len], [kv_len], H, hk, page, seed=35)
    clean, clean_lse, _ = launch(d, window=window)
    j = kv_len - q_len - window + 1               # the first key of the first query's window
    last = j // page * page + page - 1            # last key of its page
    pg = int(d["table"][0, j // page])
    bad = dict(d, vs=d["vs"].clone())
    bad["vs"][pg, 0] = float("nan")
    out, lse, status = launch(bad, window=window)
    assert status == kda.OK
    p = kv_len - q_len + torch.arange(q_len)
    sees = p - window < last
    assert bool(sees.any()) and not bool(sees.all())
    want = sees[:, None] & (torch.arange(H) < H // hk)
    assert torch.equal(out.cpu().isnan().all(-1), want) and torch.equal(out.cpu().isnan().any(-1), want)
    assert torch.equal(out.cpu()[~want], clean.cpu()[~want])
    assert torch.equal(lse.cpu()[~want], clean_lse.cpu()[~want])


def test_numbers_past_32_bits_are_refused():
    """... and not cut to their low 32 bits; others of an integer type are taken."""
    d = make([2], [90], 4, 2, 16, seed=37)
    for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(max_q=2 ** 32 + 2)):
        with pytest.raises(kda.KDAError) as e:
            launch(d, workspace=kda.alloc_attention_workspace(1, 4, 2, 2), **kw)
        assert e.value.code == kda.ERR_INVALID_ARG, kw
    x = torch.zeros(2, 256, dtype=BF16, device="cuda")
    with pytest.raises(kda.KDAError) as e:
        kda.add_rms_norm(x, None, x[0], want="fp8", group=2 ** 32 + 128)
    assert e.value.code == kda.ERR_INVALID_ARG
    numpy = pytest.importorskip("numpy")
    out, lse, status = launch(d, window=numpy.int64(7), max_q=numpy.int32(2))
    assert status == kda.OK
    check(d, out, lse, window=7)


@pytest.mark.parametrize("q_lens,kv_lens", [([6, 2], [3, 40]), ([40, 300], [30, 250]), ([8, 1], [2, 0])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
def test_windows_as_long_as_an_integer(q_lens, kv_lens, window):
    """A window that hides nothing, with queries that sit before position 0."""
    d = make(q_lens, kv_lens, 4, 2, 16, seed=39)
    out, lse, status = launch(d, window=window)
    assert status == kda.OK
    check(d, out, lse, window=window)


def test_lengths_near_two_to_the_31():
    """The last tiles below position 2^31 - 128, windows nearly as long, and a cache length past
    that bound: refused for its sequence, the others as they are."""
    page, H, hk, window = 16, 2, 1, 100
    top = 2 ** 31 - 128
    for q_len in (1, 3, 40):
        d = make([q_len, q_len], [256, 256], H, hk, page, seed=51)
        near, near_lse, status = launch(d, window=window)
        assert status == kda.OK
        width = 2 ** 27 - 1                                        # 2^31 - 16 positions
        table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
        b = (top - 256) // page
        table[0, b:b + 16] = d["table"][0, :16].cuda()
        table[1, :16] = d["table"][1, :16].cuda()
        far = dict(d, table=table, kv=torch.tensor([top, 256], dtype=torch.int32))
        out, lse, status = launch(far, window=window)
        assert status == kda.OK
        assert torch.equal(out, near) and torch.equal(lse, near_lse)
        far["kv"] = torch.tensor([top + 28, 256], dtype=torch.int32)
        out, lse, status = launch(far, window=window)
        assert status == kda.ERR_BAD_CACHE_INDEX
        assert torch.equal(out[q_len:], near[q_len:]) and torch.equal(lse[q_len:], near_lse[q_len:])
        # queries before position 0 under a window that reaches from there past the integers
        some = dict(far, kv=torch.tensor([q_len // 2, 256], dtype=torch.int32))
        table[0, :16] = d["table"][0, :16].cuda()
        few = dict(some, table=table[:, :17].cpu(), kv_lens=[q_len // 2, 256])
        for w in (2 ** 31 - 129, 2 ** 31 - 20):
            out, lse, status = launch(some, window=w)
            assert status == kda.OK
            check(few, out, lse)


@pytest.mark.parametrize("softcap", [0.01, 2.0, 30.0, 1e3, 1e4, 1e5, 1e30, 3e38, 1e-44])
@pytest.mark.parametrize("q_lens,kv_lens,H,hk", [([1, 1], [700, 90], 8, 2), ([4, 3], [300, 1000], 16, 4),
                                                 ([8, 7], [900, 130], 16, 4), ([130, 2], [400, 300], 4, 2)])
def test_caps_of_any_size(softcap, q_lens, kv_lens, H, hk):
    """A capped score keeps its relative precision whether it is small beside the cap or not: rows
    whose scores all are, rows with both, rows far beyond it.  The score's error of test_gpu_attention
    holds: capping adds 2^-21 of the capped score at most (2^-22 of a cap up to 64: 2^-16), and 2^-14 of
    a bound of the score is there (a sum of 128 magnitudes times the query's largest: 2^-13 and more)."""
    d = make(q_lens, kv_lens, H, hk, 32, seed=61)
    d["q"][:, 1] *= 0.05
    d["q"][:, 2] *= 40.0
    d["q"][0] *= 8.0
    out, lse, status = launch(d, softcap=softcap)
    assert status == kda.OK
    check(d, out, lse, softcap=softcap)


def test_mixed_calls_follow_the_work_before_them():
    """Calls with both kernels right behind the kernels that write their queries, cache and lengths,
    over one workspace, eagerly and from a graph with several such calls: the rows are those of
    the same steps with the GPU waited for between them, and the workspace's status words are left zero."""
    H, hk, page, steps = 16, 4, 64, 6
    q_lens = [1] * 40 + [70, 200]
    base = [2500 + 13 * n for n in range(42)]     # (more than the prefill kernel takes along)
    N, T = len(q_lens), sum(q_lens)
    width = (max(base) + steps * 200) // page + 2
    g = torch.Generator(device="cuda").manual_seed(71)
    table = torch.randperm(N * width, generator=g, device="cuda").int().view(N, width)
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    step = torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    rope = kda.rope_table(width * page, D)
    qkv = torch.randn(steps, T, H + 2 * hk, D, generator=g, device="cuda").to(BF16)
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ws = kda.alloc_attention_workspace(N, H, hk, 200)
    first = [torch.randint(0, 0x70, (N * width, hk, page, D), generator=g, device="cuda", dtype=torch.uint8)
             for _ in range(2)] + [torch.full((N * width, hk), 2.0 ** -7, device="cuda") for _ in range(2)]

    def run(wait, cache, lens, x):
        for a, b in zip(cache, first):
            a.copy_(b)
        lens.copy_(torch.tensor(base, dtype=torch.int32))
        rows = []
        for i in range(steps):
            lens.add_(step)
            x.copy_(qkv[i])
            q = kda.rope_append(*x.split((H, hk, hk), 1), rope, *cache, table, lens, cu, workspace=status)
            if wait:
                torch.cuda.synchronize()
            rows.append(kda.cached_attention(q, *cache, table, lens, cu, SCALE, 200, lse=True, workspace=ws))
            if wait:
                torch.cuda.synchronize()
        return [t for r in rows for t in r]

    own = lambda: ([torch.empty_like(t) for t in first], torch.empty(N, dtype=torch.int32, device="cuda"),  # noqa: E731
                   torch.empty_like(qkv[0]))
    want = run(True, *own())
    assert kda.last_device_status(ws) == kda.OK and not bool(ws[:256].any())
    args = own()
    for _ in range(5):
        got = run(False, *args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not bool(ws[:256].any()) and not bool(status.any())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pinned = torch.tensor(base, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    cache, lens, x = args
    with torch.cuda.graph(graph, stream=side):
        for a, b in zip(cache, first):
            a.copy_(b)
        lens.copy_(pinned)
        rows = []
        for i in range(steps):
            lens.add_(step)
            x.copy_(qkv[i])
            q = kda.rope_append(*x.split((H, hk, hk), 1), rope, *cache, table, lens, cu, workspace=status)
            rows += kda.cached_attention(q, *cache, table, lens, cu, SCALE, 200, lse=True, workspace=ws)
    for _ in range(4):
        for t in rows:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rows, want))
    assert not bool(ws[:256].any())


@pytest.mark.parametrize("softcap", [0.0, 30.0, 1e4])
@pytest.mark.parametrize("q_lens,kv_lens,H,hk", [([1, 3], [700, 90], 8, 2), ([4, 2], [300, 200], 32, 8), ([130, 1], [400, 300], 4, 2)])
def test_a_query_that_is_no_number_stays_in_its_row(softcap, q_lens, kv_lens, H, hk):
    """NaN or infinite entries of a query make its own row NaN (token and head), and no other."""
    d = make(q_lens, kv_lens, H, hk, 16, seed=73)
    clean, clean_lse, _ = launch(d, softcap=softcap)
    bad = dict(d, q=d["q"].clone())
    want = torch.zeros(sum(q_lens), H, dtype=torch.bool)
    for i, (t, h, x) in enumerate([(0, 0, math.nan), (0, H - 1, math.inf), (sum(q_lens) - 1, 1, -math.inf),
                                   (sum(q_lens) // 2, 2, math.nan)]):
        bad["q"][t, h, 5 * i] = x
        want[t, h] = True
    out, lse, status = launch(bad, softcap=softcap)
    assert status == kda.OK
    assert torch.equal(out.cpu().isnan().all(-1), want) and torch.equal(out.cpu().isnan().any(-1), want)
    assert torch.equal(lse.cpu().isnan(), want)
    assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse.cpu()[~want], clean_lse.cpu()[~want])


@pytest.mark.parametrize("scale", [-D ** -0.5, 0.0, 1.0])
@pytest.mark.parametrize("softcap", [0.0, 3.0])
def test_scales_of_any_sign(scale, softcap):
    q_lens, kv_lens, H, hk, page = [1, 4, 90], [300, 77, 200], 8, 2, 16
    d = make(q_lens, kv_lens, H, hk, page, seed=75)
    g = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    out, lse = kda.cached_attention(g["q"], g["k"], g["v"], g["ks"], g["vs"], g["table"], g["kv"], g["cu"], scale,
                                    90, softcap=softcap, lse=True)
    kf, vf = d["k"].view(FP8).float(), d["v"].view(FP8).float()
    for n in range(3):
        a, b = int(d["cu"][n]), int(d["cu"][n + 1])
        args = (d["ks"], d["vs"], d["table"][n], kv_lens[n], scale, softcap)
        o64, l64 = ref.attention(d["q"][a:b], kf, vf, *args)
        big, _ = ref.attention(d["q"][a:b], kf, vf.abs(), *args)
        # as in test_gpu_attention, with |k|_1 below 128 times the largest |k| (3.5 here)
        es = 2.0 ** -14 * abs(scale) * d["q"][a:b].double().abs().amax(-1) * 128 * 3.5
        assert bool(((out[a:b].cpu().double() - o64).abs()
                     <= 2.0 ** -8 * o64.abs() + (2.0 ** -7 + 2.0 ** -14 + 2 * es[..., None]) * big).all())
        assert bool(((lse[a:b].cpu().double() - l64).abs() <= es + 2.0 ** -20 * l64.abs() + 2.0 ** -20).all())


def test_the_largest_group():
    """256 query heads of one kv head, and 255: a row tile is one token."""
    for H in (256, 255):
        d = make([3, 1], [200, 500], H, 1, 64, seed=77)
        out, lse, status = launch(d)
        assert status == kda.OK
        check(d, out, lse)
