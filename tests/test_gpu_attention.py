"""cached_attention on the GPU against the definition in 64 bits.

Tolerances.  With p = softmax weights and A = sum_j p_j |v_j| (per channel), out carries
 - its own rounding to bf16: at most 2^-8 |out|;
 - the weights as they enter the matrix product: two e4m3 terms or one bf16, within 2^-8 of the
   weight each (and 2^-18 of the largest weight), so at most 2^-8 A + 2^-18 n max_j |v_j| p_max,
   the last below 2^-8 A for the lengths here; the fp32 sums and exponentials, below 2^-14 A;
 - the scores' error e_s, which moves every weight by at most a factor exp(2 e_s): 2 e_s A.
A score's products are summed in fp32 (128 terms: 2^-17 sum |q k| at most); queries split into
two e4m3 terms are exact to 2^-18 of the row's largest entry, so e_s <= scale (2^-16 |q|.|k| +
2^-18 qmax |k|_1) <= 2^-14 scale qmax |k|_1.  lse moves by e_s and by 2^-20 of itself.
"""
import math

import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, D = torch.bfloat16, 128
FP8 = torch.float8_e4m3fn
SCALE = D ** -0.5
NAN8 = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def make(q_lens, kv_lens, H, hk, page, seed=0, spread=0, extra=3):
    """A cache whose pages' scales differ by up to 2^spread; every slot that no position maps to,
    and every page that no sequence owns, holds NaN (and a NaN scale)."""
    g = torch.Generator().manual_seed(seed + 31 * len(q_lens) + page + H)
    N = len(q_lens)
    blocks = [-(-b // page) for b in kv_lens]
    width = max(blocks + [1]) + 1
    pages = sum(blocks) + extra
    perm = torch.randperm(pages, generator=g)
    table = torch.full((N, width), 1 << 30, dtype=torch.int32)
    raw = {c: torch.full((pages, hk, page, D), NAN8, dtype=torch.uint8) for c in "kv"}
    sc = {c: torch.full((pages, hk), float("nan")) for c in "kv"}
    at = 0
    for n, b in enumerate(blocks):
        table[n, :b] = perm[at:at + b].int()
        for i in range(b):
            pg, fill = int(table[n, i]), min(page, kv_lens[n] - i * page)
            for c in "kv":
                x = torch.randn(hk, fill, D, generator=g)
                e = torch.randint(0, spread + 1, (hk,), generator=g).float()
                s = 2.0 ** (-7 + e)
                raw[c][pg, :, :fill] = (x * 2.0 ** 7).clamp(-448, 448).to(FP8).view(torch.uint8)
                sc[c][pg] = s
        at += b
    q = torch.randn(sum(q_lens), H, D, generator=g).to(BF16)
    cu = torch.tensor([0] + [sum(q_lens[:i + 1]) for i in range(N)], dtype=torch.int32)
    return dict(q=q, k=raw["k"], v=raw["v"], ks=sc["k"], vs=sc["v"], table=table, cu=cu,
                kv=torch.tensor(kv_lens, dtype=torch.int32), q_lens=q_lens, kv_lens=kv_lens)


def launch(d, softcap=0.0, window=0, max_q=None, caches=None, **kw):
    ws = kw.pop("workspace", None)
    H, hk = d["q"].shape[1], d["k"].shape[1]
    max_q = max(d["q_lens"] + [1]) if max_q is None else max_q
    if ws is None:
        ws = kda.alloc_attention_workspace(len(d["q_lens"]), H, hk, max_q)
        ws[256:] = 0xFF      # what another call may have left beyond the status words: NaN here
    k, v = caches if caches else (d["k"].cuda(), d["v"].cuda())
    out, lse = kda.cached_attention(d["q"].cuda(), k, v, d["ks"].cuda(), d["vs"].cuda(),
                                    d["table"].cuda(), d["kv"].cuda(), d["cu"].cuda(), SCALE, max_q,
                                    softcap=softcap, window=window, lse=True, workspace=ws, **kw)
    return out, lse, kda.last_device_status(ws)


def check(d, out, lse, softcap=0.0, window=0, seqs=None):
    cu = d["cu"].tolist()
    kf, vf = d["k"].view(FP8).float(), d["v"].view(FP8).float()
    H, hk = d["q"].shape[1], d["k"].shape[1]
    worst = 0.0
    for n in range(len(d["q_lens"])) if seqs is None else seqs:
        a, b = cu[n], cu[n + 1]
        if a == b:
            continue
        args = (d["ks"], d["vs"], d["table"][n], d["kv_lens"][n], SCALE, softcap, window)
        o64, l64 = ref.attention(d["q"][a:b], kf, vf, *args)
        big, _ = ref.attention(d["q"][a:b], kf, vf.abs(), *args)
        pg = d["table"][n][:-(-d["kv_lens"][n] // d["k"].shape[2])].long()
        k1 = torch.nan_to_num(kf[pg].double() * d["ks"][pg].double()[..., None, None]).abs().sum(-1)
        k1 = k1.amax((0, 2)).repeat_interleave(H // hk) if pg.numel() else torch.zeros(H, dtype=torch.float64)
        es = 2.0 ** -14 * SCALE * d["q"][a:b].double().abs().amax(-1) * k1          # [t, H]
        tol = 2.0 ** -8 * o64.abs() + (2.0 ** -7 + 2.0 ** -14 + 2 * es[..., None]) * big
        got, gl = out[a:b].cpu().double(), lse[a:b].cpu().double()
        dead = torch.isinf(l64)
        assert torch.equal(torch.isinf(gl) & (gl < 0), dead)
        assert bool((got[dead] == 0).all())
        d_o = (got - o64).abs()
        assert bool((d_o <= tol).all()), (n, float((d_o / tol.clamp(min=1e-30)).max()))
        d_l = (gl - l64).abs()[~dead]
        assert bool((d_l <= (es + 2.0 ** -20 * l64.abs() + 2.0 ** -20)[~dead]).all()), (n, float(d_l.max()))
        if d_l.numel():
            worst = max(worst, float((d_o / tol.clamp(min=1e-30)).max()))
    return worst


DECODE = [
    # q_lens, kv_lens, heads, kv_heads, page
    ([1], [1], 1, 1, 16),
    ([1], [2], 8, 1, 64),
    ([1, 1, 1], [127, 128, 129], 4, 2, 16),
    ([1, 1, 1, 1], [16, 17, 63, 1000], 6, 3, 32),
    ([1] * 7, [1, 15, 16, 700, 2047, 2048, 2049], 16, 2, 64),
    ([1, 1], [5000, 3], 32, 2, 128),
    ([1], [20000], 8, 8, 64),
    ([2, 1, 0, 3], [130, 300, 77, 3], 8, 2, 16),
    ([4] * 5, [4, 5, 260, 1025, 129], 16, 4, 64),
    ([8, 7], [2000, 999], 16, 2, 32),
    ([1, 1], [512, 4000], 5, 1, 64),
    ([1, 2], [512, 4000], 24, 1, 64),
    ([5, 64], [512, 700], 1, 1, 128),
]
PREFILL = [
    ([128], [128], 2, 1, 64),
    ([65], [65], 1, 1, 16),
    ([257], [257], 4, 2, 32),
    ([200, 3, 1, 130], [500, 3, 900, 131], 4, 4, 64),
    ([512], [1111], 8, 2, 128),
    ([100, 300], [1500, 300], 5, 1, 16),
    ([1, 1, 90], [2500, 30, 90], 40, 2, 64),
    ([3], [700], 128, 1, 64),
    ([1, 1], [300, 2000], 96, 1, 32),
    ([2, 1, 140, 33], [2, 700, 140, 1300], 16, 4, 64),
]


@pytest.mark.parametrize("case", DECODE + PREFILL, ids=lambda c: f"q{c[0]}kv{c[1]}h{c[2]}-{c[3]}p{c[4]}")
def test_plain(case):
    d = make(*case)
    out, lse, status = launch(d)
    assert status == kda.OK
    check(d, out, lse)


@pytest.mark.parametrize("case", DECODE[3:9] + PREFILL[2:6], ids=lambda c: f"q{c[0]}kv{c[1]}")
@pytest.mark.parametrize("softcap,window", [(20.0, 0), (0.0, 1), (0.0, 100), (0.0, 333), (5.0, 128)])
def test_capped_and_windowed(case, softcap, window):
    d = make(*case, seed=3)
    out, lse, status = launch(d, softcap, window)
    assert status == kda.OK
    check(d, out, lse, softcap, window)


@pytest.mark.parametrize("case", [DECODE[4], DECODE[8], PREFILL[3], PREFILL[5]], ids=lambda c: f"q{c[0]}")
def test_scales_that_differ_by_page(case):
    """Scales spread over 2^12 from page to page and between keys and values; and scales that
    are no powers of two."""
    d = make(*case, seed=5, spread=12)
    d["ks"] /= 2.0 ** 8
    d["ks"] *= 1.37
    d["vs"] *= 0.71
    out, lse, status = launch(d)
    assert status == kda.OK
    check(d, out, lse)


@pytest.mark.parametrize("q_lens,kv_lens", [([3, 1], [2, 0]), ([5, 2], [0, 7]), ([40, 70, 1], [30, 0, 5]),
                                            ([200, 140], [100, 141])])
def test_queries_that_see_nothing(q_lens, kv_lens):
    """More new tokens than cached ones: the first queries sit before position 0."""
    d = make(q_lens, kv_lens, 4, 2, 16, seed=7)
    out, lse, status = launch(d)
    assert status == kda.OK
    check(d, out, lse)


@pytest.mark.parametrize("q_len,kv_len,H,hk", [(4, 300, 8, 2), (1, 200, 4, 2), (150, 400, 4, 2), (300, 300, 2, 2)])
@pytest.mark.parametrize("window", [0, 40])
def test_nan_in_one_entry_reaches_only_the_rows_that_see_it(q_len, kv_len, H, hk, window):
    d = make([q_len], [kv_len], H, hk, 16, seed=9)
    at = [j for j in (kv_len - 1, kv_len - q_len // 2 - 1, kv_len - q_len - 20) if j >= 0]
    clean = {c: d[c].clone() for c in "kv"}
    for which in "kv":
        for j in at:
            bad = dict(d)
            bad[which] = d[which].clone()
            pg = int(d["table"][0, j // 16])
            bad[which][pg, 0, j % 16, 7] = NAN8
            out, lse, status = launch(bad, window=window)
            p = kv_len - q_len + torch.arange(q_len)
            sees = (j <= p) & ((p - window < j) if window else True)
            G = H // hk
            o = out.cpu().float()
            if which == "v":     # that channel of the rows that see it
                want = torch.zeros(q_len, H, D, dtype=torch.bool)
                want[sees, :G, 7] = True
                assert torch.equal(o.isnan(), want), j
            else:                # their whole rows
                want = sees[:, None] & (torch.arange(H) < G)
                assert torch.equal(o.isnan().all(-1), want) and torch.equal(o.isnan().any(-1), want), j
                assert torch.equal(lse.cpu().isnan(), want)
            # and everything else is as without it
            keep = ~o.isnan()
            ok, okl, _ = launch({**d, **clean}, window=window)
            assert torch.equal(o[keep], ok.cpu().float()[keep])


def test_large_scores_and_flat_rows():
    """Scores of several hundred (one key takes all the weight), and a zero query (all equal)."""
    d = make([2, 1, 100], [400, 1500, 200], 4, 2, 64, seed=11)
    d["q"][:, 0] *= 300.0
    d["q"][:, 1] = 0
    out, lse, status = launch(d)
    assert status == kda.OK
    check(d, out, lse)


@pytest.mark.parametrize("layout", ["phd", "pool"])
@pytest.mark.parametrize("case", [DECODE[7], PREFILL[3]], ids=["decode", "prefill"])
def test_cache_layouts_and_strided_queries(layout, case):
    d = make(*case, seed=13)
    if layout == "phd":
        caches = [d[c].transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in "kv"]
    else:
        pool = torch.stack([d["k"], d["v"]], 1).cuda()
        caches = [pool[:, 0], pool[:, 1]]
    T, H, _ = d["q"].shape
    wide = torch.full((T, H * D + 40), 9.0, dtype=BF16, device="cuda")
    out_w = wide[:, 16:16 + H * D].unflatten(1, (H, D))
    out, lse, status = launch(d, caches=caches, out=out_w)
    assert status == kda.OK and out is out_w
    check(d, out, lse)
    assert bool((wide[:, :16] == 9).all()) and bool((wide[:, 16 + H * D:] == 9).all())
    qw = torch.zeros(T, H * D + 8, dtype=BF16)
    qw[:, 8:] = d["q"].flatten(1)
    d2 = dict(d, q=qw.cuda()[:, 8:].unflatten(1, (H, D)))
    out2, lse2, _ = launch(d2, caches=caches)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)


def test_workspace_reuse_streams_and_graph():
    """One workspace serves calls of different shapes in a row; the same call gives the same
    bits again, on a side stream and replayed from a graph."""
    a, b = make([1] * 3, [900, 40, 3000], 16, 4, 64, seed=15), make([150, 2], [800, 70], 16, 4, 64, seed=16)
    ws = kda.alloc_attention_workspace(3, 16, 4, 150)
    first = [launch(x, workspace=ws)[:2] for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, (o, l) in zip((b, a), reversed(first)):
        g = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
        torch.cuda.synchronize()
        out, lse = torch.empty_like(o), torch.empty_like(l)
        call = lambda: kda.cached_attention(g["q"], g["k"], g["v"], g["ks"], g["vs"], g["table"],  # noqa: E731
                                            g["kv"], g["cu"], SCALE, max(x["q_lens"]), out=out, lse=lse,
                                            workspace=ws, stream=side)
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        for _ in range(3):
            out.zero_(), lse.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_appended_then_read():
    """rope_append's cache under cached_attention: token by token gives what one prefill gives,
    within the tolerances of both."""
    T, H, hk, page = 70, 4, 2, 32
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, n, D, generator=g).to(BF16).cuda() for n in (H, hk, hk))
    rope = kda.rope_table(T, 128)
    pages = -(-T // page)
    table = torch.randperm(pages, generator=g).int().view(1, -1).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    def fresh():
        return [torch.full((pages, hk, page, D), NAN8, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.full((pages, hk), float("nan"), device="cuda") for _ in range(2)]
    c = fresh()
    qr = kda.rope_append(q, k, v, rope, *c, table, i32(T), i32(0, T))
    whole, _ = kda.cached_attention(qr, *c, table, i32(T), i32(0, T), SCALE, T)
    c, rows = fresh(), []
    for t in range(T):
        qt = kda.rope_append(q[t:t + 1], k[t:t + 1], v[t:t + 1], rope, *c, table, i32(t + 1), i32(0, 1))
        rows.append(kda.cached_attention(qt, *c, table, i32(t + 1), i32(0, 1), SCALE, 1)[0])
    # while a page fills its scale may still be smaller than at the end: finer, not equal, entries
    # in the subnormal range; both are within half an e4m3 step of the same keys and values
    diff = (torch.cat(rows).float() - whole.float()).abs().max()
    assert float(diff) < 0.05


def test_offsets_past_32_bits():
    """Pages more than 4 GB into the pool (byte offsets past 2^32)."""
    page, hk, pages = 128, 8, 36000      # 131072 bytes a page: 4.7 GB
    d = make([1], [300], 16, hk, page, seed=17)
    k = torch.zeros(pages, hk, page, D, dtype=torch.uint8, device="cuda")
    v = torch.zeros(pages, hk, page, D, dtype=torch.uint8, device="cuda")
    ks, vs = torch.zeros(pages, hk), torch.zeros(pages, hk)
    far = [35999, 17, 33000]
    for i, f in enumerate(far):
        src = int(d["table"][0, i])
        k[f], v[f], ks[f], vs[f] = d["k"][src].cuda(), d["v"][src].cuda(), d["ks"][src], d["vs"][src]
    for q_len in (1, 200):
        d2 = make([q_len], [300], 16, hk, page, seed=17)
        d2["table"], d2["k"], d2["v"], d2["ks"], d2["vs"] = d["table"], d["k"], d["v"], d["ks"], d["vs"]
        t = torch.tensor([far + [0]], dtype=torch.int32)
        dd = dict(d2, table=t, ks=ks, vs=vs)
        out, lse, status = launch(dd, caches=(k, v))
        assert status == kda.OK
        check(d2, out, lse)


@pytest.mark.parametrize("N,long", [(300, []), (1100, [5, 800, 1099])])
def test_many_sequences(N, long):
    """More sequences than the threads that add up the batch's work at once, empty ones among them."""
    g = torch.Generator().manual_seed(N)
    q = torch.randint(0, 3, (N,), generator=g).tolist()
    kv = [max(a, int(x)) for a, x in zip(q, torch.randint(0, 60, (N,), generator=g).tolist())]
    for n in long:
        q[n], kv[n] = 70 + n % 7, 90 + n % 200
    d = make(q, kv, 2, 1, 16, seed=21)
    out, lse, status = launch(d)
    assert status == kda.OK
    check(d, out, lse)


@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("short_kv", [2300, 40], ids=["both kernels", "one kernel"])
def test_short_sequences_beside_long_ones(short_kv, softcap):
    """Few rows a sequence, in a call that has long queries too: with enough keys in all these go
    to the kernel for few rows, else to the one for many."""
    q_lens = ([1, 2, 8, 1, 0, 1] * 8) + [100] + [1, 3] + [70]
    kv_lens = [short_kv + 3 * n for n in range(48)] + [500, 0, 2, 70]
    d = make(q_lens, kv_lens, 16, 4, 64, seed=5)
    out, lse, status = launch(d, softcap=softcap)
    assert status == kda.OK
    check(d, out, lse, softcap=softcap)


def test_device_errors_skip_and_report():
    for q_lens, kv_lens in (([1, 1], [100, 200]), ([100, 120], [100, 200])):
        for broken in ("page", "long", "more"):
            d = make(q_lens, kv_lens, 4, 2, 16, seed=19)
            b = dict(d, table=d["table"].clone(), kv=d["kv"].clone())
            max_q = None
            if broken == "page":
                b["table"][0, 2] = -1
            elif broken == "long":
                b["kv"][0] = 16 * d["table"].shape[1] + 1
            else:
                max_q = q_lens[0]
                if q_lens[1] == q_lens[0]:
                    continue
            out, lse, status = launch(b, max_q=max_q)
            assert status == (kda.ERR_INVALID_ARG if broken == "more" else kda.ERR_BAD_CACHE_INDEX), broken
            check(d, out, lse, seqs=[0 if broken == "more" else 1])


def test_refusals():
    d = make([2], [40], 4, 2, 16)
    ws = kda.alloc_attention_workspace(1, 4, 2, 2)
    a = [d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["ks"].cuda(), d["vs"].cuda(), d["table"].cuda(),
         d["kv"].cuda(), d["cu"].cuda()]
    call = lambda *x, **kw: kda.cached_attention(*x, SCALE, kw.pop("mq", 2), **kw)  # noqa: E731
    for kw, code in ((dict(window=-1), kda.ERR_INVALID_ARG), (dict(softcap=-1.0), kda.ERR_INVALID_ARG),
                     (dict(softcap=math.inf), kda.ERR_INVALID_ARG), (dict(mq=0), kda.ERR_INVALID_ARG),
                     (dict(workspace=ws[:128]), kda.ERR_WORKSPACE_TOO_SMALL)):
        with pytest.raises(kda.KDAError) as e:
            call(*a, **kw)
        assert e.value.code == code, kw
    with pytest.raises(kda.KDAError) as e:      # 3 heads over 2
        call(a[0][:, :3].contiguous(), *a[1:], workspace=ws)
    assert e.value.code == kda.ERR_INVALID_ARG
    with pytest.raises(TypeError):
        call(a[0].float(), *a[1:])
    z = torch.empty(0, 4, D, dtype=BF16, device="cuda")
    out, lse = call(z, *a[1:7], torch.zeros(2, dtype=torch.int32, device="cuda"), mq=1, lse=True)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
