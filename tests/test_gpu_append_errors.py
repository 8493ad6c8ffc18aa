"""What rope_append leaves behind a device error: the documented part of the faulty sequence, and the
rest of the batch whole -- queries, keys, values and scales.  References and tolerances as in
test_gpu_append."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
from test_gpu_append import check_cache, expect, make, on_gpu, run

pytestmark = pytest.mark.gpu

LENS, STARTS, H, HK, PAGE, ROT = [3, 4, 2], [5, 20, 30], 2, 2, 16, 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def inputs():
    return make(LENS, STARTS, H, HK, PAGE, ROT, seed=5)


def near(q, q64, size):
    return (q.cpu().double() - q64).abs() <= 2.0 ** -8 * q64.abs() + 2.0 ** -22 * size


def identity(table, row):
    """A table row that turns nothing."""
    table[row, :ROT // 2], table[row, ROT // 2:] = 1.0, 0.0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("given", [False, True], ids=["cache positions", "given positions"])
def test_a_token_outside_the_table_is_left_unrotated(inter, given):
    """Sequence 1's last token (position 23) is past a table of 23 rows, or a position is negative:
    its query and key are as they came, every other token of the batch is rotated."""
    d, good = inputs(), inputs()
    good["rope"] = kda.rope_table(40, ROT, device="cpu")
    if given:
        bad = torch.tensor([5, 6, 7, 20, -1, 22, 23, 2 ** 31 - 1, 3], dtype=torch.int32)
        say = torch.tensor([5, 6, 7, 20, 39, 22, 39, 39, 3], dtype=torch.int32)
        identity(good["rope"], 39)
    else:
        d["kv_lens"][2] = good["kv_lens"][2] = 2       # (a third sequence below the cut: positions 0, 1)
        for x in (d, good):
            x["table"][2, :2] = x["table"][2, :2].flip(0)   # a page of its own, not the one it has filled
        bad = say = None
        identity(good["rope"], 23)
    d["rope"] = kda.rope_table(40, ROT, device="cpu")[:23].contiguous()
    caches = on_gpu(d, "hpd")
    q, status = run(d, caches, inter, bad)
    assert status == kda.ERR_BAD_CACHE_INDEX
    q64, size = expect(good, inter, say)
    assert bool(near(q, q64, size).all())
    left = [4, 6, 7] if given else [6]
    assert torch.equal(q.cpu()[left], d["q"][left])
    check_cache(caches[0], caches[2], good["k_ref"], False)
    check_cache(caches[1], caches[3], good["v_ref"], True)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("broken", ["page", "negative page", "long", "short"])
def test_a_faulty_sequence_leaves_the_others_whole(broken, inter):
    """A page outside the pool, a cache longer than the table, fewer cached than new tokens: nothing
    of that sequence is stored, its own pages stay; the others' queries, keys, values and scales are
    right."""
    d, good = inputs(), inputs()
    good["rope"] = d["rope"] = kda.rope_table(40, ROT, device="cpu")
    before = {c: (d[c + "_raw"].clone(), d[c + "_scale"].clone()) for c in "kv"}
    own = int(d["table"][0, 0])
    if broken == "page":
        d["table"][0, 0] = d["k_raw"].shape[0]
    elif broken == "negative page":
        d["table"][0, 0] = -1
    elif broken == "long":
        d["kv_lens"][0] = PAGE * d["table"].shape[1] + 1
    else:
        d["kv_lens"][0] = 2
    caches = on_gpu(d, "hpd")
    q, status = run(d, caches, inter)
    assert status == kda.ERR_BAD_CACHE_INDEX
    q64, size = expect(good, inter)
    rest = slice(LENS[0], None)
    assert bool(near(q, q64, size)[rest].all())
    if "page" in broken:      # its positions are right: the queries are rotated
        assert bool(near(q, q64, size).all())
    for i, c in enumerate("kv"):
        rc = good[c + "_ref"]
        raw, scale = before[c]
        rc.q[own], rc.s[own] = raw[own].float().double(), scale[own].double()
        check_cache(caches[i], caches[2 + i], rc, c == "v")


def test_pages_past_32_bits():
    """Appends to pages more than 4 GB into the pool, one of them partly filled."""
    page, hk, pages = 128, 8, 36000      # 131072 bytes a page: 4.7 GB
    d = make([150, 1], [100, 0], 2, hk, page, 64, seed=7)
    small = on_gpu(d, "hpd")
    want_q, status = run(d, small)
    assert status == kda.OK
    big = [torch.zeros(pages, hk, page, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    big += [torch.ones(pages, hk, device="cuda") for _ in range(2)]
    far = {0: [35999, 33000], 1: [35500]}
    d2 = dict(d, table=torch.zeros_like(d["table"]))
    for n, pgs in far.items():
        for b, f in enumerate(pgs):
            src = int(d["table"][n, b])
            d2["table"][n, b] = f
            for x, raw in zip(big, (d["k_raw"], d["v_raw"], d["k_scale"], d["v_scale"])):
                x[f] = raw[src].cuda()
    q, status = run(d2, big)
    assert status == kda.OK and torch.equal(q, want_q)
    for n, pgs in far.items():
        for b, f in enumerate(pgs):
            src = int(d["table"][n, b])
            for x, y in zip(big, small):
                assert torch.equal(x[f].contiguous().view(torch.uint8), y[src].contiguous().view(torch.uint8))


@pytest.mark.parametrize("page,step", [(64, 64), (128, 128), (16, 40), (128, 9)])
def test_bad_pages_between_good_ones(page, step):
    """Every other page of a long batch is outside the pool: a CTA passes over such units between good
    ones, whose maxima are its own (rows of very different size from page to page)."""
    n, hk = 60, 4
    lens = [step] * n
    d, good = (make(lens, [0] * n, 2, hk, page, 0, seed=11) for _ in range(2))
    g = torch.Generator().manual_seed(13)
    e = torch.randint(-12, 13, (n, hk), generator=g)
    for x in (d, good):
        for c in "kv":
            x[c] = (x[c].float() * torch.ldexp(torch.ones(n, hk), e).repeat_interleave(step, 0)[..., None]).to(x[c].dtype)
    for seq in range(0, n, 2):
        d["table"][seq] = -1
    expect(good)
    for seq in range(0, n, 2):       # nothing of these is stored
        pg = good["table"][seq, :-(-step // page)].long()
        for c in "kv":
            good[c + "_ref"].q[pg] = d[c + "_raw"].float()[pg].double()
            good[c + "_ref"].s[pg] = d[c + "_scale"][pg].double()
    for _ in range(10):
        caches = on_gpu(d, "hpd")
        status = run(d, caches)[1]
        assert status == kda.ERR_BAD_CACHE_INDEX
        check_cache(caches[0], caches[2], good["k_ref"], True)
        check_cache(caches[1], caches[3], good["v_ref"], True)
