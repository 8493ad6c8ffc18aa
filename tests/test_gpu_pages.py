"""cache_accept and the page calls on the GPU against their definitions: bytes, scales, counts and tables are
compared exactly (scales are powers of two, as rope_append makes them; one test takes others)."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import tree_ref as ref
from test_gpu_attention import D, FP8, NAN8
from test_gpu_tree_attention import cu_of, i32, trees_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def status_words():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def cache_of(pages, hk, page, seed, spread=3, layout="heads"):
    """Random e4m3 bytes (no NaN) and power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    shape = (pages, hk, page, D) if layout == "heads" else (pages, page, hk, D)
    out = []
    for _ in range(2):
        raw = (torch.randn(shape, generator=g) * 40).to(FP8).cuda()
        out.append(raw if layout == "heads" else raw.transpose(1, 2))
    scales = [torch.exp2(torch.randint(-spread, 1, (pages, hk), generator=g).float()).cuda() for _ in range(2)]
    return out + scales


def table_of(kv, page, seed, extra=2):
    g = torch.Generator().manual_seed(seed)
    blocks = [-(-b // page) for b in kv]
    perm = torch.randperm(sum(blocks) + extra, generator=g).int()
    table = torch.full((len(kv), max(blocks + [1])), 1 << 30, dtype=torch.int32)
    at = 0
    for n, b in enumerate(blocks):
        table[n, :b] = perm[at:at + b]
        at += b
    return table, sum(blocks) + extra


def f64(x):
    return x.float().double().cpu()


CASES = [
    # nodes, kv_lens, kv_heads, page
    ([1], [1], 1, 16),
    ([8], [1000], 4, 64),
    ([8], [8], 2, 16),
    ([64, 5, 0, 17, 64], [64, 5, 9, 100, 300], 2, 16),
    ([64, 64, 64], [191, 130, 1000], 3, 32),
    ([33, 64], [40, 127], 1, 128),
    ([3] * 40, [3 + 5 * i for i in range(40)], 8, 64),
]


@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("kind", ["any", "chain", "roots"])
@pytest.mark.parametrize("lens,kv,hk,page", CASES)
def test_accept(lens, kv, hk, page, kind, layout):
    trees = trees_of(lens, 21, kind)
    table, pages = table_of(kv, page, 22)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        nodes = [int(torch.randint(-1, n, (1,), generator=g)) if n else -1 for n in lens]
        if seed == 2:
            nodes = [n - 1 for n in lens]       # the last of each
        cache = cache_of(pages, hk, page, seed, layout=layout)
        want = [f64(x) for x in cache]
        ends = []
        for n in range(len(lens)):
            for side in range(2):
                end = ref.accept(want[side], want[2 + side], table[n], kv[n], trees[n], nodes[n])
            ends.append(end)
        ws = status_words()
        got = kda.cache_accept(*cache, table.cuda(), i32(kv), cu_of(lens), i32([p for t in trees for p in t]),
                               i32(nodes), 64, workspace=ws)
        assert kda.last_device_status(ws) == kda.OK
        assert got.tolist() == ends
        for x, y in zip(cache, want):
            assert torch.equal(f64(x), y)


def test_accept_with_scales_that_are_no_powers_of_two():
    """Two roundings: the entry's to e4m3 (half a step, 2^-4 of it or half the smallest value), and the
    ratio's and product's in fp32, which can move it by one more step where it falls on a tie."""
    lens, kv, page = [20], [50], 16
    trees = trees_of(lens, 23)
    table, pages = table_of(kv, page, 24)
    cache = cache_of(pages, 2, page, 1)
    for s in cache[2:]:
        s.mul_(1.37)
        s[::2] *= 0.61
    was = [f64(x) for x in cache]
    node = 19
    kda.cache_accept(*cache, table.cuda(), i32(kv), cu_of(lens), i32(trees[0]), i32([node]), 64)
    path = ref.branch(trees[0], node)
    for side in range(2):
        for e, i in enumerate(path):
            a, b = 30 + i, 30 + e
            pa, pb = int(table[0, a // page]), int(table[0, b // page])
            x = was[side][pa, :, a % page] * was[2 + side][pa, :, None]
            y = f64(cache[side])[pb, :, b % page] * f64(cache[2 + side])[pb, :, None]
            tol = x.abs() * 2.0 ** -3 + f64(cache[2 + side])[pb, :, None] * 2.0 ** -9
            assert bool(((x - y).abs() <= tol).all())


def test_accept_device_errors():
    """A malformed sequence is reported and left alone, its length as it was; the other one is done."""
    lens, kv, page = [4, 6], [20, 38], 16
    trees = [[-1, -1, 1, 2], [-1, 0, -1, 2, 3, 4]]
    table, pages = table_of(kv, page, 25)
    for what, code in (("node", kda.ERR_BAD_TREE), ("short", kda.ERR_BAD_CACHE_INDEX), ("long", kda.ERR_BAD_CACHE_INDEX),
                       ("page", kda.ERR_BAD_CACHE_INDEX), ("most", kda.ERR_INVALID_ARG)):
        cache = cache_of(pages, 2, page, 2)
        want = [f64(x) for x in cache]
        nodes, k, t, most = [3, 5], list(kv), table.clone(), 6
        order = [0, 1]
        if what == "node":
            nodes[0] = 4
        elif what == "short":
            k[0] = 3
        elif what == "long":
            k[0] = 16 * table.shape[1] + 1
        elif what == "page":
            t[0, :] = pages
        else:
            order, most = [1, 0], 4
        for side in range(2):
            end = ref.accept(want[side], want[2 + side], table[order[1]], kv[order[1]], trees[order[1]], nodes[order[1]])
        ws = status_words()
        got = kda.cache_accept(*cache, t.cuda(), i32(k), cu_of(lens), i32(trees[0] + trees[1]), i32(nodes), most,
                               workspace=ws).tolist()
        assert kda.last_device_status(ws) == code, what
        assert got[order[1]] == end
        if what != "page":
            assert got[order[0]] == k[order[0]]
        for x, y in zip(cache, want):
            assert torch.equal(f64(x), y), what


# ------------------------------------------------------------------ the pool
def pool_of(lens, page, width, pages, seed):
    """Rows with their pages in random order."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(pages, generator=g).tolist()
    refs, table = [0] * pages, [[-1] * width for _ in lens]
    for r, n in enumerate(lens):
        for b in range(-(-n // page)):
            table[r][b] = perm.pop()
            refs[table[r][b]] = 1
    return refs, table, list(lens)


def on_gpu(refs, table, lens, pad=3):
    """The block table with padding behind its rows."""
    t = torch.full((len(table), len(table[0]) + pad), 9, dtype=torch.int32)
    t[:, :len(table[0])] = torch.tensor(table, dtype=torch.int32)
    return i32(refs), t.cuda()[:, :len(table[0])], i32(lens)


def same(gpu, plain):
    assert gpu[0].tolist() == plain.refs
    assert gpu[1].tolist() == plain.table
    assert gpu[2].tolist() == plain.lens


@pytest.mark.parametrize("page,rows,width,pages", [(16, 1, 4, 5), (16, 7, 40, 300), (64, 50, 30, 5001), (7, 1500, 3, 40000),
                                                   (32, 3, 2000, 20000)])
def test_a_life_of_the_pool(page, rows, width, pages):
    """Reserve, append, trim, fork, end, over and over: counts, tables and lengths after every call."""
    g = torch.Generator().manual_seed(rows)
    rnd = lambda hi, n=rows: torch.randint(0, hi + 1, (n,), generator=g).tolist()  # noqa: E731
    top = min(width * page, pages * page // (2 * rows))
    state = pool_of([x // 2 for x in rnd(top)], page, width, pages, 3)
    plain, gpu = ref.Pool(*state, page), on_gpu(*state)
    ws = status_words()
    for _ in range(4):
        new = [min(a, width * page - n) for a, n in zip(rnd(top // 2), plain.lens)]
        kda.reserve_pages(*gpu, i32(new), page, workspace=ws)
        plain.reserve(new)
        same(gpu, plain)
        assert max(plain.refs) >= 0 and all(x >= 0 for x in plain.refs)
        kept = [n + (a * k // 4 if a else 0) for n, a, k in zip(plain.lens, new, rnd(4))]
        gpu[2].copy_(i32(kept))
        plain.lens = kept
        kda.free_pages(*gpu, page, workspace=ws)
        plain.free()
        same(gpu, plain)
        order = torch.randperm(rows, generator=g).tolist()
        dst = order[:rows // 3]
        src = [order[rows // 3 + i % max(1, rows // 5)] for i in range(len(dst))]
        if dst:
            kda.free_pages(*gpu, page, rows=i32(dst + dst[:2]), workspace=ws)     # (named twice: once)
            plain.free(dst)
            same(gpu, plain)
            got = kda.fork_pages(*gpu, i32(src), i32(dst), page, workspace=ws)
            want = plain.fork(src, dst)
            assert [x.tolist() for x in got] == [want[0], want[1]]
            same(gpu, plain)
        assert kda.last_device_status(ws) == kda.OK
    kda.free_pages(*gpu, page, rows=i32(list(range(rows))), workspace=ws)
    assert kda.last_device_status(ws) == kda.OK
    assert int(gpu[0].abs().max()) == 0 and int(gpu[2].max()) == 0 and bool((gpu[1] == -1).all())


def test_too_few_pages():
    """The first requests are served; the others' entries stay -1."""
    refs, table, lens = pool_of([20, 5, 40], 16, 6, 8, 4)
    gpu, plain, ws = on_gpu(refs, table, lens), ref.Pool(refs, table, lens, 16), status_words()
    kda.reserve_pages(*gpu, i32([30, 30, 30]), 16, workspace=ws)
    plain.reserve([30, 30, 30])
    assert kda.last_device_status(ws) == kda.ERR_OUT_OF_PAGES
    same(gpu, plain)
    refs, table, lens = pool_of([20, 0, 0], 16, 6, 3, 4)
    gpu, plain = on_gpu(refs, table, lens), ref.Pool(refs, table, lens, 16)
    got = kda.fork_pages(*gpu, i32([0, 0]), i32([1, 2]), 16, workspace=ws)
    want = plain.fork([0, 0], [1, 2])
    assert kda.last_device_status(ws) == kda.ERR_OUT_OF_PAGES
    assert [x.tolist() for x in got] == [want[0], want[1]] and want[1][1] == -1
    same(gpu, plain)


def test_pool_device_errors():
    """What is malformed is reported and left out; what is beside it is done."""
    bad, ws = kda.ERR_BAD_CACHE_INDEX, status_words()
    state = pool_of([20, 33, 40, 0, 0], 16, 4, 12, 5)
    # pairs: a dst twice, a dst that is a source, rows that are none; one in order
    gpu, plain = on_gpu(*state), ref.Pool(*state, 16)
    got = kda.fork_pages(*gpu, i32([0, 0, 1, 2, -1, 7]), i32([3, 3, 2, 4, 1, 1]), 16, workspace=ws)
    assert kda.last_device_status(ws) == bad
    fro, to = plain.fork([2], [4])
    assert got[0].tolist() == [-1, -1, -1, fro[0], -1, -1] and got[1].tolist() == [-1, -1, -1, to[0], -1, -1]
    same(gpu, plain)
    # rows that are none
    gpu, plain = on_gpu(*state), ref.Pool(*state, 16)
    kda.free_pages(*gpu, 16, rows=i32([-1, 1, 5]), workspace=ws)
    plain.free([1])
    assert kda.last_device_status(ws) == bad
    same(gpu, plain)
    # a page outside the pool, and one that nobody held
    gpu, plain = on_gpu(*state), ref.Pool(*state, 16)
    gpu[1][0, 1] = 12
    gpu[0][plain.table[0][0]] = 0
    kda.free_pages(*gpu, 16, rows=i32([0]), workspace=ws)
    assert kda.last_device_status(ws) == bad
    plain.free([0])
    plain.refs[state[1][0][1]] = 1          # (its entry was overwritten: it stays held)
    same(gpu, plain)
    # lengths beyond the table, negative lengths and requests, a page behind an empty block
    gpu, plain = on_gpu(*state), ref.Pool(*state, 16)
    gpu[1][3, 2] = plain.table[3][2] = 11
    kda.reserve_pages(*gpu, i32([45, -1, 24, 40, 5]), 16, workspace=ws)
    assert kda.last_device_status(ws) == bad
    plain.reserve([0, 0, 24, 0, 5])
    same(gpu, plain)
    gpu[2].copy_(i32([65, -1, 40, 0, 0]))
    kda.free_pages(*gpu, 16, workspace=ws)
    assert kda.last_device_status(ws) == bad
    plain.lens = [65, -1, 40, 0, 0]
    for r in (2, 3, 4):
        for b in range(-(-plain.lens[r] // 16), 4):
            if plain.table[r][b] >= 0:
                plain.refs[plain.table[r][b]] -= 1
            plain.table[r][b] = -1
    plain.refs[11] = int(gpu[0][11])        # (whether page 11 was held is this test's own making)
    same(gpu, plain)


@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("page,hk", [(16, 1), (32, 5), (64, 2), (128, 8)])
def test_copy_pages(page, hk, layout):
    cache = cache_of(30, hk, page, 7, layout=layout)
    for c in cache[:2]:
        c.view(torch.uint8)[3] = NAN8       # bytes are copied whatever they are
    want = [x.clone() for x in cache]
    fro, to = [3, 3, 4, -1, 5, 29, 6], [10, 11, 0, 12, -1, 28, 6]
    for a, b in zip(fro, to):
        if a >= 0 and b >= 0:
            for x, y in zip(want, cache):
                x.view(torch.uint8 if x.dtype == FP8 else x.dtype)[b] = y.view(torch.uint8 if y.dtype == FP8 else y.dtype)[a]
    ws = status_words()
    kda.copy_pages(*cache, i32(fro), i32(to), workspace=ws)
    assert kda.last_device_status(ws) == kda.OK
    kda.copy_pages(*cache, i32([30, 7]), i32([1, 30]), workspace=ws)
    assert kda.last_device_status(ws) == kda.ERR_BAD_CACHE_INDEX
    for x, y in zip(want, cache):
        raw = torch.uint8 if x.dtype == FP8 else x.dtype
        assert torch.equal(x.view(raw), y.view(raw))


def test_graph_of_a_fork():
    """Free, fork, copy and reserve captured together, replayed as the lengths change."""
    page, hk = 16, 2
    state = pool_of([100, 37, 0, 0, 0], page, 12, 60, 8)
    plain, gpu = ref.Pool(*state, page), on_gpu(*state)
    cache = cache_of(60, hk, page, 9)
    src, dst, new = i32([0, 1, 0]), i32([2, 3, 4]), i32([20] * 5)
    ws = status_words()

    def step():
        kda.free_pages(*gpu, page, rows=dst, workspace=ws)
        fro, to = kda.fork_pages(*gpu, src, dst, page, workspace=ws)
        kda.copy_pages(*cache, fro, to, workspace=ws)
        kda.reserve_pages(*gpu, new, page, workspace=ws)
        return fro, to

    def expect():
        plain.free(dst.tolist())
        fro, to = plain.fork(src.tolist(), dst.tolist())
        plain.reserve(new.tolist())
        return fro, to

    step()
    expect()
    same(gpu, plain)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fro, to = step()
    for lens in ([110, 40], [112, 48], [33, 50]):
        plain.lens[:2] = lens
        gpu[2][:2] = i32(lens)
        graph.replay()
        want = expect()
        assert fro.tolist() == want[0] and to.tolist() == want[1]
        same(gpu, plain)
        for a, b in zip(*want):
            if a >= 0:
                assert torch.equal(cache[0][a].view(torch.uint8), cache[0][b].view(torch.uint8))
                assert torch.equal(cache[3][a], cache[3][b])
    assert kda.last_device_status(ws) == kda.OK


def test_pages_past_4_gb():
    """Copies between the ends of a cache of more than 2^32 bytes a side, and a branch accepted there."""
    page, hk = 16, 8
    pages = 2 ** 32 // (page * hk * D) + 1000
    k, v = (torch.empty(pages, hk, page, D, dtype=torch.uint8, device="cuda").view(FP8) for _ in "kv")
    ks, vs = (torch.ones(pages, hk, device="cuda") for _ in "kv")
    g = torch.Generator(device="cuda").manual_seed(1)
    ends = [0, 1, pages - 3, pages - 2, pages - 1]
    for c in (k, v):
        for p in ends:
            c[p] = (40 * torch.randn(hk, page, D, generator=g, device="cuda")).to(FP8)
    raw = lambda c, p: c[p].view(torch.uint8).clone()  # noqa: E731
    was = {p: (raw(k, p), raw(v, p)) for p in ends}
    ws = status_words()
    kda.copy_pages(k, v, ks, vs, i32([pages - 1, 0]), i32([1, pages - 2]), workspace=ws)
    assert torch.equal(raw(k, 1), was[pages - 1][0]) and torch.equal(raw(v, pages - 2), was[0][1])
    # 20 cached tokens and 12 nodes in the last two pages; nodes 1, 5, 9 are kept
    table = i32([[pages - 1, pages - 3]])
    tree = [-1, -1, 0, 0, 2, 1, 3, 4, 2, 5, 6, 7]
    lens = kda.cache_accept(k, v, ks, vs, table, i32([32]), i32([0, 12]), i32(tree), i32([9]), 12, workspace=ws)
    assert lens.tolist() == [23] and kda.last_device_status(ws) == kda.OK
    for c, old in ((k, was[pages - 3][0]), (v, was[pages - 3][1])):
        got = raw(c, pages - 3)
        for e, node in enumerate((1, 5, 9)):
            assert torch.equal(got[:, 4 + e], old[:, 4 + node])
        assert torch.equal(got[:, :4], old[:, :4]) and torch.equal(got[:, 7:], old[:, 7:])


def test_the_largest_pool_calls():
    """16384 rows at once; a pool searched to its end."""
    rows, page, pages = 16384, 16, 60000
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[:30000] = 1
    table = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ws = status_words()
    half = rows // 2
    new = torch.zeros(rows, dtype=torch.int32, device="cuda")
    new[:half] = 5
    kda.reserve_pages(refs, table, lens, new, page, workspace=ws)
    assert table[:half, 0].tolist() == list(range(30000, 30000 + half)) and int((table[half:] >= 0).sum()) == 0
    lens[:half] = 5
    src, dst = torch.arange(half, dtype=torch.int32, device="cuda"), torch.arange(half, rows, dtype=torch.int32, device="cuda")
    fro, to = kda.fork_pages(refs, table, lens, src, dst, page, workspace=ws)
    assert fro.tolist() == list(range(30000, 30000 + half)) and to.tolist() == list(range(30000 + half, 30000 + rows))
    assert torch.equal(table[half:, 0], to) and torch.equal(lens[half:], lens[:half])
    assert kda.last_device_status(ws) == kda.OK
    new[:] = 20                      # a second page for every row: 16384 more than the 13616 that are left
    kda.reserve_pages(refs, table, lens, new, page, workspace=ws)
    assert kda.last_device_status(ws) == kda.ERR_OUT_OF_PAGES
    left = pages - 30000 - rows
    assert int((table[:, 1] >= 0).sum()) == left and int((refs == 0).sum()) == 0
    assert table[:left, 1].tolist() == list(range(30000 + rows, pages))
