"""tree_plan and tree_attention on the GPU against their definitions in 64 bits.

Attention's tolerances are those derived in test_gpu_attention: the kernels are the same but for what a
row sees.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import tree_ref as ref
from test_gpu_attention import BF16, D, FP8, NAN8, SCALE, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def trees_of(lens, seed, kind="any"):
    g = torch.Generator().manual_seed(seed)
    return [ref.random_tree(n, g, kind) for n in lens]


def masks_of(trees):
    return [[ref.mask_of(t, i) for i in range(len(t))] for t in trees]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32([sum(lens[:i]) for i in range(len(lens) + 1)])


# ------------------------------------------------------------------ masks and positions
@pytest.mark.parametrize("kind", ["any", "chain", "roots"])
@pytest.mark.parametrize("lens", [[1], [64], [0, 3, 64, 1, 0, 33, 32, 31], [2] * 300])
def test_plan(lens, kind):
    trees = trees_of(lens, 3, kind)
    kv = [n + 17 * i for i, n in enumerate(lens)]
    flat = [p for t in trees for p in t]
    T = len(flat)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    mask = torch.full((T + 2,), 77, dtype=torch.int64, device="cuda")      # two rows of padding
    pos = torch.full((T + 2,), 77, dtype=torch.int32, device="cuda")
    got = kda.tree_plan(i32(flat + [5, 5]), cu_of(lens), i32(kv), 64, mask=mask, positions=pos, workspace=ws)
    assert got[0] is mask and got[1] is pos and kda.last_device_status(ws) == kda.OK
    want = [m for t in masks_of(trees) for m in t]
    assert mask.tolist() == want + [77, 77]
    where = [kv[n] - len(t) + len(ref.branch(t, i)) - 1 for n, t in enumerate(trees) for i in range(len(t))]
    assert pos.tolist() == where + [77, 77]


@pytest.mark.parametrize("parents,kv,most,code", [
    ([0, 0, 1], 9, 8, kda.ERR_BAD_TREE), ([-2, 0, 1], 9, 8, kda.ERR_BAD_TREE), ([-1, 0, 2], 9, 8, kda.ERR_BAD_TREE),
    ([-1, 0, 1], 2, 8, kda.ERR_BAD_CACHE_INDEX), ([-1, 0, 1], 9, 2, kda.ERR_INVALID_ARG)])
def test_plan_device_errors(parents, kv, most, code):
    """The malformed sequence is reported; the one beside it is done all the same."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    mask, pos = kda.tree_plan(i32(parents + [-1, 0]), cu_of([3, 2]), i32([kv, 7]), most, workspace=ws)
    assert kda.last_device_status(ws) == code
    assert mask.tolist()[3:] == [1, 3] and pos.tolist()[3:] == [5, 6]
    if code == kda.ERR_BAD_TREE:     # (a parent that is none counts as the cached text)
        fixed = [p if -1 <= p < i else -1 for i, p in enumerate(parents)]
        assert mask.tolist()[:3] == [ref.mask_of(fixed, i) for i in range(3)]


# ------------------------------------------------------------------ attention
def launch(d, masks, softcap=0.0, window=0, max_q=None, pad=0, **kw):
    H, hk = d["q"].shape[1], d["k"].shape[1]
    max_q = max(d["q_lens"] + [1]) if max_q is None else max_q
    ws = kda.alloc_attention_workspace(len(d["q_lens"]), H, hk, max_q)
    ws[256:] = 0xFF
    q = torch.cat([d["q"], torch.ones(pad, H, D, dtype=BF16)]).cuda()
    m = torch.tensor([x for t in masks for x in t] + [-1] * pad, dtype=torch.int64, device="cuda")
    out, lse = kda.tree_attention(q, d["k"].cuda(), d["v"].cuda(), d["ks"].cuda(), d["vs"].cuda(),
                                  d["table"].cuda(), d["kv"].cuda(), d["cu"].cuda(), m, SCALE, max_q,
                                  softcap=softcap, window=window, lse=True, workspace=ws, **kw)
    return out, lse, kda.last_device_status(ws)


def check(d, masks, out, lse, softcap=0.0, window=0):
    cu = d["cu"].tolist()
    kf, vf = d["k"].view(FP8).float(), d["v"].view(FP8).float()
    H, hk = d["q"].shape[1], d["k"].shape[1]
    for n in range(len(d["q_lens"])):
        a, b = cu[n], cu[n + 1]
        if a == b:
            continue
        q = d["q"][a:b]
        o64, l64, big = ref.attention(q, masks[n], kf, vf, d["ks"], d["vs"], d["table"][n], d["kv_lens"][n],
                                      SCALE, softcap, window)
        pg = d["table"][n][:-(-d["kv_lens"][n] // d["k"].shape[2])].long()
        k1 = torch.nan_to_num(kf[pg].double() * d["ks"][pg].double()[..., None, None]).abs().sum(-1)
        k1 = k1.amax((0, 2)).repeat_interleave(H // hk)
        es = 2.0 ** -14 * SCALE * q.double().abs().amax(-1) * k1
        tol = 2.0 ** -8 * o64.abs() + (2.0 ** -7 + 2.0 ** -14 + 2 * es[..., None]) * big
        got, gl = out[a:b].cpu().double(), lse[a:b].cpu().double()
        dead = torch.isinf(l64)
        assert torch.equal(torch.isinf(gl) & (gl < 0), dead)
        assert bool((got[dead] == 0).all())
        d_o = (got - o64).abs()
        assert bool((d_o <= tol).all()), (n, float((d_o / tol.clamp(min=1e-30)).max()))
        d_l = (gl - l64).abs()[~dead]
        assert bool((d_l <= (es + 2.0 ** -20 * l64.abs() + 2.0 ** -20)[~dead]).all()), (n, float(d_l.max()))


CASES = [
    # nodes, kv_lens, heads, kv_heads, page
    ([1], [1], 4, 4, 16),
    ([1, 1], [700, 129], 8, 2, 64),
    ([8], [8], 4, 1, 32),                       # nothing cached but the tree
    ([8], [1000], 16, 4, 64),                   # 32 rows: the last that the decode kernel takes
    ([9], [1000], 16, 4, 64),
    ([5, 8, 1, 0, 3], [300, 128, 127, 50, 640], 8, 2, 16),
    ([32, 17], [129, 400], 4, 4, 128),
    ([64], [64], 8, 8, 16),
    ([64, 2, 33], [1000, 130, 640], 16, 2, 32),   # both kernels, rows in two and more tiles
    ([64, 64], [191, 320], 4, 4, 64),           # the nodes in two key tiles
    ([31, 1, 64, 7], [2000, 1500, 70, 1024], 16, 1, 128),
    ([3] * 90, [40 + 13 * i for i in range(90)], 4, 2, 16),
]


@pytest.mark.parametrize("kind", ["any", "chain", "roots"])
@pytest.mark.parametrize("lens,kv,H,hk,page", CASES)
def test_attention(lens, kv, H, hk, page, kind):
    d = make(lens, kv, H, hk, page, seed=5, spread=3)
    masks = masks_of(trees_of(lens, 9, kind))
    out, lse, status = launch(d, masks)
    assert status == kda.OK
    check(d, masks, out, lse)


@pytest.mark.parametrize("lens,kv,H,hk,page", CASES)
def test_any_masks(lens, kv, H, hk, page):
    """Masks that are no tree's: empty ones, nodes that do not see themselves or see later ones, bits
    past the sequence's nodes."""
    d = make(lens, kv, H, hk, page, seed=6)
    g = torch.Generator().manual_seed(1)
    masks = [[0 if (i + n) % 3 == 0 else int(torch.randint(-2 ** 62, 2 ** 62, (1,), generator=g)) * 2 + 1
              for i in range(x)] for n, x in enumerate(lens)]
    out, lse, status = launch(d, masks)
    assert status == kda.OK
    check(d, masks, out, lse)


@pytest.mark.parametrize("softcap", [0.0, 5.0, 100.0])
@pytest.mark.parametrize("lens,kv,H,hk,page,window", [
    ([8, 3], [1000, 300], 16, 4, 16, 8), ([8, 3], [1000, 300], 16, 4, 64, 150), ([64, 20], [900, 700], 8, 2, 32, 64),
    ([64, 5, 1], [1500, 900, 400], 16, 2, 16, 333), ([6], [70], 4, 4, 16, 2 ** 31 - 1), ([64], [200], 8, 2, 16, 70)])
def test_window_and_cap(lens, kv, H, hk, page, window, softcap):
    """Pages wholly before every node's window are not read: their table entries are stale."""
    d = make(lens, kv, H, hk, page, seed=8)
    for n, (a, b) in enumerate(zip(lens, kv)):
        first = max(0, b - a + 0 - window)           # (a node that saw no other one would see from here)
        d["table"][n, :first // page] = 1 << 29
    masks = masks_of(trees_of(lens, 4))
    out, lse, status = launch(d, masks, softcap=softcap, window=window)
    assert status == kda.OK
    safe = dict(d, table=d["table"].clamp(max=d["k"].shape[0] - 1))
    check(safe, masks, out, lse, softcap, window)


@pytest.mark.parametrize("lens,H,hk", [([8] * 20, 8, 2), ([24] * 6, 16, 2)])
def test_nan_entries_reach_the_nodes_that_see_them(lens, H, hk):
    """NaN values in the nodes' own entries and in the cached text's end of the window."""
    kv, page, window = [400 + 7 * n for n in range(len(lens))], 16, 100
    d = make(lens, kv, H, hk, page, seed=11)
    masks = masks_of(trees_of(lens, 12))
    clean, clean_lse, status = launch(d, masks, window=window)
    assert status == kda.OK
    bad = dict(d, v=d["v"].clone())
    want = torch.zeros(sum(lens), H, D, dtype=torch.bool)
    at = 0
    for n, (a, b) in enumerate(zip(lens, kv)):
        seen = [set(ref.seen_of(m, a, b, window)) for m in masks[n]]
        some = [j for j in range(b - a - window, b) if 0 < sum(j in s for s in seen) < a]
        for i, j in enumerate(some):
            h, c = (n + i) % hk, 32 * (i % 4)
            bad["v"][int(d["table"][n, j // page]), h, j % page, c:c + 16] = NAN8
            for r in range(a):
                if j in seen[r]:
                    want[at + r, h * (H // hk):(h + 1) * (H // hk), c:c + 16] = True
        at += a
    assert bool(want.any())
    for _ in range(10):
        out, lse, status = launch(bad, masks, window=window)
        assert status == kda.OK
        assert torch.equal(out.isnan().cpu(), want)
        assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse, clean_lse)


def test_rows_behind_the_last_sequence_stay():
    lens, kv = [5, 40], [77, 300]
    d = make(lens, kv, 8, 2, 16, seed=13)
    masks = masks_of(trees_of(lens, 14))
    out = torch.full((45 + 6, 8, D), 3.0, dtype=BF16, device="cuda")
    got, lse, status = launch(d, masks, pad=6, out=out)
    assert got is out and status == kda.OK and bool((out[45:] == 3.0).all())
    check(d, masks, out, lse)


def test_device_errors():
    """A cache shorter than the tree, and a tree of more nodes than max_q_len: reported, not written."""
    lens = [4, 9]
    d = make(lens, [60, 70], 8, 2, 16, seed=15)
    masks = masks_of(trees_of(lens, 16))
    for kv, most, code in (([3, 70], 9, kda.ERR_BAD_CACHE_INDEX), ([60, 70], 8, kda.ERR_INVALID_ARG)):
        out = torch.full((13, 8, D), 3.0, dtype=BF16, device="cuda")
        e = dict(d, kv=torch.tensor(kv, dtype=torch.int32))
        _, _, status = launch(e, masks, max_q=most, out=out)
        gone, done = (slice(0, 4), slice(4, 13)) if code == kda.ERR_BAD_CACHE_INDEX else (slice(4, 13), slice(0, 4))
        assert status == code
        assert bool((out[gone] == 3.0).all()) and not bool((out[done] == 3.0).all(-1).any())


def test_graph_and_stream():
    """Captured on one stream and replayed after the inputs have changed; run on a named stream."""
    lens, kv = [8, 30, 1], [200, 500, 90]
    d = make(lens, kv, 16, 4, 16, seed=17)
    t = {k: d[k].cuda() for k in ("q", "k", "v", "ks", "vs", "table", "kv", "cu")}
    trees = [trees_of(lens, s) for s in (18, 19)]
    parents = i32([p for x in trees[0] for p in x])
    ws = kda.alloc_attention_workspace(3, 16, 4, 30)
    plan_ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step(stream=None):
        mask, pos = kda.tree_plan(parents, t["cu"], t["kv"], 30, workspace=plan_ws, stream=stream)
        return kda.tree_attention(t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["kv"], t["cu"], mask,
                                  SCALE, 30, lse=True, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for x in trees:
        parents.copy_(i32([p for y in x for p in y]))
        graph.replay()
        check(d, masks_of(x), out, lse)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o2, l2 = step(other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert kda.last_device_status(ws) == kda.OK and kda.last_device_status(plan_ws) == kda.OK


@pytest.mark.parametrize("n,H,hk,page", [(16, 16, 4, 128), (16, 16, 4, 16), (32, 16, 4, 64), (64, 16, 4, 32), (64, 32, 4, 64),
                                         (3, 16, 4, 64)])
def test_many_tiles_a_cta(n, H, hk, page):
    """Long caches: every CTA takes dozens of key tiles one after the other, and starts and ends inside
    sequences."""
    lens, kv = [n] * 8, [15000 + 131 * i for i in range(8)]
    d = make(lens, kv, H, hk, page, seed=41)
    masks = masks_of(trees_of(lens, 42))
    out, lse, status = launch(d, masks)
    assert status == kda.OK
    again = launch(d, masks)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    some = [0, 3, 7]
    cu = [0, n, 2 * n, 3 * n]
    part = dict(d, q_lens=[n] * 3, kv_lens=[kv[i] for i in some], cu=torch.tensor(cu, dtype=torch.int32),
                table=d["table"][some], q=torch.cat([d["q"][n * i:n * (i + 1)] for i in some]))
    pick = lambda x: torch.cat([x[n * i:n * (i + 1)] for i in some])  # noqa: E731
    check(part, [masks[i] for i in some], pick(out), pick(lse))


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (5.0, 0), (100.0, 150), (0.0, 64)])
@pytest.mark.parametrize("lens,kv,H,hk,page", [
    ([40, 3, 5, 8, 64, 2], [300, 900, 131, 128, 1000, 70], 16, 4, 32),     # row tiles of 128: two, and one beside
    ([20, 9, 32], [900, 700, 33], 8, 2, 16),
    ([16, 1, 16], [129, 1500, 640], 16, 2, 64)])
def test_half_filled_row_tiles(lens, kv, H, hk, page, softcap, window):
    """Batches whose trees fill less than half of the largest row tile, with windows and capped scores."""
    d = make(lens, kv, H, hk, page, seed=51, spread=2)
    masks = masks_of(trees_of(lens, 52))
    out, lse, status = launch(d, masks, softcap=softcap, window=window)
    assert status == kda.OK
    check(d, masks, out, lse, softcap, window)


def test_nan_entries_in_half_filled_row_tiles():
    """As above at 128 rows and at 160 beside small trees."""
    for lens in ([16] * 6, [20, 2, 3, 9]):
        test_nan_entries_reach_the_nodes_that_see_them(lens, 16, 2)


def test_a_node_that_is_no_number():
    """A NaN or infinite query makes its own rows NaN and no others, in both kernels and both orders."""
    for lens, H, hk in (([6, 3], 8, 2), ([20, 9], 8, 2), ([40, 64], 16, 2)):
        d = make(lens, [300, 400], H, hk, 16, seed=53)
        masks = masks_of(trees_of(lens, 54))
        clean, clean_lse, status = launch(d, masks)
        bad = dict(d, q=d["q"].clone())
        bad["q"][2, 1, 5] = float("nan")
        bad["q"][4, 3, 7] = float("inf")
        out, lse, status = launch(bad, masks)
        assert status == kda.OK
        want = torch.zeros(sum(lens), H, dtype=torch.bool)
        want[2, 1] = want[4, 3] = True
        assert torch.equal(out.isnan().all(-1).cpu(), want) and torch.equal(out.isnan().any(-1).cpu(), want)
        assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse.cpu()[~want], clean_lse.cpu()[~want])
