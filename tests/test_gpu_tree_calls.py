"""The operators on drafted trees and pages in calls as a server makes them: strided tensors, padded batches whose
lengths change between replays, graphs that share a workspace, several streams at once, pages without a
scale.  Results are compared with the same call made plainly, bit for bit."""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import kda_workloads as W
import test_gpu_pages as pages_test
import test_gpu_tree_recurrent as rec
from test_gpu_attention import BF16, D, SCALE, make
from test_gpu_tree_attention import check, cu_of, i32, launch, masks_of, trees_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


# few rows a sequence; row tiles of 256; row tiles of 128 in turns; several of these in one batch
SHAPES = [([8, 3, 1], 16, 4), ([64, 60], 16, 2), ([16, 12], 16, 4), ([2, 40, 7, 30], 16, 4)]


@pytest.mark.parametrize("lens,H,hk", SHAPES)
@pytest.mark.parametrize("page", [16, 128])
def test_strided_attention(lens, H, hk, page):
    """Queries in a fused projection, caches with tokens outside heads and spare rows between, a table inside
    a wider one, outputs in a wider row."""
    kv = [500 + 77 * n for n in range(len(lens))]
    d = make(lens, kv, H, hk, page, seed=61)
    masks = masks_of(trees_of(lens, 62))
    want, lse, status = launch(d, masks)
    assert status == kda.OK
    check(d, masks, want, lse)
    T, N = sum(lens), len(lens)
    fused = torch.full((T, (H + 2) * D), float("nan"), dtype=BF16, device="cuda")
    q = fused[:, D:(H + 1) * D].view(T, H, D)
    q.copy_(d["q"])
    caches = []
    for c in "kv":
        raw = torch.full((d[c].shape[0], page, hk + 1, D), 0x7F, dtype=torch.uint8, device="cuda")
        raw[:, :, :hk] = d[c].transpose(1, 2).cuda()
        caches.append(raw[:, :, :hk].transpose(1, 2))
    table = torch.full((N, d["table"].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :d["table"].shape[1]] = d["table"].cuda()
    rows = torch.full((T, H + 3, D), 3.0, dtype=BF16, device="cuda")
    m = torch.tensor([x for t in masks for x in t], dtype=torch.int64, device="cuda")
    ws = kda.alloc_attention_workspace(N, H, hk, max(lens))
    out, l2 = kda.tree_attention(q, *caches, d["ks"].cuda(), d["vs"].cuda(), table[:, :d["table"].shape[1]],
                                 d["kv"].cuda(), d["cu"].cuda(), m, SCALE, max(lens), out=rows[:, 1:H + 1], lse=True,
                                 workspace=ws)
    assert kda.last_device_status(ws) == kda.OK
    assert torch.equal(out, want) and torch.equal(l2, lse)
    assert bool((rows[:, 0] == 3.0).all()) and bool((rows[:, H + 1:] == 3.0).all())


@pytest.mark.parametrize("kind", ["roots", "chain"])
@pytest.mark.parametrize("n,H,hk", [(8, 16, 4), (16, 16, 4), (40, 16, 2)])
def test_a_page_of_nodes_without_a_scale(n, H, hk, kind):
    """The last page holds the later half of the nodes and a value scale that is NaN: those that see one of
    them are NaN, the others as without it."""
    page = 16
    later = min(n // 2, 16)
    kv = 320 + later                 # the last page: nodes n - later .. n - 1
    d = make([n], [kv], H, hk, page, seed=63)
    masks = masks_of(trees_of([n], 64, kind))
    clean, clean_lse, status = launch(d, masks)
    assert status == kda.OK
    bad = dict(d, vs=d["vs"].clone())
    bad["vs"][int(d["table"][0, (kv - 1) // page]), 1] = float("nan")
    out, lse, status = launch(bad, masks)
    assert status == kda.OK
    G = H // hk
    want = (torch.arange(n) >= n - later)[:, None] & (torch.arange(H) // G == 1)
    assert torch.equal(out.cpu().isnan().all(-1), want) and torch.equal(out.cpu().isnan().any(-1), want)
    assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse.cpu()[~want], clean_lse.cpu()[~want])


def test_graphs_that_share_a_workspace():
    """Four captured calls of different shapes (and a causal one) on one workspace, replayed in any order."""
    big = kda.alloc_attention_workspace(4, 16, 4, 64)
    runs = []
    for i, (lens, H, hk) in enumerate(SHAPES):
        d = make(lens, [3000 + 500 * n for n in range(len(lens))], H, hk, 64, seed=65 + i)
        masks = masks_of(trees_of(lens, 66))
        m = torch.tensor([x for t in masks for x in t], dtype=torch.int64, device="cuda")
        a = [d[x].cuda() for x in ("q", "k", "v", "ks", "vs", "table", "kv", "cu")]
        own = kda.alloc_attention_workspace(len(lens), H, hk, 64)
        if own.numel() > big.numel():
            big = own

        def tree(ws, a=a, m=m, lens=lens):
            return kda.tree_attention(*a, m, SCALE, max(lens), lse=True, workspace=ws)

        def causal(ws, a=a, lens=lens):
            return kda.cached_attention(*a, SCALE, max(lens), lse=True, workspace=ws)
        runs += [(f, f(own)) for f in (tree, causal)]
    torch.cuda.synchronize()
    graphs = []
    for f, _ in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f(big)
        graphs.append((g, out))
    order = torch.randperm(4 * len(runs), generator=torch.Generator().manual_seed(1)) % len(runs)
    for i in order.tolist():
        for t in graphs[i][1]:
            t.fill_(7.0)
        graphs[i][0].replay()
        assert all(torch.equal(x, y) for x, y in zip(graphs[i][1], runs[i][1])), i
    assert kda.last_device_status(big) == kda.OK


def test_streams_at_once():
    """Attention, recurrence and a prefill of another batch on streams of their own, each with its workspace."""
    lens = [16, 64, 3, 30] * 4
    trees = trees_of(lens, 67)
    parents = [p for t in trees for p in t]
    d = make(lens, [2000 + 111 * n for n in range(len(lens))], 16, 4, 64, seed=68)
    m = torch.tensor([x for t in masks_of(trees) for x in t], dtype=torch.int64, device="cuda")
    a = [d[x].cuda() for x in ("q", "k", "v", "ks", "vs", "table", "kv", "cu")]
    r = rec.make(lens, 16, seed=69)
    cu, up, nodes = cu_of(lens), i32(parents), i32([n - 1 for n in lens])
    inp = W.make_inputs(W.custom([700, 900], 16, seed=70))
    f = [x.cuda() if isinstance(x, torch.Tensor) else x
         for x in (inp[n] for n in ("q", "k", "v", "g", "beta", "A_log", "dt_bias", "lower_bound", "scale",
                                    "initial_state", "cu_seqlens"))]
    ws = [kda.alloc_attention_workspace(len(lens), 16, 4, 64), rec.status_words(), None]

    def attend():
        return kda.tree_attention(*a, m, SCALE, 64, lse=True, workspace=ws[0])

    def recur():
        out, u = kda.tree_recurrent_fwd(r["q"], r["k"], r["v"], r["g"], r["beta"], r["A_log"], r["dt_bias"], -5.0,
                                        W.SCALE, r["state"], cu, up, 64, workspace=ws[1])
        fin = kda.tree_commit(r["k"], r["g"], r["A_log"], r["dt_bias"], -5.0, r["state"], cu, up, u, nodes, 64,
                              workspace=ws[1])
        return out, u, fin

    def prefill():
        return kda.chunk_prefill_fwd(*f)

    calls = [attend, recur, prefill]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(10):
        for i, (s, c) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for w, all_ in zip(want, got):
        for x in all_:
            assert all(torch.equal(p, q) for p, q in zip(w, x) if isinstance(p, torch.Tensor))
    assert kda.last_device_status(ws[0]) == kda.OK and kda.last_device_status(ws[1]) == kda.OK


def test_a_padded_step_whose_lengths_change():
    """A captured step of room for 40 tokens and 4 sequences: plan, recurrence, commit and accept are replayed
    with fewer, and none, of them.  Rows behind the last sequence hold NaN (parents: nonsense) and stay."""
    T, N, H, hk, page, most = 40, 4, 4, 2, 16, 16
    d = rec.make([10] * N, H, seed=71)
    for x in ("q", "k", "v", "g", "beta"):
        d[x] = d[x].clone()
    full = {x: d[x].clone() for x in ("q", "k", "v", "g", "beta")}
    cu, up, kv, nodes = i32([0] * (N + 1)), i32([9] * T), i32([0] * N), i32([-1] * N)
    kc, vc, ks, vs = pages_test.cache_of(60, hk, page, 72)
    first = [x.clone() for x in (kc, vc, ks, vs)]
    table = torch.randperm(60, generator=torch.Generator().manual_seed(3)).int().cuda().view(N, 15)
    ws = rec.status_words()
    mask = torch.empty(T, dtype=torch.int64, device="cuda")
    pos = torch.empty(T, dtype=torch.int32, device="cuda")
    out = torch.empty(T, H, D, dtype=BF16, device="cuda")
    u = torch.empty(T, H, D, device="cuda")
    fin = torch.empty_like(d["state"])
    after = torch.empty_like(kv)

    def step():
        kda.tree_plan(up, cu, kv, most, mask=mask, positions=pos, workspace=ws)
        kda.tree_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["A_log"], d["dt_bias"], -5.0, W.SCALE,
                               d["state"], cu, up, most, out=out, u=u, workspace=ws)
        kda.tree_commit(d["k"], d["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], cu, up, u, nodes, most,
                        final_state=fin, workspace=ws)
        kda.cache_accept(kc, vc, ks, vs, table, kv, cu, up, nodes, most, lens_out=after, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([10, 10, 10, 10], [16, 1, 0, 7], [0, 0, 0, 0], [0, 3, 16, 0]):
        n = sum(lens)
        trees = trees_of(lens, 73)
        flat = [p for t in trees for p in t]
        for x in full:
            d[x].copy_(full[x])
            d[x][n:] = float("nan")
        for x, y in zip((kc, vc, ks, vs), first):
            x.copy_(y)
        cu.copy_(cu_of(lens))
        up.copy_(i32(flat + [99] * (T - n)))
        kv.copy_(i32([x + 50 * i for i, x in enumerate(lens)]))
        ends = [x - 1 for x in lens]
        nodes.copy_(i32(ends))
        for x in (mask, pos, out, u, fin, after):
            x.fill_(7)
        graph.replay()
        assert kda.last_device_status(ws) == kda.OK
        for x in (mask, pos, out, u):
            assert bool((x[n:] == 7).all())
        assert mask[:n].tolist() == [m for t in masks_of(trees) for m in t]
        rec.check(d, lens, trees, ends, out, u, fin)
        short = {x: d[x][:n].contiguous() for x in full}
        got = [x.clone() for x in (out[:n], u[:n], fin, after, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
        for x, y in zip((kc, vc, ks, vs), first):
            x.copy_(y)
        o2, u2 = kda.tree_recurrent_fwd(*short.values(), d["A_log"], d["dt_bias"], -5.0, W.SCALE, d["state"], cu,
                                        up[:n], most, workspace=ws)
        f2 = kda.tree_commit(short["k"], short["g"], d["A_log"], d["dt_bias"], -5.0, d["state"], cu, up[:n], u2, nodes,
                             most, workspace=ws)
        l2 = kda.cache_accept(kc, vc, ks, vs, table, kv, cu, up[:n], nodes, most, workspace=ws)
        plain = (o2, u2, f2, l2, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)
        assert all(torch.equal(x, y) for x, y in zip(got, plain))
        assert kda.last_device_status(ws) == kda.OK


def test_two_sequences_that_read_the_same_pages():
    """Forked prompts: sequences whose cached text is one and the same, each with nodes of its own."""
    lens = [8, 8, 20]
    d = make(lens, [512 + n for n in lens], 16, 4, 64, seed=75)
    d["table"][1, :8] = d["table"][0, :8]
    d["table"][2, :8] = d["table"][0, :8]
    masks = masks_of(trees_of(lens, 76))
    out, lse, status = launch(d, masks)
    assert status == kda.OK
    check(d, masks, out, lse)
