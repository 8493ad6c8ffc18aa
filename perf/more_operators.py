"""Timed cases of the operators for drafted trees: the tree's masks and positions, attention of its
nodes over the paged 8-bit cache, the KDA recurrence along its branches, what acceptance does to
the cache, and the cache's pages (freeing, forking, copying, reserving).

A drafted tree is at most 64 new tokens of a sequence; ``parents[t]`` is the index, among the
sequence's new tokens, of the one that token t follows, or -1 for one that follows the cached text.

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges; ``prepare`` makes a
case's inputs on the GPU from a seed, ``run`` makes one pass through the operator.  With ``own``
false the pass is made of elementary torch operations in 32 bits; with ``own`` true it is the
calls of this package.  ``exact`` restates each operator in 64 bits.
"""
import math

import torch

own = False

D = 128            # head dim
FP8 = torch.float8_e4m3fn
SCALE = D ** -0.5
LOWER_BOUND = -5.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest verify of a tree: 8 nodes of one sequence behind a short prompt
        dict(name="attend_tree_1x8", op="attend", seqs=1, n_lo=8, n_hi=8, tree="wide", kv_lo=1000,
             kv_hi=1000, heads=16, kv_heads=4, page=64, window=0, softcap=0.0),
        # a serving batch that verifies 16 nodes a sequence over ragged contexts, small pages
        dict(name="attend_tree_16x16", op="attend", seqs=16, n_lo=16, n_hi=16, tree="wide",
             kv_lo=1000, kv_hi=16384, heads=32, kv_heads=8, page=16, window=0, softcap=0.0),
        # large trees over long contexts
        dict(name="attend_tree_4x64_at_65536", op="attend", seqs=4, n_lo=64, n_hi=64, tree="deep",
             kv_lo=65536, kv_hi=65536, heads=32, kv_heads=4, page=128, window=0, softcap=0.0),
        # trees of very unequal size, a sliding window and capped scores
        dict(name="attend_tree_64_ragged_window", op="attend", seqs=64, n_lo=1, n_hi=31,
             tree="deep", kv_lo=64, kv_hi=16384, heads=16, kv_heads=2, page=32, window=2048,
             softcap=30.0),
        # what a step computes of its trees before the layers run: one tree, and a full batch
        dict(name="plan_1x8", op="plan", seqs=1, n_lo=8, n_hi=8, tree="wide", kv_lo=1000,
             kv_hi=1000),
        dict(name="plan_512_ragged", op="plan", seqs=512, n_lo=1, n_hi=64, tree="deep", kv_lo=64,
             kv_hi=16384),
        # a KDA layer's verify and, with the accepted node known, its state's step: one sequence
        # over a bf16 state, and a serving batch of 64 over fp32 states
        dict(name="recur_tree_1x8_h16", op="recur", seqs=1, n_lo=8, n_hi=8, tree="wide", heads=16,
             state="bf16"),
        dict(name="recur_tree_64x32_h32", op="recur", seqs=64, n_lo=32, n_hi=32, tree="deep",
             heads=32, state="f32"),
        # the accepted branch moved together in one layer's cache: one sequence, a serving batch
        dict(name="accept_1x8", op="accept", seqs=1, n_lo=8, n_hi=8, tree="deep", kv_lo=1000,
             kv_hi=1000, kv_heads=4, page=64),
        dict(name="accept_128_ragged", op="accept", seqs=128, n_lo=3, n_hi=64, tree="deep",
             kv_lo=64, kv_hi=16384, kv_heads=8, page=16),
        # parallel sampling: 7 more samples of one prompt; and 16 prompts of 4 samples each over
        # a pool of 24000 pages
        dict(name="pages_fork_1x7", op="pages", prompts=1, samples=7, kv_lo=1000, kv_hi=1000,
             kv_heads=2, page=16, spare=1000, new=8),
        dict(name="pages_fork_16x4", op="pages", prompts=16, samples=4, kv_lo=4097, kv_hi=65535,
             kv_heads=2, page=64, spare=16000, new=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "recur", "recur", "plan", "accept", "pages"])
    tree = rng.choice(["wide", "deep", "chain"])
    if op == "pages":
        prompts, samples = _log(rng, 1, 16), _log(rng, 1, 9)
        kv_hi = _log(rng, 65, 65535)
        return dict(op=op, prompts=prompts, samples=samples, kv_lo=max(1, kv_hi // 9), kv_hi=kv_hi,
                    kv_heads=rng.choice([1, 2, 4]), page=rng.choice([16, 32, 64]),
                    spare=_log(rng, 10, 16000), new=_log(rng, 1, 64))
    seqs = _log(rng, 1, 64)
    n_hi = _log(rng, 1, 64)
    n_lo = max(1, n_hi // rng.choice([1, 1, 3, 20]))
    if op == "plan":
        seqs = _log(rng, 1, 512)
    kv_hi = _log(rng, 80, min(65536, 262144 // seqs)) | 1
    base = dict(op=op, seqs=seqs, n_lo=n_lo, n_hi=n_hi, tree=tree)
    if op == "recur":
        heads = rng.choice([1, 3, 8, 16, 32])
        base.update(seqs=min(seqs, max(1, 65536 // (heads * n_hi))), heads=heads,
                    state=rng.choice(["f32", "bf16"]))
        return base
    base.update(kv_lo=max(n_hi, kv_hi // 7), kv_hi=max(n_hi, kv_hi))
    if op == "plan":
        return base
    heads, kv_heads = rng.choice([(8, 8), (8, 2), (16, 4), (16, 2), (32, 8), (32, 4), (16, 1)])
    base.update(kv_heads=kv_heads, page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        window, softcap = rng.choice([(0, 0.0), (0, 0.0), (999, 0.0), (0, 50.0)])
        base.update(heads=heads, window=window, softcap=softcap)
    return base


def _spread(n, lo, hi, step):
    """n whole numbers, evenly spread over the logarithm of [lo, hi], in a mixed-up order
    (multiples of an irrational step); the first is hi."""
    out = []
    for i in range(n):
        u = 1.0 - (i * step) % 1.0
        out.append(min(hi, max(lo, int(round(lo * (hi / lo) ** u)))))
    return out


def _lengths(case):
    """Nodes and cache length (nodes included) of each sequence."""
    n = case["seqs"]
    q = _spread(n, case["n_lo"], case["n_hi"], 0.6180339887)
    if "kv_lo" not in case:
        return q, None
    kv = _spread(n, case["kv_lo"], case["kv_hi"], 0.7548776662)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _parents(case, shift=0.0):
    """One list of parents per sequence.  "wide": a node follows any earlier node or the cached
    text; "deep": every second one follows the node before it; "chain": all do.  Another shift
    gives other trees."""
    out = []
    for n, t in enumerate(_lengths(case)[0]):
        p = []
        for i in range(t):
            u = ((i + 1) * 0.6180339887 + n * 0.7548776662 + shift) % 1.0
            if case["tree"] == "chain" or (case["tree"] == "deep" and (i + n) % 2):
                p.append(i - 1)
            else:
                p.append(int(u * (i + 1)) - 1)
        out.append(p)
    return out


def _depths(parents):
    """Ancestors of each node."""
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def work(case):
    op = case["op"]
    if op == "pages":
        m = case["prompts"] * case["samples"]
        kv = _spread(case["prompts"], case["kv_lo"], case["kv_hi"], 0.6180339887)
        blocks = case["samples"] * sum(-(-b // case["page"]) for b in kv)
        copies = case["samples"] * sum(b % case["page"] != 0 for b in kv)
        return {"bytes": 4 * 8 * blocks + copies * case["kv_heads"] * (4 * case["page"] * D + 16) + 16 * m,
                "flops": 0}
    q, kv = _lengths(case)
    t, deep = sum(q), [_depths(p) for p in _parents(case)]
    pairs = sum(sum(d) + len(d) for d in deep)           # (node, ancestor or itself)
    if op == "plan":
        return {"bytes": 4 * t + 8 * len(q) + 12 * t, "flops": t}
    if op == "recur":
        h, s = case["heads"], 4 if case["state"] == "f32" else 2
        return {"bytes": h * (2 * case["seqs"] * D * D * s + t * (5 * 2 * D + 2)),
                "flops": h * (4 * t * D * D + 8 * D * pairs + 4 * case["seqs"] * D * D)}
    if op == "accept":
        hk = case["kv_heads"]
        path = sum(d[-1] + 1 for d in deep)
        return {"bytes": path * hk * 4 * D + case["seqs"] * (hk * 16 + 16) + 4 * t, "flops": 0}
    h, hk, w = case["heads"], case["kv_heads"], case["window"]
    keys = sum(b if not w else min(b, w + a) for a, b in zip(q, kv))
    pages = sum(-(-b // case["page"]) for b in kv)
    seen = 0
    for a, b, d in zip(q, kv, deep):
        seen += sum((b - a if not w else min(b - a, w - 1 - x)) + x + 1 for x in d)
    return {"bytes": 2 * keys * hk * D + 8 * pages * hk + t * (h * (4 * D + 4) + 8),
            "flops": 4 * D * h * seen}


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """The least power of two 2^e with amax <= 448 * 2^e, at least 2^-64."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-64)
    e = torch.where(amax > 0, e, torch.full_like(e, -64))
    return torch.ldexp(torch.ones_like(amax), e)


def _cache(pages, hk, page, g):
    """A cache of normal keys or values whose pages differ in size: [pages, kv heads, page, 128]
    e4m3, scale [pages, kv heads]."""
    out = torch.empty((pages, hk, page, D), dtype=FP8, device="cuda")
    scale = torch.empty((pages, hk), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (hk * page * D))
    for a in range(0, pages, step):
        b = min(step, pages - a)
        x = torch.randn((b, hk, page, D), generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-1, 2, (b, hk, 1, 1), generator=g, device="cuda").float())
        s = _pow2_scale(x.abs().amax((2, 3)))
        out[a:a + b] = (x / s[:, :, None, None]).to(FP8)
        scale[a:a + b] = s
    return out, scale


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_pages(case, g, st):
    """`prompts` sequences with their pages, `prompts * samples` rows for their samples, a pool."""
    n, m, page, hk = case["prompts"], case["samples"], case["page"], case["kv_heads"]
    kv = _spread(n, case["kv_lo"], case["kv_hi"], 0.6180339887)
    blocks = [-(-b // page) for b in kv]
    most = max(-(-(b + case["new"]) // page) for b in kv)
    pages = sum(blocks) + case["spare"] + n * (m + 1) * (-(-case["new"] // page) + 1)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    rows = n * (m + 1)
    table = torch.full((rows, most), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for i, b in enumerate(blocks):
        table[i * (m + 1), :b] = perm[at:at + b]
        refs[perm[at:at + b].long()] = 1
        at += b
    lens = torch.zeros(rows, dtype=torch.int32)
    lens[::m + 1] = torch.tensor(kv, dtype=torch.int32)
    st["refs"], st["block_table"], st["kv_lens"] = refs.cuda(), table.cuda(), lens.cuda()
    st["dst"] = _i32([i for i in range(rows) if i % (m + 1)])
    st["src"] = st["dst"] // (m + 1) * (m + 1)
    st["new"] = torch.full((rows,), case["new"], dtype=torch.int32, device="cuda")
    st["k_cache"], st["k_scale"] = _cache(pages, hk, page, g)
    st["v_cache"], st["v_scale"] = _cache(pages, hk, page, g)
    if own:
        st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    st = dict(case=dict(case))
    if case["op"] == "pages":
        return _prepare_pages(case, g, st)
    q, kv = _lengths(case)
    n, t = case["seqs"], sum(q)
    cu = [0]
    for a in q:
        cu.append(cu[-1] + a)
    st["cu_seqlens"], st["max_q_len"] = _i32(cu), max(q)
    trees = _parents(case)
    st["parents"] = _i32([p for tree in trees for p in tree])
    if case["op"] in ("recur", "accept"):
        # the node that verification ends at, -1 where it accepts none
        u = torch.rand(n, generator=g, device="cuda")
        st["accepted"] = ((u * (_i32(q) + 1)).int() - 1).clamp(max=_i32(q) - 1)
    if case["op"] == "recur":
        h = case["heads"]
        # one fused projection's output: q, k, v, g and beta are column ranges of it
        p = rand(t, 4 * h * D + -(-h // 8) * 8).to(torch.bfloat16)
        st["q"], st["k"], st["v"], st["g"] = (p[:, i * h * D:(i + 1) * h * D].view(t, h, D)
                                              for i in range(4))
        st["beta"] = p[:, 4 * h * D:][:, :h]
        st["A_log"] = torch.log(1 + 15 * torch.rand(h, generator=g, device="cuda"))
        st["dt_bias"] = 0.1 * rand(h, D)
        st["state"] = (0.1 * rand(n, h, D, D)).to(
            torch.float32 if case["state"] == "f32" else torch.bfloat16)
        if own:
            st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    st["kv_lens"] = _i32(kv)
    if case["op"] == "plan":
        trees = _parents(case, float(torch.rand((), generator=g, device="cuda")))
        st["parents"] = _i32([p for tree in trees for p in tree])
        st["kv_lens"] += torch.randint(0, 1000, (n,), generator=g, device="cuda").int()
        if own:
            st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    hk, page = case["kv_heads"], case["page"]
    blocks = [-(-b // page) for b in kv]
    pages = sum(blocks) + 3                    # a few that no sequence owns
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros((n, max(blocks)), dtype=torch.int32)
    at = 0
    for i, b in enumerate(blocks):
        table[i, :b] = perm[at:at + b]
        at += b
    st["block_table"] = table.cuda()
    st["k_cache"], st["k_scale"] = _cache(pages, hk, page, g)
    st["v_cache"], st["v_scale"] = _cache(pages, hk, page, g)
    if case["op"] == "accept":
        if own:
            st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    h = case["heads"]
    st["q"] = rand(t, h, D).to(torch.bfloat16)
    masks = []
    for tree in trees:
        bits = []
        for i, p in enumerate(tree):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        masks += [b - (1 << 64) if b >> 63 else b for b in bits]
    st["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    # slots of the last pages that no token has filled hold whatever was there: NaN
    seq = torch.arange(n, device="cuda")
    last = st["block_table"][seq, (st["kv_lens"].long() - 1) // page].long()
    free = torch.arange(page, device="cuda") > ((st["kv_lens"] - 1) % page)[:, None]
    for c in (st["k_cache"], st["v_cache"]):
        raw = c.view(torch.uint8)
        raw[last] = torch.where(free[:, None, :, None], torch.full_like(raw[last], 0x7F), raw[last])
    if own:
        import kda_gated_delta_chunk_gb300 as kda
        st["workspace"] = kda.alloc_attention_workspace(n, h, hk, max(q))
    return st


# ------------------------------------------------------------------ one pass
def _to_fp8(x):
    return x.clamp(-448.0, 448.0).to(FP8)      # NaN stays NaN


def _tokens(st):
    """Sequence of every new token, and its index among that sequence's."""
    cu = st["cu_seqlens"].long()
    i = torch.arange(st["parents"].numel(), device="cuda")
    seq = torch.searchsorted(cu, i, right=True) - 1
    return seq, i - cu[seq]


def _plan_plain(st):
    seq, i = _tokens(st)
    cu, kv = st["cu_seqlens"].long(), st["kv_lens"].long()
    parents = st["parents"].long()
    one = torch.ones_like(i)
    mask, depth, at = one << i, torch.zeros_like(i), parents
    for _ in range(st["max_q_len"] - 1):
        up = at >= 0
        j = at.clamp(min=0)
        mask = torch.where(up, mask | (one << j), mask)
        depth = depth + up
        at = torch.where(up, parents[cu[seq] + j], at)
    start = kv - (cu[1:] - cu[:-1])
    return dict(mask=mask, positions=(start[seq] + depth).int())


def _attend_plain(st):
    c = st["case"]
    n, h, hk, page = c["seqs"], c["heads"], c["kv_heads"], c["page"]
    kv, cu = st["kv_lens"].long(), st["cu_seqlens"].long()
    seq, i = _tokens(st)
    m = st["max_q_len"]
    bt = st["block_table"].long()
    L = bt.shape[1] * page
    # queries padded to the largest tree: [n, kv heads, group * m, 128]
    q = torch.zeros((n, m, h, D), device="cuda")
    q[seq, i] = st["q"].float()
    q = q.view(n, m, hk, h // hk, D).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, D)
    mask = torch.zeros((n, m), dtype=torch.int64, device="cuda")
    mask[seq, i] = st["mask"]
    bits = (mask[:, :, None] >> torch.arange(64, device="cuda")) & 1          # [n, m, 64]
    j = torch.arange(L, device="cuda")
    start = kv - (cu[1:] - cu[:-1])
    new = j - start[:, None]                                                  # [n, L]
    filled = (j < kv[:, None])
    see = torch.gather(bits, 2, new.clamp(0, 63)[:, None].expand(n, m, L)) > 0
    see = torch.where((new < 0)[:, None], True, see & filled[:, None])
    if c["window"]:
        first = start[:, None] + bits.sum(2) - c["window"]                    # first position seen
        see &= j >= first[:, :, None]
    k = (st["k_cache"][bt].float() * st["k_scale"][bt][..., None, None]).transpose(1, 2)
    s = torch.matmul(q, k.reshape(n, hk, L, D).transpose(2, 3)).mul_(SCALE)
    del k
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    s = s.view(n, hk, h // hk, m, L).masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top.clamp(min=-3e38)).exp_()
    total = s.sum(-1, keepdim=True)
    v = (st["v_cache"][bt].float() * st["v_scale"][bt][..., None, None]).transpose(1, 2)
    v = torch.where(filled[:, None, :, None], v.reshape(n, hk, L, D), 0.0)
    o = torch.matmul(s.view(n, hk, -1, L), v).view(n, hk, h // hk, m, D)
    o = o / total.clamp(min=1e-38)
    lse = (top + total.log())[..., 0]
    out = o.permute(0, 3, 1, 2, 4).reshape(n, m, h, D)[seq, i].to(torch.bfloat16)
    return dict(out=out, lse=lse.permute(0, 3, 1, 2).reshape(n, m, h)[seq, i])


def _recur_plain(st):
    c = st["case"]
    n, h, m = c["seqs"], c["heads"], st["max_q_len"]
    seq, i = _tokens(st)

    def padded(x):
        y = torch.zeros((n, m) + x.shape[1:], device="cuda")
        y[seq, i] = x.float()
        return y

    unit = lambda x: x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    q, k, v = unit(padded(st["q"])) * SCALE, unit(padded(st["k"])), padded(st["v"])
    gate = st["A_log"].exp()[:, None] * (padded(st["g"]) + st["dt_bias"])
    decay = torch.exp(LOWER_BOUND * torch.sigmoid(gate))
    beta = torch.sigmoid(padded(st["beta"]))
    parents = torch.full((n, m), -1, dtype=torch.long, device="cuda")
    parents[seq, i] = st["parents"].long()
    rows = torch.arange(n, device="cuda")
    # states[:, 0]: before the tree; states[:, 1 + j]: after node j
    states = torch.empty((n, m + 1, h, D, D), device="cuda")
    states[:, 0] = st["state"].float()
    out = torch.empty((n, m, h, D), device="cuda")
    for j in range(m):
        s = states[rows, 1 + parents[:, j]] * decay[:, j, :, :, None]
        u = beta[:, j, :, None] * (v[:, j] - torch.matmul(k[:, j, :, None], s)[:, :, 0])
        s += k[:, j, :, :, None] * u[:, :, None]
        out[:, j] = torch.matmul(q[:, j, :, None], s)[:, :, 0]
        states[:, 1 + j] = s
    final = states[rows, 1 + st["accepted"].long()].to(st["state"].dtype)
    return dict(out=out[seq, i].to(torch.bfloat16), final_state=final)


def _path(st):
    """[n, m]: the accepted branch's nodes from the first on, -1 past its end; its length [n]."""
    cu, parents = st["cu_seqlens"].long(), st["parents"].long()
    n, m = st["case"]["seqs"], st["max_q_len"]
    at = st["accepted"].long()
    back = torch.full((n, m), -1, dtype=torch.long, device="cuda")
    for e in range(m):
        back[:, e] = at
        at = torch.where(at >= 0, parents[cu[:-1] + at.clamp(min=0)], at)
    length = (back >= 0).sum(1)
    e = torch.arange(m, device="cuda")
    path = back.gather(1, (length[:, None] - 1 - e).clamp(min=0))
    return torch.where(e < length[:, None], path, -1), length


def _accept_plain(st):
    page = st["case"]["page"]
    path, length = _path(st)
    kv, cu = st["kv_lens"].long(), st["cu_seqlens"].long()
    bt = st["block_table"].long()
    start = kv - (cu[1:] - cu[:-1])
    seq, e = torch.nonzero(path >= 0, as_tuple=True)
    to, src = start[seq] + e, start[seq] + path[seq, e]
    to_page, src_page = bt[seq, to // page], bt[seq, src // page]
    # the page of each sequence that holds cached tokens and takes accepted ones
    tail = bt.gather(1, (start // page).clamp(max=bt.shape[1] - 1)[:, None])[:, 0]
    part = (start % page > 0) & (length > 0)
    kept = (torch.arange(page, device="cuda") < (start % page)[:, None]) & part[:, None]
    for cache, scale in ((st["k_cache"], st["k_scale"]), (st["v_cache"], st["v_scale"])):
        raw = cache.view(torch.uint8)
        x = raw[src_page, :, src % page].view(FP8).float()
        was = scale[src_page]
        old = scale[tail]
        fresh = torch.zeros_like(scale).index_reduce_(0, to_page, was, "amax")
        fresh = fresh.index_reduce_(0, tail[part], old[part], "amax")
        scale[to_page] = fresh[to_page]
        ratio = (old / scale[tail])[:, :, None, None]
        again = _to_fp8(raw[tail].view(FP8).float() * ratio).view(torch.uint8)
        some = part.nonzero()[:, 0]
        raw[tail[some]] = torch.where(kept[:, None, :, None] & (ratio != 1.0), again,
                                      raw[tail])[some]
        raw[to_page, :, to % page] = _to_fp8(x * (was / scale[to_page])[:, :, None]).view(torch.uint8)
    return dict(lens=(start + length).int(), k_cache=st["k_cache"], v_cache=st["v_cache"],
                k_scale=st["k_scale"], v_scale=st["v_scale"])


def _pages_plain(st):
    page = st["case"]["page"]
    refs, bt, lens = st["refs"], st["block_table"], st["kv_lens"]
    src, dst = st["src"].long(), st["dst"].long()
    blocks = torch.arange(bt.shape[1], device="cuda")
    # the samples' rows end: their pages lose a reference
    gone = bt[dst]
    refs.index_add_(0, gone[gone >= 0].long(), torch.full_like(gone[gone >= 0], -1))
    bt[dst] = -1
    # each becomes a copy of its prompt's row: whole pages shared, the partial one a page of its own
    have = lens[src].long()
    whole, part = have // page, have % page > 0
    row = torch.where(blocks < whole[:, None], bt[src], -1)
    shared = row[row >= 0].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    free = torch.nonzero(refs == 0)[:, 0].int()
    to = torch.full_like(st["dst"], -1)
    to[part] = free[:int(part.sum())]
    refs[to[part].long()] = 1
    fro = torch.where(part, bt[src, whole.clamp(max=bt.shape[1] - 1)], -1)
    row = torch.where(part[:, None] & (blocks == whole[:, None]), to[:, None], row)
    bt[dst] = row
    lens[dst] = have.int()
    a, b = fro[part].long(), to[part].long()
    for x in (st["k_cache"].view(torch.uint8), st["v_cache"].view(torch.uint8), st["k_scale"],
              st["v_scale"]):
        x[b] = x[a]
    # pages for the next tokens of every row
    need = (lens.long() + st["new"].long() + page - 1) // page
    want = (blocks >= (lens.long() // page)[:, None]) & (blocks < need[:, None]) & (bt < 0)
    free = torch.nonzero(refs == 0)[:, 0].int()[:int(want.sum())]
    bt[want] = free
    refs[free.long()] = 1
    return dict(from_pages=fro, to_pages=to, refs=refs, block_table=bt, kv_lens=lens,
                k_cache=st["k_cache"], v_cache=st["v_cache"], k_scale=st["k_scale"],
                v_scale=st["v_scale"])


def run(st):
    c = st["case"]
    if not own:
        return {"plan": _plan_plain, "attend": _attend_plain, "recur": _recur_plain,
                "accept": _accept_plain, "pages": _pages_plain}[c["op"]](st)
    import kda_gated_delta_chunk_gb300 as kda
    if c["op"] == "plan":
        mask, positions = kda.tree_plan(st["parents"], st["cu_seqlens"], st["kv_lens"],
                                        st["max_q_len"], workspace=st["workspace"])
        return dict(mask=mask, positions=positions)
    if c["op"] == "attend":
        out, lse = kda.tree_attention(st["q"], st["k_cache"], st["v_cache"], st["k_scale"],
                                      st["v_scale"], st["block_table"], st["kv_lens"],
                                      st["cu_seqlens"], st["mask"], SCALE, st["max_q_len"],
                                      softcap=c["softcap"], window=c["window"], lse=True,
                                      workspace=st["workspace"])
        return dict(out=out, lse=lse)
    if c["op"] == "recur":
        out, u = kda.tree_recurrent_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["A_log"],
                                        st["dt_bias"], LOWER_BOUND, SCALE, st["state"],
                                        st["cu_seqlens"], st["parents"], st["max_q_len"],
                                        workspace=st["workspace"])
        final = kda.tree_commit(st["k"], st["g"], st["A_log"], st["dt_bias"], LOWER_BOUND,
                                st["state"], st["cu_seqlens"], st["parents"], u, st["accepted"],
                                st["max_q_len"], workspace=st["workspace"])
        return dict(out=out, final_state=final)
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if c["op"] == "accept":
        lens = kda.cache_accept(*cache, st["block_table"], st["kv_lens"], st["cu_seqlens"],
                                st["parents"], st["accepted"], st["max_q_len"],
                                workspace=st["workspace"])
        return dict(lens=lens, k_cache=cache[0], v_cache=cache[1], k_scale=cache[2], v_scale=cache[3])
    pool = (st["refs"], st["block_table"], st["kv_lens"])
    kda.free_pages(*pool, c["page"], rows=st["dst"], workspace=st["workspace"])
    fro, to = kda.fork_pages(*pool, st["src"], st["dst"], c["page"], workspace=st["workspace"])
    kda.copy_pages(*cache, fro, to, workspace=st["workspace"])
    kda.reserve_pages(*pool, st["new"], c["page"], workspace=st["workspace"])
    return dict(from_pages=fro, to_pages=to, refs=pool[0], block_table=pool[1], kv_lens=pool[2],
                k_cache=cache[0], v_cache=cache[1], k_scale=cache[2], v_scale=cache[3])


# ------------------------------------------------------------------ in 64 bits
def _grid_e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), as float64."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    if case["op"] in ("plan", "pages"):
        return None                            # whole numbers and copies
    st = prepare(case, seed)
    return {"attend": _exact_attend, "recur": _exact_recur, "accept": _exact_accept}[case["op"]](case, st)


def _branch(tree, node):
    """The nodes from the cached text to `node`."""
    out = []
    while node >= 0:
        out.append(node)
        node = tree[node]
    return out[::-1]


def _exact_attend(case, st):
    q_lens, kv_lens = _lengths(case)
    h, hk, page, w = case["heads"], case["kv_heads"], case["page"], case["window"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for n, (a, b, tree) in enumerate(zip(q_lens, kv_lens, _parents(case))):
        pg = st["block_table"][n, :-(-b // page)].long()
        hide = torch.ones((a, b), dtype=torch.bool)
        for i in range(a):
            seen = list(range(b - a)) + [b - a + x for x in _branch(tree, i)]
            hide[i, seen[-w:]] = False
        hide = hide.cuda()
        for x in range(hk):
            k = st["k_cache"][pg, x].double() * st["k_scale"][pg, x].double()[:, None, None]
            v = st["v_cache"][pg, x].double() * st["v_scale"][pg, x].double()[:, None, None]
            k, v = k.reshape(-1, D)[:b], v.reshape(-1, D)[:b]
            for y in range(x * (h // hk), (x + 1) * (h // hk)):
                s = st["q"][at:at + a, y].double() @ k.T / math.sqrt(D)
                if case["softcap"]:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                s[hide] = -math.inf
                out[at:at + a, y] = torch.softmax(s, 1) @ v
                lse[at:at + a, y] = torch.logsumexp(s, 1)
        at += a
    return dict(out=out, lse=lse)


def _exact_recur(case, st):
    q, k, v, g, beta = (st[x].double() for x in ("q", "k", "v", "g", "beta"))
    k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6) / math.sqrt(D)
    x = torch.exp(st["A_log"].double())[:, None] * (g + st["dt_bias"].double())
    decay = torch.exp(LOWER_BOUND / (1.0 + torch.exp(-x)))
    beta = 1.0 / (1.0 + torch.exp(-beta))
    out, final = torch.empty_like(q), st["state"].double()
    ends, at = st["accepted"].tolist(), 0
    for n, tree in enumerate(_parents(case)):
        after = []
        before = st["state"][n].double()
        for i, p in enumerate(tree):
            t = at + i
            s = decay[t][:, :, None] * (after[p] if p >= 0 else before)
            u = beta[t][:, None] * (v[t] - (s * k[t][:, :, None]).sum(1))
            s = s + k[t][:, :, None] * u[:, None, :]
            out[t] = (s * q[t][:, :, None]).sum(1)
            after.append(s)
        if ends[n] >= 0:
            final[n] = after[ends[n]]
        at += len(tree)
    return dict(out=out, final_state=final)


def _exact_accept(case, st):
    page = case["page"]
    table, ends = st["block_table"].cpu().long(), st["accepted"].tolist()
    res = {}
    for name in ("k", "v"):
        cache, scale = st[name + "_cache"].double(), st[name + "_scale"].double()
        for n, (a, b, tree) in enumerate(zip(*_lengths(case), _parents(case))):
            path, start = _branch(tree, ends[n]), b - a
            old_s = {int(p): scale[p].clone() for p in table[n, start // page:-(-b // page)]}
            old = {p: cache[p].clone() for p in old_s}
            where = [(int(table[n, (start + x) // page]), (start + x) % page) for x in path]
            for blk in range(start // page, (start + len(path) - 1) // page + 1 if path else 0):
                lo, hi = max(start, blk * page), min(start + len(path), (blk + 1) * page)
                pg, kept = int(table[n, blk]), lo - blk * page
                parts = [old_s[pg]] if kept else []
                parts += [old_s[where[i - start][0]] for i in range(lo, hi)]
                s = torch.stack(parts).amax(0)
                scale[pg] = s
                cache[pg, :, :kept] = _grid_e4m3(old[pg][:, :kept] * (old_s[pg] / s)[:, None, None])
                for i in range(lo, hi):
                    sp, slot = where[i - start]
                    cache[pg, :, i - blk * page] = _grid_e4m3(old[sp][:, slot] * (old_s[sp] / s)[:, None])
        res[name + "_cache"], res[name + "_scale"] = cache, scale
    return dict(lens=None, k_cache=res["k_cache"], v_cache=res["v_cache"], k_scale=res["k_scale"],
                v_scale=res["v_scale"])
