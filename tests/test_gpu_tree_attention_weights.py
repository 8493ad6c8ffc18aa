"""tree_attention where a few keys outweigh the others by far.

The bound of test_gpu_tree_attention with one term more.  A weight enters the product with the values to 2^-8 of
itself (in it already) and to a step of its own format at the tile's largest: for sequences of at most 32 rows
2^-18, as two e4m3 terms, else 2^-31, as f16, both of the largest p_j s_j with s_j the value's page's scale.  A key's
value is s_j e_j, so what that adds to an output is at most 2^-18 max(p_j s_j) sum |e_j| over the keys seen (no
tile's largest exceeds the row's).  Where one key has nearly all of the weight and nothing in a channel, that term is
larger than all the others, which shrink with the sum of p_j |v_j|.
"""
import pytest
import torch

import kda_gated_delta_chunk_gb300 as kda
import tree_ref as ref
from test_gpu_attention import D, FP8, SCALE, make
from test_gpu_tree_attention import launch, masks_of, trees_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_gated_delta_chunk_gb300 import build as kbuild
    kbuild.build()


def step_of(d, masks, n, q, l64, kf, vf, window, softcap):
    """2^-18 or 2^-31 of max p_j s_j, times sum |e_j|: [nodes, heads, D]."""
    H, hk, P = q.shape[1], d["k"].shape[1], d["k"].shape[2]
    G, kv = H // hk, d["kv_lens"][n]
    pg = d["table"][n][:-(-kv // P)].long()
    out = torch.zeros(*q.shape, dtype=torch.float64)
    for h in range(hk):
        k = (kf[pg, h].double() * d["ks"][pg, h].double()[:, None, None]).reshape(-1, D)
        e = vf[pg, h].double().reshape(-1, D).abs()
        s = d["vs"][pg, h].double().repeat_interleave(P)
        for i in range(len(masks[n])):
            keys = ref.seen_of(masks[n][i], len(masks[n]), kv, window)
            if not keys:
                continue
            x = q[i, h * G:(h + 1) * G].double() @ k[keys].T * SCALE
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            top = (torch.exp(x - l64[i, h * G:(h + 1) * G, None]) * s[keys]).amax(1)
            out[i, h * G:(h + 1) * G] = top[:, None] * e[keys].sum(0)
    return out * 2.0 ** (-18 if len(masks[n]) * G <= 32 else -31)


def check(d, masks, out, softcap=0.0, window=0):
    """The largest error as a part of the bound."""
    cu = d["cu"].tolist()
    kf, vf = d["k"].view(FP8).float(), d["v"].view(FP8).float()
    H, hk = d["q"].shape[1], d["k"].shape[1]
    worst = 0.0
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
        off = (out[a:b].cpu().double() - o64).abs()
        tol += step_of(d, masks, n, q, l64, kf, vf, window, softcap)
        worst = max(worst, float((off / tol.clamp(min=1e-30)).max()))
    return worst


@pytest.mark.parametrize("n,H,hk", [(8, 4, 1), (3, 16, 2), (16, 4, 1), (64, 8, 2)])
def test_one_key_with_nearly_all_of_the_weight(n, H, hk):
    """It has weight 1 to 2^21 times that of each other key, a ratio a row, and values in every second channel
    only; the others have 1 in all of them."""
    kv, page = 700, 64
    d = make([n], [kv], H, hk, page, seed=31)
    k, v = torch.zeros(d["k"].shape), torch.ones(d["v"].shape)
    first = int(d["table"][0, 0])
    k[first, :, 3, 0] = 16.0
    v[first, :, 3, 1::2] = 0.0
    d["k"], d["v"] = k.to(FP8).view(torch.uint8), v.to(FP8).view(torch.uint8)
    d["ks"][:] = d["vs"][:] = 1.0
    gap = torch.arange(n * H).view(n, H) / (n * H) * 21 * 0.6931
    d["q"][:] = 0
    d["q"][:, :, 0] = (gap / (16.0 * SCALE)).to(d["q"].dtype)
    masks = masks_of(trees_of([n], 32))
    out, lse, status = launch(d, masks)
    assert status == kda.OK
    assert check(d, masks, out) <= 1.0


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (50.0, 0), (0.0, 200)])
@pytest.mark.parametrize("lens,kv,H,hk,page", [
    ([8, 3, 1], [700, 129, 64], 4, 1, 16), ([2] * 6, [40, 130, 256, 300, 301, 800], 16, 2, 32), ([30, 9], [500, 222], 8, 2, 64)])
def test_queries_with_few_keys_that_count(lens, kv, H, hk, page, softcap, window):
    """Random caches whose pages' scales differ, with queries of 1 to 16 times the usual size."""
    d = make(lens, kv, H, hk, page, seed=33, spread=3)
    size = torch.exp2(torch.arange(sum(lens)) % 5).to(d["q"].dtype)
    d["q"] = d["q"] * size[:, None, None]
    masks = masks_of(trees_of(lens, 34))
    out, lse, status = launch(d, masks, softcap=softcap, window=window)
    assert status == kda.OK
    assert check(d, masks, out, softcap, window) <= 1.0
