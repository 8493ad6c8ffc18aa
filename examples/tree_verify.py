"""Speculative steps with trees of drafts, over a KDA layer and a full-attention layer on one GPU.

    python examples/tree_verify.py [--steps 4] [--hidden 1024]

Prompts are prefilled and forked into samples (fork_pages, copy_pages; the KDA states are copied).  A
step then reserves pages, plans its trees (tree_plan), runs every drafted node through both layers
(tree_recurrent_fwd; rope_append at the nodes' positions and tree_attention), keeps one branch a
sequence (tree_commit, cache_accept) and gives back what is left over (free_pages).  The rows of the kept
branches are compared with one prefill of each sequence's kept tokens.  Drafts, the choice of a branch,
weights and inputs are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_chunk_gb300 as kda  # noqa: E402
from examples.hybrid_layers import SCALE, AttentionLayer, KDALayer  # noqa: E402

D = kda.HEAD_DIM


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(counts):
    return _i32([sum(counts[:i]) for i in range(len(counts) + 1)])


def _kda_verify(layer, x, residual, state, cu, parents, most, status):
    """The KDA layer's outputs at a step's nodes, and what its commit needs."""
    residual, y, _, _ = kda.add_rms_norm(x, residual, layer.norm)
    p = y @ layer.w_in.T
    H = layer.heads
    q, k, v, gate = (p[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(4))
    beta = p[:, 4 * H * D:][:, :H]
    out, u = kda.tree_recurrent_fwd(q, k, v, gate, beta, layer.A_log, layer.dt_bias, -5.0, SCALE, state, cu, parents,
                                    most, workspace=status)
    return out.flatten(1) @ layer.w_out.T, residual, (k, gate, u)


def _attention_verify(layer, x, residual, table, lens, cu, mask, positions, most, workspace):
    """The attention layer's outputs at a step's nodes, their keys and values appended to its cache."""
    residual, y, _, _ = kda.add_rms_norm(x, residual, layer.norm)
    p = (y @ layer.w_qkv.T).unflatten(1, (-1, D))
    q, k, v = p.split((layer.heads, layer.kv_heads, layer.kv_heads), 1)
    q = kda.rope_append(q, k, v, layer.rope, *layer.cache, table, lens, cu, positions=positions,
                        workspace=layer.status)
    out, _ = kda.tree_attention(q, *layer.cache, table, lens, cu, mask, SCALE, most, workspace=workspace)
    return out.flatten(1) @ layer.w_out.T, residual


def run(prompts, samples, steps, nodes=12, hidden=1024, heads=8, kv_heads=2, page=16, seed=0):
    """`samples` sequences of each prompt through `steps` steps of `nodes` drafts.  Returns (rows of the
    kept branches, the same rows of one prefill), fp32 [kept tokens, hidden]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pick = torch.Generator().manual_seed(seed)
    N, first = len(prompts) * samples, [n for n in prompts for _ in range(samples)]
    longest = max(prompts) + steps * nodes
    pages = N * (-(-longest // page) + 1)
    kda_layer = KDALayer(hidden, 4, g)
    attn = AttentionLayer(hidden, heads, kv_heads, longest, page, pages, g)
    token = lambda n: torch.randn(n, hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((N, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")

    def prefill(rows, state, attention, index):
        """Whole sequences through both layers; index: their table, lengths and cu_seqlens."""
        x = torch.cat(rows)
        batch = dict(cu=index[2], kv_lens=index[1], table=index[0], max_q=max(len(r) for r in rows),
                     workspace=kda.alloc_attention_workspace(len(rows), heads, kv_heads, max(len(r) for r in rows)))
        y, residual, state = kda_layer.forward(x, torch.zeros_like(x), state, batch)
        y, residual = attention.forward(y, residual, batch)
        return kda.add_rms_norm(y, residual, attention.norm)[0].float(), state

    # ---- prompts: the first sample of each is prefilled, the others are forked from it
    texts = [token(n) for n in prompts]
    lead = list(range(0, N, samples))
    kda.reserve_pages(refs, table, lens, _i32([n if i % samples == 0 else 0 for i, n in enumerate(first)]), page,
                      workspace=status)
    lens[lead] = _i32(prompts)
    _, made = prefill(texts, torch.zeros(len(prompts), 4, D, D, device="cuda"), attn,
                      (table[lead].contiguous(), lens[lead].contiguous(), _cu(prompts)))
    state = made.repeat_interleave(samples, 0)
    others = [i for i in range(N) if i % samples]
    if others:
        src, dst = _i32([i - i % samples for i in others]), _i32(others)
        kda.copy_pages(*attn.cache, *kda.fork_pages(refs, table, lens, src, dst, page, workspace=status),
                       workspace=status)
    kept = [[texts[i // samples]] for i in range(N)]
    rows = [[] for _ in range(N)]
    workspace = kda.alloc_attention_workspace(N, heads, kv_heads, nodes)
    # ---- steps
    for step in range(steps):
        counts = [nodes if (i + step) % 3 else max(1, nodes // 3) for i in range(N)]
        trees = [[-1] + [int(torch.randint(-1, i, (1,), generator=pick)) for i in range(1, n)] for n in counts]
        ends = [int(torch.randint(-1, n, (1,), generator=pick)) for n in counts]
        parents, accepted, cu = _i32([p for t in trees for p in t]), _i32(ends), _cu(counts)
        kda.reserve_pages(refs, table, lens, _i32(counts), page, workspace=status)
        drafted = lens + _i32(counts)
        mask, positions = kda.tree_plan(parents, cu, drafted, nodes, workspace=status)
        x = token(sum(counts))
        y, residual, tape = _kda_verify(kda_layer, x, torch.zeros_like(x), state, cu, parents, nodes, status)
        y, residual = _attention_verify(attn, y, residual, table, drafted, cu, mask, positions, nodes, workspace)
        out = kda.add_rms_norm(y, residual, attn.norm)[0].float()
        k, gate, u = tape
        state = kda.tree_commit(k, gate, kda_layer.A_log, kda_layer.dt_bias, -5.0, state, cu, parents, u, accepted, nodes,
                                final_state=state, workspace=status)
        lens = kda.cache_accept(*attn.cache, table, drafted, cu, parents, accepted, nodes, workspace=status)
        kda.free_pages(refs, table, lens, page, workspace=status)
        at = 0
        for i, (tree, end) in enumerate(zip(trees, ends)):
            branch = []
            while end >= 0:
                branch.insert(0, at + end)
                end = tree[end]
            kept[i].append(x[branch])
            rows[i].append(out[branch])
            at += len(tree)
    # ---- one prefill of every sequence's kept tokens, over a cache of its own
    whole = [torch.cat(t) for t in kept]
    total = [len(t) for t in whole]
    assert lens.tolist() == total
    assert int((refs > 0).sum()) == len(set(table[table >= 0].tolist()))
    cache = attn.cache
    attn.cache = [torch.zeros_like(c.view(torch.uint8)).view(c.dtype) if c.dtype == torch.float8_e4m3fn
                  else torch.ones_like(c) for c in cache]
    blocks = -(-max(total) // page)
    index = (torch.arange(N * blocks, dtype=torch.int32, device="cuda").view(N, blocks), _i32(total), _cu(total))
    want, _ = prefill(whole, torch.zeros(N, 4, D, D, device="cuda"), attn, index)
    attn.cache = cache
    starts = index[2].tolist()
    got = torch.cat([torch.cat(r) for r in rows])
    want = torch.cat([want[starts[i] + first[i]:starts[i + 1]] for i in range(N)])
    for ws in (status, attn.status, workspace):
        assert kda.last_device_status(ws) == kda.OK
    return got, want


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    got, want = run([100, 37, 256], 2, a.steps, hidden=a.hidden)
    off = float((got - want).norm() / want.norm())
    print(f"{got.shape[0]} kept tokens of 6 sequences in {a.steps} steps; relative difference to one prefill: {off:.2e}")
    return 0 if off < 0.02 else 1


if __name__ == "__main__":
    sys.exit(main())
