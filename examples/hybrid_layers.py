"""A KDA layer and a full-attention layer of a hybrid model, prefilled and decoded on one GPU.

    python examples/hybrid_layers.py [--steps 8] [--hidden 1024]

Each layer is: residual norm (add_rms_norm), a projection (a torch product), the layer's own
kernels, an output projection.  The KDA layer keeps a state per sequence and head, the attention
layer a paged 8-bit cache that grows by a token a step.  The example prefills ragged prompts,
decodes token by token, and compares the decoded rows with one prefill of the full sequences.
Weights and inputs are random.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_chunk_gb300 as kda  # noqa: E402

D = kda.HEAD_DIM
SCALE = D ** -0.5


def _weight(g, rows, cols):
    return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).to(torch.bfloat16)


class KDALayer:
    """Gated delta rule over a [128, 128] state per sequence and head."""

    def __init__(self, hidden, heads, g):
        self.heads = heads
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        # q, k, v, gate, beta; the kernels want rows that start on 16 bytes, so beta is padded
        self.w_in = _weight(g, 4 * heads * D + -(-heads // 8) * 8, hidden)
        self.w_out = _weight(g, hidden, heads * D)
        self.A_log = torch.log(1 + 15 * torch.rand(heads, generator=g, device="cuda"))
        self.dt_bias = 0.1 * torch.randn(heads, D, generator=g, device="cuda")

    def forward(self, x, residual, state, batch):
        residual, y, _, _ = kda.add_rms_norm(x, residual, self.norm)
        p = y @ self.w_in.T
        H = self.heads
        q, k, v, gate = (p[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(4))
        beta = p[:, 4 * H * D:][:, :H]
        args = (self.A_log, self.dt_bias, -5.0, SCALE, state, batch["cu"])
        if batch["max_q"] == 1:      # one token a sequence: the recurrent form, on dense inputs
            out, state, _ = kda.recurrent_fwd(*(t.contiguous() for t in (q, k, v, gate, beta)), *args)
        else:
            out, state = kda.chunk_prefill_fwd(q, k, v, gate, beta, *args)
        return out.flatten(1) @ self.w_out.T, residual, state


class AttentionLayer:
    """Grouped-query attention with rotary positions over a paged e4m3 cache."""

    def __init__(self, hidden, heads, kv_heads, max_positions, page, pages, g):
        self.heads, self.kv_heads = heads, kv_heads
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.w_qkv = _weight(g, (heads + 2 * kv_heads) * D, hidden)
        self.w_out = _weight(g, hidden, heads * D)
        self.rope = kda.rope_table(max_positions, D)
        pool = torch.zeros(2, pages, kv_heads, page, D, dtype=torch.uint8, device="cuda")
        self.cache = [pool[0].view(torch.float8_e4m3fn), pool[1].view(torch.float8_e4m3fn),
                      torch.ones(pages, kv_heads, device="cuda"), torch.ones(pages, kv_heads, device="cuda")]
        self.status = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def forward(self, x, residual, batch):
        residual, y, _, _ = kda.add_rms_norm(x, residual, self.norm)
        p = (y @ self.w_qkv.T).unflatten(1, (-1, D))
        q, k, v = p.split((self.heads, self.kv_heads, self.kv_heads), 1)
        index = (batch["table"], batch["kv_lens"], batch["cu"])
        q = kda.rope_append(q, k, v, self.rope, *self.cache, *index, workspace=self.status)
        out, _ = kda.cached_attention(q, *self.cache, *index, SCALE, batch["max_q"],
                                      workspace=batch["workspace"])
        return out.flatten(1) @ self.w_out.T, residual


def run(lens, steps, hidden=1024, heads=8, kv_heads=2, page=16, seed=0):
    """Prefill of the prompts and `steps` decode steps, against one prefill of everything.
    Returns (decoded rows, the same rows of the one prefill), fp32 [steps, sequences, hidden]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, total = len(lens), [a + steps for a in lens]
    blocks = [-(-t // page) for t in total]
    table = torch.zeros(N, max(blocks), dtype=torch.int32)
    for n, b in enumerate(blocks):
        table[n, :b] = torch.arange(sum(blocks[:n]), sum(blocks[:n]) + b)
    table = table.cuda()
    kda_layer = KDALayer(hidden, 4, g)
    attn = AttentionLayer(hidden, heads, kv_heads, max(total), page, sum(blocks), g)
    tokens = [torch.randn(t, hidden, generator=g, device="cuda").to(torch.bfloat16) for t in total]

    def batch(counts, cached):
        cu = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
        return dict(cu=cu, kv_lens=torch.tensor(cached, dtype=torch.int32, device="cuda"), table=table,
                    max_q=max(counts),
                    workspace=kda.alloc_attention_workspace(N, heads, kv_heads, max(counts)))

    def step(rows, state, b):
        x = torch.cat(rows)
        y, residual, state = kda_layer.forward(x, torch.zeros_like(x), state, b)
        y, residual = attn.forward(y, residual, b)
        assert kda.last_device_status(b["workspace"]) == kda.OK
        return kda.add_rms_norm(y, residual, attn.norm)[0].float(), state

    state = torch.zeros(N, 4, D, D, device="cuda")
    _, state = step([t[:a] for t, a in zip(tokens, lens)], state, batch(lens, lens))
    decoded = []
    for i in range(steps):
        rows, state = step([t[a + i:a + i + 1] for t, a in zip(tokens, lens)], state,
                           batch([1] * N, [a + i + 1 for a in lens]))
        decoded.append(rows)
    whole, _ = step(tokens, torch.zeros_like(state), batch(total, total))
    ends = torch.tensor(total).cumsum(0)
    want = [torch.stack([whole[int(ends[n]) - steps + i] for n in range(N)]) for i in range(steps)]
    assert kda.last_device_status(attn.status) == kda.OK
    return torch.stack(decoded), torch.stack(want)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    got, want = run([100, 37, 256, 1], a.steps, a.hidden)
    off = float((got - want).norm() / want.norm())
    print(f"decoded {a.steps} steps of 4 sequences; relative difference to one prefill: {off:.2e}")
    return 0 if off < 0.02 else 1


if __name__ == "__main__":
    sys.exit(main())
