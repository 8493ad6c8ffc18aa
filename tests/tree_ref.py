"""The operators on drafted trees restated in 64 bits on the host, from their definitions.

Plain loops over sequences, heads and nodes; shares nothing with the library or with
perf/more_operators.py.
"""
import math

import torch

D = 128
F64 = torch.float64


def random_tree(n, gen, kind="any"):
    """Parents of n nodes: "any" earlier node or none, a "chain", or all "roots"."""
    out = []
    for i in range(n):
        if kind == "chain":
            out.append(i - 1)
        elif kind == "roots":
            out.append(-1)
        else:
            out.append(int(torch.randint(-1, i, (1,), generator=gen)) if i else -1)
    return out


def branch(parents, i):
    """The nodes from the cached text to node i."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


def mask_of(parents, i):
    m = sum(1 << j for j in branch(parents, i))
    return m - (1 << 64) if m >> 63 else m


def seen_of(mask, n, kv_len, window=0):
    """Cache positions that a node with this mask sees, of a sequence with n nodes."""
    start = kv_len - n
    keys = list(range(start)) + [start + j for j in range(n) if (mask >> j) & 1]
    return keys[-window:] if window else keys


def attention(q, masks, kc, vc, ks, vs, table, kv_len, scale, softcap=0.0, window=0):
    """q [n, heads, 128] of one sequence's nodes over its cache; out, lse, and sum_j p_j |v_j|."""
    n, H, _ = q.shape
    hk, P = kc.shape[1], kc.shape[2]
    G = H // hk
    out = torch.zeros(n, H, D, dtype=F64)
    big = torch.zeros(n, H, D, dtype=F64)
    lse = torch.full((n, H), -math.inf, dtype=F64)
    pg = table[:(kv_len + P - 1) // P].long()
    for g in range(hk):
        k = (kc[pg, g].to(F64) * ks[pg, g].to(F64)[:, None, None]).reshape(-1, D)
        v = (vc[pg, g].to(F64) * vs[pg, g].to(F64)[:, None, None]).reshape(-1, D)
        for i in range(n):
            keys = seen_of(masks[i], n, kv_len, window)
            if not keys:
                continue
            s = q[i, g * G:(g + 1) * G].to(F64) @ k[keys].T * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            p = torch.softmax(s, 1)
            lse[i, g * G:(g + 1) * G] = torch.logsumexp(s, 1)
            out[i, g * G:(g + 1) * G] = p @ v[keys]
            big[i, g * G:(g + 1) * G] = p @ v[keys].abs()
    return out, lse, big
