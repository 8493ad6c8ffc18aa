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


def accept(values, scales, table, kv_len, parents, node):
    """One side of one layer's cache after a sequence's branch to `node` was accepted.  values: float64
    e4m3 values [pages, heads, slots, D], scales float64 [pages, heads]; both changed in place.  Returns
    the sequence's new length."""
    from layer_ref import e4m3_grid
    P, n = values.shape[2], len(parents)
    start, path = kv_len - n, branch(parents, node)
    was, old = values.clone(), scales.clone()
    at = lambda pos: (int(table[pos // P]), pos % P)  # noqa: E731
    for blk in range(start // P, (start + len(path) - 1) // P + 1 if path else 0):
        pg = int(table[blk])
        mine = [e for e in range(len(path)) if (start + e) // P == blk]
        if all(path[e] == e for e in mine):
            continue
        kept = max(0, start - blk * P)
        for h in range(values.shape[1]):
            froms = [at(start + path[e]) for e in mine]
            s = max([float(old[q, h]) for q, _ in froms] + ([float(old[pg, h])] if kept else []))
            scales[pg, h] = s
            if float(old[pg, h]) != s:
                values[pg, h, :kept] = e4m3_grid(was[pg, h, :kept] * (float(old[pg, h]) / s))
            for e, (q, slot) in zip(mine, froms):
                x = was[q, h, slot]
                values[pg, h, (start + e) % P] = x if float(old[q, h]) == s else e4m3_grid(x * (float(old[q, h]) / s))
    return start + len(path)


class Pool:
    """The pool's calls in plain Python."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = list(refs), [list(r) for r in table], list(lens), page

    def free(self, rows=None):
        for r in range(len(self.lens)) if rows is None else dict.fromkeys(rows):
            if rows is not None:
                self.lens[r] = 0
            for b in range(-(-self.lens[r] // self.page), len(self.table[r])):
                if self.table[r][b] >= 0:
                    self.refs[self.table[r][b]] -= 1
                self.table[r][b] = -1

    def take(self):
        if 0 not in self.refs:
            return -1
        pg = self.refs.index(0)
        self.refs[pg] = 1
        return pg

    def reserve(self, new):
        for r, a in enumerate(new):
            if a == 0:
                continue
            for b in range(self.lens[r] // self.page, -(-(self.lens[r] + a) // self.page)):
                if self.table[r][b] < 0:
                    self.table[r][b] = self.take()

    def fork(self, src, dst):
        """The rows share whole pages first, then the partial ones are given out."""
        fro, to = [-1] * len(src), [-1] * len(src)
        for s, d in zip(src, dst):
            whole = self.lens[s] // self.page
            self.table[d] = [self.table[s][b] if b < whole else -1 for b in range(len(self.table[d]))]
            for b in range(whole):
                self.refs[self.table[s][b]] += 1
            self.lens[d] = self.lens[s]
        for i, (s, d) in enumerate(zip(src, dst)):
            if self.lens[s] % self.page:
                whole = self.lens[s] // self.page
                fro[i], to[i] = self.table[s][whole], self.take()
                self.table[d][whole] = to[i]
        return fro, to


def recurrence(q, k, v, g, beta, A_log, dt_bias, lower_bound, scale, state, parents):
    """One sequence's nodes [n, heads, 128] (beta [n, heads]) from state [heads, 128, 128], all float64.
    Returns out, u, the state after each node, and magnitudes of the last three: the same sums over
    absolute values, which bound every term that enters."""
    n, H, _ = q.shape
    unit = lambda x: x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    qh, kh = unit(q) * scale, unit(k)
    a = torch.exp(lower_bound / (1 + torch.exp(-A_log.exp()[:, None] * (g + dt_bias))))
    b = 1 / (1 + torch.exp(-beta))
    out, us, after = [], [], []
    big_out, big_u, big_after = [], [], []
    for i in range(n):
        p = parents[i]
        s = (after[p] if p >= 0 else state) * a[i][:, :, None]
        u = b[i][:, None] * (v[i] - torch.einsum("hkv,hk->hv", s, kh[i]))
        s = s + kh[i][:, :, None] * u[:, None]
        m = (big_after[p] if p >= 0 else state.abs()) * a[i][:, :, None]
        mu = b[i][:, None] * (v[i].abs() + torch.einsum("hkv,hk->hv", m, kh[i].abs()))
        m = m + kh[i].abs()[:, :, None] * mu[:, None]
        out.append(torch.einsum("hkv,hk->hv", s, qh[i]))
        big_out.append(torch.einsum("hkv,hk->hv", m, qh[i].abs()))
        us.append(u)
        big_u.append(mu)
        after.append(s)
        big_after.append(m)
    return tuple(torch.stack(x) for x in (out, us, after, big_out, big_u, big_after))
