"""The full-attention layer's operators restated in 64 bits on the host, from their definitions.

Shares nothing with the library or with perf/operators.py: plain loops over sequences, heads
and tokens on float64 tensors.
"""
import math

import torch

D = 128
F64 = torch.float64


def e4m3_grid(x):
    """Nearest e4m3 value (ties to even; beyond 448 to +-448; NaN stays)."""
    x = x.to(F64)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def add_rms_norm(x, r, w, eps):
    s = x.to(F64) if r is None else x.to(F64) + r.to(F64)
    return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.to(F64)


def rotate(x, table, pos, interleaved):
    """x [..., 128] at table row pos (rows cos | sin); float64."""
    x = x.to(F64).clone()
    rot = table.shape[1]
    cos, sin = table[pos, :rot // 2].to(F64), table[pos, rot // 2:].to(F64)
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        u, v = x[..., a].clone(), x[..., b].clone()
        x[..., a] = u * cos[j] - v * sin[j]
        x[..., b] = v * cos[j] + u * sin[j]
    return x


def pow2_scale(top):
    """The least power of two s >= 2^-64 with top <= 448 s."""
    s = 2.0 ** -64
    while top > 448.0 * s:
        s *= 2.0
    return s


class Cache:
    """A paged cache's values and scales in float64, one side (keys or values)."""

    def __init__(self, raw, scale):
        self.q = raw.cpu().to(torch.float32).to(F64)        # e4m3 values
        self.s = scale.cpu().to(F64).clone()

    def append(self, x, table, kv_len):
        """x [t, kv_heads, 128]: the sequence's new entries; kv_len counts them."""
        t, hk = x.shape[:2]
        P = self.q.shape[2]
        start = kv_len - t
        for b in range(start // P, (kv_len - 1) // P + 1 if t else start // P):
            lo, hi = max(start, b * P), min(kv_len, (b + 1) * P)
            pg = int(table[b])
            for h in range(hk):
                new = x[lo - start:hi - start, h]
                fin = new[torch.isfinite(new)]
                s = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                if lo > b * P:
                    old = float(self.s[pg, h])
                    if s > old:
                        kept = self.q[pg, h, :lo - b * P]
                        self.q[pg, h, :lo - b * P] = e4m3_grid(kept * (old / s))
                    s = max(s, old)
                self.s[pg, h] = s
                self.q[pg, h, lo - b * P:hi - b * P] = e4m3_grid(new / s)


def attention(q, kc, vc, ks, vs, table, kv_len, scale, softcap=0.0, window=0):
    """q [t, heads, 128] of one sequence over its cache; returns out, lse in float64.  kc / vc:
    e4m3 values [pages, kv_heads, page, 128] in any float type.  Masked entries are not read."""
    t, H, _ = q.shape
    hk, P = kc.shape[1], kc.shape[2]
    G = H // hk
    out = torch.zeros(t, H, D, dtype=F64)
    lse = torch.full((t, H), -math.inf, dtype=F64)
    if kv_len == 0 or t == 0:
        return out, lse
    pg = table[:(kv_len + P - 1) // P].long()
    for g in range(hk):
        k = (kc[pg, g].to(F64) * ks[pg, g].to(F64)[:, None, None]).reshape(-1, D)[:kv_len]
        v = (vc[pg, g].to(F64) * vs[pg, g].to(F64)[:, None, None]).reshape(-1, D)[:kv_len]
        for i in range(t):
            p = kv_len - t + i
            lo = max(0, p - window + 1) if window else 0
            if p < lo:
                continue
            s = q[i, g * G:(g + 1) * G].to(F64) @ k[lo:p + 1].T * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            lse[i, g * G:(g + 1) * G] = torch.logsumexp(s, 1)
            out[i, g * G:(g + 1) * G] = torch.softmax(s, 1) @ v[lo:p + 1]
    return out, lse
