"""The operators of include/gdn_attn.h and include/gdn_norm.h in 64 bits on the CPU, from their definitions
(numpy, one sequence, token or row after another; no code of the library)."""
import math

import numpy as np


def f64(t):
    return t.detach().double().cpu().numpy()


def attn(q, k, v, table, lens, K, Hq, Hkv, d, gate=None, scale=None, absent=()):
    """q, gate [B*K][Hq*d]; k, v [page][token][head][channel]; keys whose page is in `absent` are left out."""
    ps, G, scale = k.shape[1], Hq // Hkv, 1 / math.sqrt(d) if scale is None else scale
    out = np.zeros((len(lens) * K, Hq, d))
    qh = q.reshape(-1, Hq, d)
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * ps))
        j = np.arange(n)
        page = table[b, j // ps]
        there = ~np.isin(page, list(absent))
        j, page = j[there], page[there]
        for h in range(Hkv):
            kh, vh = k[page, j % ps, h], v[page, j % ps, h]
            for p in range(K):
                see = j <= n - K + p
                if not see.any():
                    continue
                s = scale * (qh[b * K + p, h * G:(h + 1) * G] @ kh[see].T)
                e = np.exp(s - s.max(-1, keepdims=True))
                out[b * K + p, h * G:(h + 1) * G] = (e / e.sum(-1, keepdims=True)) @ vh[see]
    out = out.reshape(-1, Hq * d)
    return out if gate is None else out / (1 + np.exp(-gate))


class Pages:
    """Lengths, held pages, block table and free stack of B sequences, one step after another."""

    def __init__(self, ps, table, free, n_free, lens, held):
        self.ps, self.table, self.lens, self.held = ps, [list(r) for r in table], list(lens), list(held)
        self.n_pages, self.free, self.rest = len(free), list(free[:n_free]), list(free[n_free:])

    def extend(self, new, T):
        P, B = len(self.table[0]) if self.table else 1, len(self.lens)
        most = min(P, self.n_pages)
        slots, pos, cu, refused = [], [], [0], []
        asked_pages = asked_rows = 0
        n_free = len(self.free)
        for b in range(B):
            L, a, h = self.lens[b], new[b], self.held[b]
            total = -(-(L + a) // self.ps)
            if L < 0 or a < 0 or h < 0 or h > most or total > most:
                refused.append(b)
                cu.append(len(slots))
                continue
            need = max(0, total - h) if a > 0 else 0
            asked_pages += need
            asked_rows += a
            if (need and asked_pages > n_free) or (a and asked_rows > T):
                refused.append(b)
                cu.append(len(slots))
                continue
            for _ in range(need):
                self.table[b][self.held[b]] = self.free.pop()
                self.held[b] += 1
            for i in range(a):
                slots.append(self.table[b][(L + i) // self.ps] * self.ps + (L + i) % self.ps)
                pos.append(L + i)
            self.lens[b] = L + a
            cu.append(len(slots))
        pad = T - len(slots)
        return slots + [-1] * pad, pos + [0] * pad, cu, refused

    def truncate(self, keep):
        """Refusals first (in order), then the pages go back: the last sequence's last page first."""
        P = len(self.table[0]) if self.table else 1
        refused, stay, asked, room = [], [], 0, self.n_pages - len(self.free)
        for b, n in enumerate(keep):
            L, h = self.lens[b], self.held[b]
            stay.append(h)
            if n < 0 or n > L or h < 0 or h > P:
                refused.append(b)
                continue
            s = min(h, -(-n // self.ps))
            asked += h - s
            if h > s and asked > room:
                refused.append(b)
                continue
            stay[b] = s
        for b in reversed(range(len(keep))):
            if b in refused:
                continue
            while self.held[b] > stay[b]:
                self.held[b] -= 1
                self.free.append(self.table[b][self.held[b]])
            self.lens[b] = keep[b]
        return refused


def heads(x, d, w=None, cos=None, sin=None, eps=1e-6):
    """Norm and rotation of [T][H*d]; cos, sin [T][rope_dim/2]."""
    x = x.reshape(x.shape[0], -1, d).copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if cos is not None:
        r = cos.shape[1]
        a, b = x[..., :r].copy(), x[..., r:2 * r].copy()
        x[..., :r] = a * cos[:, None] - b * sin[:, None]
        x[..., r:2 * r] = b * cos[:, None] + a * sin[:, None]
    return x


def norm_residual(h, y=None, gate=None, post=None, chan=None, pre=None, alpha=1.0, eps=1e-6):
    def rms(x, w):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w

    if y is not None:
        u = y if post is None else rms(y, post)
        u = u if gate is None else u / (1 + np.exp(-gate))
        u = u if chan is None else u * chan
        h = h + alpha * u
    return h, None if pre is None else rms(h, pre)
