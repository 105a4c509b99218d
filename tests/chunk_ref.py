"""gdn_attn_chunk in 64 bits on the CPU, from its definition, and inputs for it (no code of the library)."""
import math

import numpy as np
import torch

from tests.attn_ref import f64


def chunk(q, k, v, table, lens, cu, Hq, Hkv, d, gate=None, scale=None, absent=()):
    """q, gate [T][Hq*d]; k, v [page][token][head][channel]; keys whose page is in `absent` are left out.  Returns the result
    and, of the same shape, sum_j w_j |v_j| (with the gate), by which errors of weights and sums are measured."""
    ps, G, scale = k.shape[1], Hq // Hkv, 1 / math.sqrt(d) if scale is None else scale
    out, size = np.zeros((q.shape[0], Hq, d)), np.zeros((q.shape[0], Hq, d))
    qh = q.reshape(-1, Hq, d)
    for b, n in enumerate(lens):
        n = max(0, min(n, table.shape[1] * ps))
        rows = cu[b + 1] - cu[b]
        if rows <= 0:
            continue
        j = np.arange(n)
        page = table[b, j // ps]
        there = ~np.isin(page, list(absent))
        j, page = j[there], page[there]
        see = j[None, :] <= (n - rows + np.arange(rows))[:, None]
        for h in range(Hkv):
            kh, vh = k[page, j % ps, h], v[page, j % ps, h]
            for g in range(G):
                s = np.where(see, scale * (qh[cu[b]:cu[b + 1], h * G + g] @ kh.T), -np.inf)
                m = s.max(-1, keepdims=True, initial=-np.inf)
                e = np.exp(s - np.where(np.isinf(m), 0, m))
                z = e.sum(-1, keepdims=True)
                w = e / np.where(z == 0, 1, z)
                out[cu[b]:cu[b + 1], h * G + g] = w @ vh
                size[cu[b]:cu[b + 1], h * G + g] = w @ np.abs(vh)
    sig = 1.0 if gate is None else 1 / (1 + np.exp(-gate))
    return out.reshape(-1, Hq * d) * sig, size.reshape(-1, Hq * d) * sig


class Batch:
    """Sequences with `new` tokens, `lens` long with them, in shuffled pages."""

    def __init__(self, new, lens, Hq, Hkv, d, ps, dt=torch.bfloat16, layout="thd", gate=False, pad=0, seed=0, fill=None, wide=False):
        g = torch.Generator().manual_seed(seed)
        held = [-(-max(0, n) // ps) for n in lens]
        pages = sum(held) + 2
        perm, at = torch.randperm(pages, generator=g).to(torch.int32), 0
        table = torch.zeros(len(lens), max(held + [0]) + 1, dtype=torch.int32)
        for b, h in enumerate(held):
            table[b, :h] = perm[at:at + h]
            at += h
        shape = (pages, ps, Hkv, d)
        rn = lambda *s: torch.randn(*s, generator=g)
        k, v = rn(*shape), rn(*shape)
        if fill is not None:   # what no sequence has: the other pages and the ends of the last ones
            mine = torch.zeros(pages, ps, dtype=torch.bool)
            for b, n in enumerate(lens):
                for i in range(held[b]):
                    mine[table[b, i], : max(0, min(ps, n - i * ps))] = True
            k[~mine], v[~mine] = fill, fill
        self.T = sum(new) + pad
        # wide: q and gate as column slices of one row
        n, w = Hq * d, 3 * Hq * d if wide else Hq * d
        q, gt = rn(self.T, w) * 1.5, rn(self.T, w) if gate else None
        dev = lambda t: t.to(dt).cuda()
        self.k, self.v = dev(k), dev(v)
        if layout == "htd":
            self.k, self.v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (self.k, self.v))
        elif layout == "both":
            t = torch.cat([self.k, self.v], -1)
            self.k, self.v = t[..., :d], t[..., d:]
        self.q = dev(q)[:, n:2 * n] if wide else dev(q)
        self.gate = None if gt is None else dev(gt)[:, 2 * n:] if wide else dev(gt)
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.cu = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32).cuda()
        self.new, self.len_list, self.Hq, self.Hkv, self.d, self.dt, self.ps = new, lens, Hq, Hkv, d, dt, ps

    def want(self, scale=None, absent=()):
        k, v = f64(self.k), f64(self.v)
        return chunk(f64(self.q), k, v, self.table.cpu().numpy(), self.len_list, self.cu.tolist(), self.Hq, self.Hkv, self.d,
                     None if self.gate is None else f64(self.gate), scale, absent)

    def spread(self, scale=None):
        """The largest scale * sum_i |q_i k_i| there may be (of tokens that a sequence has: the others may be anything)."""
        s = 1 / math.sqrt(self.d) if scale is None else abs(scale)
        k = self.k.float().norm(dim=-1)
        return s * float(self.q.float().norm(dim=-1).max()) * float(k[k < 1e15].max())


def half_step(dt):
    return torch.finfo(dt).eps / 2


def bound(want, size, b, out_dtype, scale=None, joins=2):
    """What a result may be off by, from the roundings there are: its own (half a step); of a bf16 result's weights (half a step
    of bf16 each); of the scores (d products and sums in fp32, each half a step of the largest sum there may be, twice: in the
    weight and in the sum of weights); 2^-21 of a power, a gate, a quotient each; and of sums over len keys, by blocks of
    at most 64 or 128 (2^-24 a step, 2^-23 where the tensor cores cut instead of rounding)."""
    n = max(b.len_list + [1])
    weights = (half_step(torch.bfloat16) if out_dtype == torch.bfloat16 else 0.0)
    weights += 2 * b.d * 2.0 ** -23 * b.spread(scale) + 8 * 2.0 ** -21 + (n + 128 * joins) * 2.0 ** -23
    return half_step(out_dtype) * np.abs(want) + (1 + half_step(out_dtype)) * weights * size + 1e-30
