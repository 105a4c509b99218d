"""Cases for the paged-attention side of a hybrid layer stack: the KV cache's page bookkeeping, the append of
new tokens to the cache, the attention of new tokens over it, and the norms around a block.

`run` computes an operator in its plain form (elementary torch operations, 32-bit arithmetic, one rounding at
the end) or, with `own` set, through the package's entry points."""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases
def _attn(name, B, K, Hq, Hkv, d, ps, max_len, dtype="bf16", out="bf16", gate=True, ragged=True, layout="thd"):
    return {"name": name, "op": "attn", "B": B, "K": K, "Hq": Hq, "Hkv": Hkv, "d": d, "ps": ps, "max_len": max_len,
            "dtype": dtype, "out": out, "gate": gate, "ragged": ragged, "layout": layout}


def _extend(name, B, ps, max_len, new, pad=0):
    return {"name": name, "op": "extend", "B": B, "ps": ps, "max_len": max_len, "new": new, "pad": pad}


def _truncate(name, B, ps, max_len, K):
    return {"name": name, "op": "truncate", "B": B, "ps": ps, "max_len": max_len, "K": K}


def _append(name, T, Hq, Hkv, d, rope, ps, dtype="bf16", layout="thd"):
    return {"name": name, "op": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "rope": rope, "ps": ps,
            "dtype": dtype, "layout": layout}


def _norm(name, T, H, dtype="bf16", res="bf16", post=True, gate="none", chan=False):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "res": res, "post": post, "gate": gate,
            "chan": chan}


def listed():
    return [
        # one user's next token early in a conversation: latency
        _attn("attn_one_short", 1, 1, 16, 2, 256, 16, 777, ragged=False),
        # one user's next token at the end of a very long document: few rows, a long axis
        _attn("attn_one_long", 1, 1, 16, 2, 256, 64, 262139, ragged=False, layout="htd"),
        # a full decode batch of the 64 sequences the decode workload uses, lengths from nothing to 16k
        _attn("attn_batch_ragged", 64, 1, 24, 4, 256, 16, 16384),
        # a speculative verify of three drafted tokens for 64 sequences, as in the verify workload
        _attn("attn_verify_k3", 64, 3, 16, 2, 256, 16, 8192),
        # 32-bit activations and cache, a page size that divides nothing, every head its own keys in pairs
        _attn("attn_f32_odd", 9, 2, 6, 3, 64, 11, 5001, dtype="f32", out="f32", gate=False),
        # the next page-table step of a decode batch
        _extend("kv_extend_decode", 64, 16, 16384, "one", pad=0),
        # eight packed prompts of the varlen prefill workload, 65,536 tokens in all, into an empty cache
        _extend("kv_extend_prefill", 8, 16, 0, "prompt", pad=64),
        # after a verify: each sequence keeps what was accepted, some are finished
        _truncate("kv_truncate_verify", 64, 16, 16384, 3),
        # the decode batch's new tokens
        _append("kv_append_decode", 64, 16, 2, 256, 64, 16),
        # a prefill of 8,192 tokens into the cache
        _append("kv_append_prefill", 8192, 24, 4, 256, 64, 16),
        # around a block of a decode batch, hidden 2048
        _norm("norm_decode", 64, 2048, gate="token"),
        # around a block of a prefill, hidden 5120, 32-bit residual stream, gate per element and a channel scale
        _norm("norm_prefill", 8192, 5120, res="f32", gate="element", chan=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "extend", "truncate", "append", "norm"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        G, Hkv, d = rng.choice([1, 2, 3, 5, 6, 8, 12, 16]), rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
        K = rng.choice([1, 1, 1, 2, 3, 4, 7, 16])
        B = _log(rng, 1, 256)
        # the bytes of keys and values stay under the largest listed case's
        most = int(1.9e9 / (B * Hkv * d * 2 * ES[dtype]))
        # and so do the operations, at 50 a byte
        most = min(most, int(2.5e10 / (B * Hkv * G * K * d)), 262144)
        L = _log(rng, 1, max(2, most))
        c = _attn("", B, K, G * Hkv, Hkv, d, rng.choice([1, 5, 16, 16, 32, 64, 100, 256]), L, dtype,
                  rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32", rng.random() < 0.5, B > 1 and rng.random() < 0.8,
                  rng.choice(["thd", "htd"]))
    elif op == "extend":
        new = rng.choice(["one", "some", "prompt"])
        c = _extend("", _log(rng, 1, 64 if new == "prompt" else 1500), rng.choice([1, 7, 16, 32, 64]),
                    0 if new == "prompt" else _log(rng, 1, 16384), new, rng.choice([0, 5, 64]))
    elif op == "truncate":
        c = _truncate("", _log(rng, 1, 1500), rng.choice([1, 7, 16, 32, 64]), _log(rng, 1, 16384), rng.choice([1, 2, 3, 5, 16]))
    elif op == "append":
        d = rng.choice([64, 128, 256])
        G, Hkv = rng.choice([1, 2, 3, 6, 8]), rng.choice([1, 2, 4])
        c = _append("", _log(rng, 1, 8192), G * Hkv, Hkv, d, rng.choice([0, d // 4, d // 2, d]), rng.choice([1, 16, 20, 64]),
                    rng.choice(["bf16", "bf16", "f32"]), rng.choice(["thd", "htd"]))
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = _norm("", _log(rng, 1, 8192), rng.choice([_log(rng, 1, 5120), 2048, 5120, 8 * _log(rng, 1, 640)]), dtype,
                  "f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), rng.random() < 0.6,
                  rng.choice(["none", "token", "element"]), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ lengths
GOLD = 0.6180339887498949


def _spread(n, lo, hi, at=0.0):
    """n whole numbers spread evenly over lo..hi, always the same ones."""
    return [lo + int((hi - lo) * math.fmod((i + 0.5) * GOLD + at, 1.0)) for i in range(n)]


def _attn_lens(c):
    if not c["ragged"]:
        return [c["max_len"]] * c["B"]
    lens = _spread(c["B"], 1, c["max_len"])
    if c["B"] > 4:
        lens[3] = 0   # an idle slot of the batch
    lens[0] = c["max_len"]
    return lens


def _cdiv(a, b):
    return -(-a // b)


def _extend_lens(c):
    """(current lengths, new tokens)"""
    B = c["B"]
    if c["new"] == "prompt":
        w = _spread(B, 200, 1000)
        n = [65536 * x // sum(w) for x in w]
        n[-1] += 65536 - sum(n)
        return [0] * B, n
    cur = _spread(B, 0, c["max_len"])
    return cur, ([1] * B if c["new"] == "one" else _spread(B, 0, 40, 0.3))


def _truncate_lens(c):
    """(current lengths, kept lengths)"""
    cur = [x + c["K"] for x in _spread(c["B"], 0, c["max_len"])]
    keep = [x - int((c["K"] + 1) * math.fmod((i + 0.5) * GOLD + 0.2, 1.0)) for i, x in enumerate(cur)]
    keep = [0 if i % 11 == 10 else x for i, x in enumerate(keep)]
    return cur, keep


# ------------------------------------------------------------------------------------------------ work
def work(c):
    op = c["op"]
    if op == "attn":
        es, eo = ES[c["dtype"]], ES[c["out"]]
        lens, K, n_row = _attn_lens(c), c["K"], c["B"] * c["K"] * c["Hq"] * c["d"]
        kv = sum(lens) * c["Hkv"] * c["d"] * 2 * es
        table = sum(_cdiv(x, c["ps"]) for x in lens) * 4 + 4 * c["B"]
        seen = sum(max(0, x - K + p + 1) for x in lens for p in range(K))
        return {"bytes": kv + table + n_row * (es * (2 if c["gate"] else 1) + eo), "flops": 4 * seen * c["Hq"] * c["d"]}
    if op == "extend":
        cur, new = _extend_lens(c)
        pages = sum(_cdiv(x + n, c["ps"]) - _cdiv(x, c["ps"]) for x, n in zip(cur, new))
        # lengths, new counts and held pages in and out, the new pages read and written, the old page of a token that needs it, rows
        return {"bytes": 24 * c["B"] + 8 * pages + 8 * (sum(new) + c["pad"]), "flops": 0}
    if op == "truncate":
        cur, keep = _truncate_lens(c)
        pages = sum(_cdiv(x, c["ps"]) - _cdiv(y, c["ps"]) for x, y in zip(cur, keep))
        return {"bytes": 20 * c["B"] + 8 * pages, "flops": 0}
    if op == "append":
        es, T, d = ES[c["dtype"]], c["T"], c["d"]
        return {"bytes": T * d * es * (2 * c["Hq"] + 4 * c["Hkv"]) + T * (8 + 4 * c["rope"]) + 8 * d,
                "flops": T * d * (c["Hq"] + c["Hkv"]) * 6}
    es, er, n = ES[c["dtype"]], ES[c["res"]], c["T"] * c["H"]
    gate = {"none": 0, "token": c["T"] * es, "element": n * es}[c["gate"]]
    return {"bytes": n * (2 * es + 2 * er) + gate + 4 * c["H"] * (1 + c["post"] + c["chan"]), "flops": 10 * n}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _cache(g, pages, c, dt):
    """One of the two halves of a cache, seen as [page][token][head][channel]; "htd" keeps a page's heads apart."""
    if c["layout"] == "thd":
        shape = (pages, c["ps"], c["Hkv"], c["d"])
    else:
        shape = (pages, c["Hkv"], c["ps"], c["d"])
    t = torch.empty(shape, device=DEV, dtype=dt)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        m = min(1 << 28, flat.numel() - i)
        flat[i:i + m] = torch.randn(m, generator=g, device=DEV, dtype=dt)
    return t if c["layout"] == "thd" else t.transpose(1, 2)


def _tables(g, held, ps, spare=0):
    """A block table of shuffled pages for `held` pages a sequence, the stack of free pages and their number."""
    n = sum(held) + spare
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=g, device=DEV))))
    width = max(1, max(held) + spare)
    table, at = torch.zeros(len(held), min(width, n) or 1, dtype=torch.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h].to(torch.int32)
        at += h
    free = torch.zeros(max(1, n), dtype=torch.int32)
    free[: n - at] = perm[at:].to(torch.int32)
    return table.to(DEV), free.to(DEV), torch.tensor([n - at], dtype=torch.int32, device=DEV)


def _shuffled(lens, seed):
    order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()
    return [lens[i] for i in order]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    if own:
        import gated_deltanet_linear_decode_gb300 as gdn
        s["gdn"] = gdn
    op = c["op"]
    if op == "attn":
        dt, odt = DT[c["dtype"]], DT[c["out"]]
        lens = _shuffled(_attn_lens(c), seed)
        held = [_cdiv(x, c["ps"]) for x in lens]
        table, _, _ = _tables(g, held, c["ps"], 3)
        pages = sum(held) + 3
        s["k"], s["v"] = _cache(g, pages, c, dt), _cache(g, pages, c, dt)
        T = c["B"] * c["K"]
        # normalised heads with learned weights somewhat above one: scores of a few units
        s["q"] = _randn(g, T, c["Hq"] * c["d"], dtype=dt, scale=1.5)
        s["gate"] = _randn(g, T, c["Hq"] * c["d"], dtype=dt) if c["gate"] else None
        s["table"], s["lens"] = table, _i32(lens)
        s["out"] = torch.empty(T, c["Hq"] * c["d"], device=DEV, dtype=odt)
        if own:
            s["dims"] = gdn.make_attn_dims(c["Hq"], c["Hkv"], c["d"], dt, odt)
            s["cache"] = gdn.KvCache(s["k"], s["v"])
            n = gdn.gdn_attn_decode_workspace_bytes(s["dims"], c["B"], c["K"])
            s["ws"] = torch.zeros(n, device=DEV, dtype=torch.uint8)
    elif op in ("extend", "truncate"):
        B = c["B"]
        cur, other = _extend_lens(c) if op == "extend" else _truncate_lens(c)
        order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
        cur, other = [cur[i] for i in order], [other[i] for i in order]
        held = [_cdiv(x, c["ps"]) for x in cur]
        more = sum(_cdiv(x + n, c["ps"]) - h for x, n, h in zip(cur, other, held)) if op == "extend" else 0
        s["table"], s["free"], s["n_free"] = _tables(g, held, c["ps"], more + 37)
        s["lens"], s["held"] = _i32(cur), _i32(held)
        s["new" if op == "extend" else "keep"] = _i32(other)
        s["lens_out"], s["held_out"], s["n_free_out"] = (torch.empty_like(s[k]) for k in ("lens", "held", "n_free"))
        if op == "extend":
            s["T"] = sum(other) + c["pad"]
            s["slots"] = torch.empty(s["T"], device=DEV, dtype=torch.int32)
            s["pos"] = torch.empty(s["T"], device=DEV, dtype=torch.int32)
            s["cu"] = torch.empty(B + 1, device=DEV, dtype=torch.int32)
    elif op == "append":
        dt, T, d = DT[c["dtype"]], c["T"], c["d"]
        pages = _cdiv(T, c["ps"]) + 2
        s["k"], s["v"] = _cache(g, pages, c, dt), _cache(g, pages, c, dt)
        # one projection's rows hold q, k and v side by side
        qkv = _randn(g, T, (c["Hq"] + 2 * c["Hkv"]) * d, dtype=dt)
        nq, nk = c["Hq"] * d, c["Hkv"] * d
        s["xq"], s["xk"], s["xv"] = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
        s["slots"] = torch.randperm(pages * c["ps"], generator=g, device=DEV)[:T].to(torch.int32)
        s["pos"] = torch.randint(0, 40960, (T,), generator=g, device=DEV).to(torch.int32)
        s["wq"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
        s["wk"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
        if c["rope"]:
            f = torch.arange(c["rope"] // 2, dtype=torch.float64, device=DEV)
            a = torch.arange(40960, dtype=torch.float64, device=DEV)[:, None] * 1e7 ** (-2 * f / c["rope"])
            s["cos"], s["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
        else:
            s["cos"] = s["sin"] = None
        s["q_out"] = torch.empty(T, nq, device=DEV, dtype=dt)
        if own:
            s["dims"] = gdn.make_attn_dims(c["Hq"], c["Hkv"], d, dt, dt, rope_dim=c["rope"])
            s["cache"] = gdn.KvCache(s["k"], s["v"])
    else:
        dt, rt, T, H = DT[c["dtype"]], DT[c["res"]], c["T"], c["H"]
        s["y"], s["h"] = _randn(g, T, H, dtype=dt), _randn(g, T, H, dtype=rt, scale=3.0)
        s["gate"] = None if c["gate"] == "none" else _randn(g, T, H if c["gate"] == "element" else 1, dtype=dt)
        s["post"] = 1 + 0.1 * torch.randn(H, generator=g, device=DEV) if c["post"] else None
        s["pre"] = 1 + 0.1 * torch.randn(H, generator=g, device=DEV)
        s["chan"] = 0.5 + 0.1 * torch.randn(H, generator=g, device=DEV) if c["chan"] else None
        s["alpha"] = 0.75
        s["h_out"] = torch.empty(T, H, device=DEV, dtype=rt)
        s["x"] = torch.empty(T, H, device=DEV, dtype=dt)
        if own:
            s["dims"] = gdn.make_norm_dims(H, dt, rt, alpha=s["alpha"])
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _OWN[op](s, s["gdn"])
    return _PLAIN[op](s)


def _own_attn(s, gdn):
    gdn.gdn_attn_decode(s["dims"], s["cache"], s["c"]["K"], s["q"], s["table"], s["lens"], s["out"], gate=s["gate"],
                        workspace=s["ws"])
    return s["out"]


def _own_extend(s, gdn):
    gdn.gdn_kv_extend(s["c"]["ps"], s["new"], s["lens"], s["held"], s["table"], s["free"], s["n_free"], s["slots"],
                      s["pos"], s["cu"], seq_len_out=s["lens_out"], n_pages_out=s["held_out"],
                      free_count_out=s["n_free_out"])
    return {"slots": s["slots"], "pos": s["pos"], "cu": s["cu"], "lens": s["lens_out"], "held": s["held_out"],
            "n_free": s["n_free_out"], "table": s["table"]}


def _own_truncate(s, gdn):
    gdn.gdn_kv_truncate(s["c"]["ps"], s["keep"], s["lens"], s["held"], s["table"], s["free"], s["n_free"],
                        seq_len_out=s["lens_out"], n_pages_out=s["held_out"], free_count_out=s["n_free_out"])
    return {"lens": s["lens_out"], "held": s["held_out"], "n_free": s["n_free_out"], "free": s["free"]}


def _own_append(s, gdn):
    gdn.gdn_kv_append(s["dims"], s["cache"], s["xq"], s["xk"], s["xv"], s["pos"], s["slots"], s["q_out"],
                      q_norm_w=s["wq"], k_norm_w=s["wk"], rope_cos=s["cos"], rope_sin=s["sin"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_norm(s, gdn):
    gdn.gdn_norm_residual(s["dims"], s["h"], s["h_out"], y=s["y"], gate=s["gate"], post_w=s["post"],
                          chan_scale=s["chan"], pre_w=s["pre"], x=s["x"])
    return {"h": s["h_out"], "x": s["x"]}


_OWN = {"attn": _own_attn, "extend": _own_extend, "truncate": _own_truncate, "append": _own_append, "norm": _own_norm}


def _plain_attn(s):
    c = s["c"]
    B, K, Hq, Hkv, d = c["B"], c["K"], c["Hq"], c["Hkv"], c["d"]
    G, L = Hq // Hkv, max(1, c["max_len"])
    j = torch.arange(L, device=DEV)
    page = s["table"].long()[:, j // c["ps"]]                                       # [B][L]
    q = s["q"].float().view(B, K, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, K * G, d)
    k = s["k"][page, j % c["ps"]].permute(0, 2, 3, 1).float()                       # [B][Hkv][d][L]
    sc = torch.matmul(q, k).view(B, Hkv, K, G, L) * (1.0 / math.sqrt(d))
    del k
    p = torch.arange(K, device=DEV)
    seen = j[None, None, :] < (s["lens"].long()[:, None] - K + 1 + p)[:, :, None]   # [B][K][L]
    sc = torch.where(seen[:, None, :, None, :], sc, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(m == float("-inf"), 0.0, m))
    z = e.sum(-1, keepdim=True)
    e = e / torch.where(z == 0, 1.0, z)
    v = s["v"][page, j % c["ps"]].permute(0, 2, 1, 3).float()                       # [B][Hkv][L][d]
    o = torch.matmul(e.view(B, Hkv, K * G, L), v)
    o = o.view(B, Hkv, K, G, d).permute(0, 2, 1, 3, 4).reshape(B * K, Hq * d)
    if s["gate"] is not None:
        o = o / (1 + torch.exp(-s["gate"].float()))
    return o.to(DT[c["out"]])


def _plain_extend(s):
    ps, B, table = s["c"]["ps"], s["c"]["B"], s["table"]
    P = table.shape[1]
    L, a, held = s["lens"].long(), s["new"].long(), s["held"].long()
    total = (L + a + ps - 1) // ps
    need = (total - held).clamp(min=0)
    before = need.cumsum(0) - need
    ok = (total <= P) & ((need == 0) | (before + need <= s["n_free"]))
    got = torch.where(ok, need, 0)
    add = torch.where(ok, a, 0)
    col = torch.arange(P, device=DEV)
    fresh = (col >= held[:, None]) & (col < (held + got)[:, None])
    at = (s["n_free"] - 1 - before[:, None] - (col - held[:, None])).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), add.cumsum(0)])
    t = torch.arange(s["T"], device=DEV)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = L[b] + t - cu[b]
    slot = table[b, (pos // ps).clamp(0, P - 1)].long() * ps + pos % ps
    i = torch.int32
    return {"slots": torch.where(real, slot, -1).to(i), "pos": torch.where(real, pos, 0).to(i), "cu": cu.to(i),
            "lens": (L + add).to(i), "held": (held + got).to(i), "n_free": (s["n_free"] - got.sum()).to(i), "table": table}


def _plain_truncate(s):
    ps, table, free = s["c"]["ps"], s["table"], s["free"]
    held, keep = s["held"].long(), s["keep"].long()
    stay = torch.minimum((keep + ps - 1) // ps, held)
    back = held - stay
    before, n = back.cumsum(0) - back, back.sum()
    col = torch.arange(table.shape[1], device=DEV)
    gone = (col >= stay[:, None]) & (col < held[:, None])
    at = s["n_free"] + n - 1 - (before[:, None] + col - stay[:, None])
    free[at[gone]] = table[gone]
    i = torch.int32
    return {"lens": keep.to(i), "held": stay.to(i), "n_free": (s["n_free"] + n).to(i), "free": free}


def _plain_append(s):
    c = s["c"]
    T, d, r, ps = c["T"], c["d"], c["rope"], c["ps"]

    def head(x, w):
        x = x.float().reshape(T, -1, d)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        if r:
            co, si = s["cos"][s["pos"].long()][:, None], s["sin"][s["pos"].long()][:, None]
            x1, x2 = x[..., :r // 2], x[..., r // 2:r]
            x = torch.cat([x1 * co - x2 * si, x2 * co + x1 * si, x[..., r:]], -1)
        return x

    slot = s["slots"].long()
    s["k"][slot // ps, slot % ps] = head(s["xk"], s["wk"]).to(s["k"].dtype)
    s["v"][slot // ps, slot % ps] = s["xv"].reshape(T, -1, d)
    return {"q": head(s["xq"], s["wq"]).reshape(T, -1).to(s["k"].dtype), "k": s["k"], "v": s["v"]}


def _plain_norm(s):
    def rms(x, w):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    u = s["y"].float()
    if s["post"] is not None:
        u = rms(u, s["post"])
    if s["gate"] is not None:
        u = u / (1 + torch.exp(-s["gate"].float()))
    if s["chan"] is not None:
        u = u * s["chan"]
    h = s["h"].float() + s["alpha"] * u
    return {"h": h.to(s["h"].dtype), "x": rms(h, s["pre"]).to(s["y"].dtype)}


_PLAIN = {"attn": _plain_attn, "extend": _plain_extend, "truncate": _plain_truncate, "append": _plain_append, "norm": _plain_norm}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "attn":
        d, K, ps, G = c["d"], c["K"], c["ps"], c["Hq"] // c["Hkv"]
        out = torch.zeros(c["B"], K, c["Hq"], d, dtype=torch.float64, device=DEV)
        lens, table = s["lens"].tolist(), s["table"].long()
        q = s["q"].double().view(c["B"], K, c["Hq"], d)
        for b, n in enumerate(lens):
            rows = (table[b, : _cdiv(n, ps), None] * ps + torch.arange(ps, device=DEV)).reshape(-1)[:n]
            for h in range(c["Hkv"]):
                kh, vh = s["k"][rows // ps, rows % ps, h].double(), s["v"][rows // ps, rows % ps, h].double()
                for p in range(K):
                    m = n - K + p + 1
                    if m > 0:
                        w = torch.softmax(q[b, p, h * G:(h + 1) * G] @ kh[:m].T / math.sqrt(d), -1)
                        out[b, p, h * G:(h + 1) * G] = w @ vh[:m]
        out = out.view(c["B"] * K, -1)
        return out * torch.sigmoid(s["gate"].double()) if c["gate"] else out
    if op == "extend":
        ps = c["ps"]
        table, free = s["table"].tolist(), s["free"].tolist()[: int(s["n_free"])]
        lens, held, new = s["lens"].tolist(), s["held"].tolist(), s["new"].tolist()
        slots, pos, cu = [], [], [0]
        for b in range(c["B"]):
            for _ in range(new[b]):
                if lens[b] == held[b] * ps:
                    table[b][held[b]] = free.pop()
                    held[b] += 1
                slots.append(table[b][lens[b] // ps] * ps + lens[b] % ps)
                pos.append(lens[b])
                lens[b] += 1
            cu.append(len(slots))
        slots += [-1] * c["pad"]
        pos += [0] * c["pad"]
        out = {"slots": slots, "pos": pos, "cu": cu, "lens": lens, "held": held, "n_free": [len(free)], "table": table}
        return {k: np.array(v, dtype=np.int32) for k, v in out.items()}
    if op == "truncate":
        ps = c["ps"]
        table, held, n = s["table"].tolist(), s["held"].tolist(), int(s["n_free"])
        free, keep = s["free"].tolist(), s["keep"].tolist()
        for b in reversed(range(c["B"])):   # the last sequence's last page first
            while held[b] > _cdiv(keep[b], ps):
                held[b] -= 1
                free[n] = table[b][held[b]]
                n += 1
        out = {"lens": keep, "held": held, "n_free": [n], "free": free}
        return {k: np.array(v, dtype=np.int32) for k, v in out.items()}
    if op == "append":
        T, d, r, ps = c["T"], c["d"], c["rope"], c["ps"]
        pos, slot = s["pos"].long(), s["slots"].long()
        k, v = s["k"].double(), s["v"].double()

        def turned(x, w):
            x = x.double().reshape(T, -1, d)
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            if r:
                z = torch.complex(x[..., :r // 2].clone(), x[..., r // 2:r].clone())
                z = z * torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None]
                x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
            return x

        k[slot // ps, slot % ps] = turned(s["xk"], s["wk"])
        v[slot // ps, slot % ps] = s["xv"].double().reshape(T, -1, d)
        return {"q": turned(s["xq"], s["wq"]).reshape(T, -1), "k": k, "v": v}
    u = s["y"].double()
    if c["post"]:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["post"].double()
    if c["gate"] != "none":
        u = u * torch.sigmoid(s["gate"].double())
    h = s["h"].double() + s["alpha"] * u * (s["chan"].double() if c["chan"] else 1.0)
    return {"h": h, "x": h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["pre"].double()}
