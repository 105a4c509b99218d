"""Cases for prompts and shared pages on the attention side of a hybrid layer stack: the attention of a chunk of new
tokens over the paged KV cache, pages shared between sequences (forked and released), the compaction of a cache, and
the copies of pages that these ask for.

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
def _chunk(name, B, new, ctx, Hq, Hkv, d, ps, mix="even", dtype="bf16", out="bf16", gate=True, layout="thd", pad=0):
    """B sequences with up to `new` new tokens each after up to `ctx` earlier ones; mix "even": all of them so many,
    "ragged": from none to so many, "step": the first has them, the others one token each; pad rows behind the last."""
    return {"name": name, "op": "chunk", "B": B, "new": new, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "d": d, "ps": ps, "mix": mix,
            "dtype": dtype, "out": out, "gate": gate, "layout": layout, "pad": pad}


def _share(name, parents, children, ps, max_len, whole):
    """Every child is forked from a parent (at its whole length or somewhere in it), then the children are released."""
    return {"name": name, "op": "share", "parents": parents, "children": children, "ps": ps, "max_len": max_len, "whole": whole}


def _compact(name, B, ps, max_len, fill, shared):
    """`fill` of the cache's pages are held, `shared` of the sequences share the first half of another's pages."""
    return {"name": name, "op": "compact", "B": B, "ps": ps, "max_len": max_len, "fill": fill, "shared": shared}


def _copy(name, n, pages, Hkv, d, ps, dtype="bf16", layout="thd", skip=0.0):
    """n pairs of a cache of so many pages, a part of them empty."""
    return {"name": name, "op": "copy", "n": n, "pages": pages, "Hkv": Hkv, "d": d, "ps": ps, "dtype": dtype, "layout": layout,
            "skip": skip}


def listed():
    return [
        # the next message of one user, early in a conversation: latency
        _chunk("chunk_short", 1, 37, 740, 16, 2, 256, 16),
        # the prompt of the prefill workload, 8,192 tokens into an empty cache
        _chunk("chunk_prompt", 1, 8192, 0, 24, 4, 256, 16),
        # a serving step: a piece of 2,048 tokens of a long document beside the next tokens of 31 other sequences
        _chunk("chunk_step", 32, 2048, 32768, 16, 2, 256, 64, mix="step", layout="htd"),
        # ragged prompts of a batch, some with a cached prefix, generic heads of 128
        _chunk("chunk_prompts", 8, 4096, 1000, 64, 8, 128, 32, mix="ragged", pad=64),
        # 64 tokens each of 16 sequences scored again, 32-bit results
        _chunk("chunk_rescore", 16, 64, 4096, 16, 4, 64, 16, mix="ragged", out="f32", gate=False),
        # 32-bit activations and cache, a page size that divides nothing, every head its own keys in pairs
        _chunk("chunk_f32", 9, 301, 1500, 6, 3, 64, 11, mix="ragged", dtype="f32", out="f32", gate=False),
        # 63 answers to one prompt
        _share("share_answers", 1, 63, 16, 16391, True),
        # 992 requests on 32 cached prefixes
        _share("share_prefixes", 32, 992, 16, 8192, False),
        # a small cache after a few requests have ended
        _compact("compact_small", 8, 64, 2048, 0.5, 0.25),
        # the cache of a long-running server, 64 sequences of up to 16,384 tokens, half of the pages free
        _compact("compact_server", 64, 16, 16384, 0.5, 0.25),
        # the partly filled pages of 63 forks
        _copy("copy_forks", 63, 2048, 2, 256, 16, skip=0.1),
        # the moves of a compaction
        _copy("copy_compaction", 16000, 40960, 4, 256, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "chunk", "share", "compact", "copy"])
    if op == "chunk":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        out = rng.choice(["bf16", "bf16", "f32"]) if dtype == "bf16" else "f32"
        G, Hkv, d = rng.choice([1, 2, 3, 5, 6, 8, 12, 16]), rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 256])
        B = _log(rng, 1, 64)
        mix = rng.choice(["even", "ragged", "step"]) if B > 1 else "even"
        new, ctx = _log(rng, 1, 8192), rng.choice([0, _log(rng, 1, 32768)])
        # the operations and the bytes of the cache stay under the largest listed case's
        most = 4e11 if out == "bf16" else 1e11
        full = 1 if mix == "step" else B
        while 4 * G * Hkv * d * full * new * (ctx + new) > most or B * (ctx + new) * Hkv * d * ES[dtype] > 5e8:
            new, ctx = (new + 1) // 2, ctx // 2
        c = _chunk("", B, new, ctx, G * Hkv, Hkv, d, rng.choice([1, 5, 16, 16, 32, 64, 100, 256]), mix, dtype, out,
                   rng.random() < 0.5, rng.choice(["thd", "htd"]), rng.choice([0, 0, 7]))
    elif op == "share":
        c = _share("", _log(rng, 1, 32), _log(rng, 1, 992), rng.choice([1, 7, 16, 32, 64]), _log(rng, 1, 8192), rng.random() < 0.5)
    elif op == "compact":
        c = _compact("", _log(rng, 1, 300), rng.choice([1, 7, 16, 32, 64]), _log(rng, 1, 3000), rng.choice([0.1, 0.5, 0.9]),
                     rng.choice([0.0, 0.25]))
    else:
        Hkv, d, ps, dtype = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 5, 16, 64, 256]), rng.choice(["bf16", "f32"])
        n = max(1, min(_log(rng, 1, 16000), int(5e8 / (Hkv * d * ps * ES[dtype]))))
        c = _copy("", n, 2 * n + rng.choice([0, 1, 17]), Hkv, d, ps, dtype, rng.choice(["thd", "htd"]), rng.choice([0.0, 0.3]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ lengths
GOLD = 0.6180339887498949


def _spread(n, lo, hi, at=0.0):
    """n whole numbers spread evenly over lo..hi, always the same ones."""
    return [lo + int((hi - lo + 1) * math.fmod((i + 0.5) * GOLD + at, 1.0)) for i in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _chunk_lens(c):
    """(new tokens, lengths with them) of every sequence"""
    B = c["B"]
    if c["mix"] == "even":
        new, ctx = [c["new"]] * B, [c["ctx"]] * B
    elif c["mix"] == "ragged":
        new, ctx = _spread(B, 1, c["new"]), _spread(B, 0, c["ctx"], 0.4)
        new[0] = c["new"]
        if B > 4:
            new[3] = 0   # a sequence that has nothing to do in this step
    else:
        new, ctx = [c["new"]] + [1] * (B - 1), [c["ctx"]] + _spread(B - 1, 0, min(c["ctx"], 16384))
    return new, [a + b for a, b in zip(new, ctx)]


def _share_lens(c):
    """(lengths of the parents, parent of each child, tokens that it takes over)"""
    n, m = c["parents"], c["children"]
    lens = [c["max_len"]] + _spread(n - 1, 1, c["max_len"])
    parent = [i % n for i in range(m)]
    return lens, parent, [lens[p] if c["whole"] else int(lens[p] * math.fmod((i + 0.5) * GOLD, 1.0)) for i, p in enumerate(parent)]


def _compact_held(c):
    """(pages of every sequence, pages of it that are another's: sequence b and its number of first pages)"""
    held = [_cdiv(x, c["ps"]) for x in [c["max_len"]] + _spread(c["B"] - 1, 0, c["max_len"])]
    take, every = {}, int(round(1 / c["shared"])) if c["shared"] else 0
    for b in range(1, c["B"]):
        if every and b % every == 1:
            take[b] = min(held[b], held[b - 1]) // 2
    return held, take


def _compact_pages(c):
    held, take = _compact_held(c)
    used = sum(held) - sum(take.values())
    return used, max(used + 1, int(used / c["fill"]))


# ------------------------------------------------------------------------------------------------ work
def work(c):
    op = c["op"]
    if op == "chunk":
        es, eo = ES[c["dtype"]], ES[c["out"]]
        new, lens = _chunk_lens(c)
        n_row = sum(new) * c["Hq"] * c["d"]
        kv = sum(x for x, n in zip(lens, new) if n) * c["Hkv"] * c["d"] * 2 * es
        table = sum(_cdiv(x, c["ps"]) for x, n in zip(lens, new) if n) * 4 + 8 * c["B"] + 4
        seen = sum(n * (x - n) + n * (n + 1) // 2 for x, n in zip(lens, new))
        return {"bytes": kv + table + n_row * (es * (2 if c["gate"] else 1) + eo), "flops": 4 * seen * c["Hq"] * c["d"]}
    if op == "share":
        _, _, take = _share_lens(c)
        full, part = sum(t // c["ps"] for t in take), sum(t % c["ps"] > 0 for t in take)
        # fork: shared entries read and written, their counts read and written; release: entries read, counts again
        return {"bytes": 28 * full + 40 * part + 60 * len(take), "flops": 0}
    if op == "compact":
        held, _ = _compact_held(c)
        used, pages = _compact_pages(c)
        # tables read and written; counts, map and free stack written, a pair for every page that moves
        return {"bytes": 8 * sum(held) + 8 * pages + 4 * (pages - used) + 8 * int(used * (pages - used) / pages), "flops": 0}
    return {"bytes": int(c["n"] * (1 - c["skip"])) * c["ps"] * c["Hkv"] * c["d"] * ES[c["dtype"]] * 4 + 8 * c["n"], "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _cache(g, pages, c, dt):
    """One of the two halves of a cache, seen as [page][token][head][channel]; "htd" keeps a page's heads apart."""
    shape = (pages, c["ps"], c["Hkv"], c["d"]) if c["layout"] == "thd" else (pages, c["Hkv"], c["ps"], c["d"])
    t = torch.empty(shape, device=DEV, dtype=dt)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        m = min(1 << 28, flat.numel() - i)
        flat[i:i + m] = torch.randn(m, generator=g, device=DEV, dtype=dt)
    return t if c["layout"] == "thd" else t.transpose(1, 2)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _empty(n):
    return torch.zeros(n, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g, h = dict(case), _gen(seed), torch.Generator().manual_seed(seed)
    s = {"c": c}
    if own:
        import gated_deltanet_linear_decode_gb300 as gdn
        s["gdn"] = gdn
    op = c["op"]
    if op == "chunk":
        dt, odt, ps = DT[c["dtype"]], DT[c["out"]], c["ps"]
        new, lens = _chunk_lens(c)
        order = torch.randperm(c["B"], generator=h).tolist()
        new, lens = [new[i] for i in order], [lens[i] for i in order]
        held = [_cdiv(x, ps) for x in lens]
        pages = sum(held) + 3
        perm, table, at = torch.randperm(pages, generator=h).to(torch.int32), torch.zeros(c["B"], max(held) + 1, dtype=torch.int32), 0
        for b, n in enumerate(held):
            table[b, :n] = perm[at:at + n]
            at += n
        s["table"], s["lens"], s["new"], s["host_lens"] = table.to(DEV), _i32(lens), new, lens
        s["cu"] = _i32([0] + np.cumsum(new).tolist())
        s["k"], s["v"] = _cache(g, pages, c, dt), _cache(g, pages, c, dt)
        T = sum(new) + c["pad"]
        # normalised heads with learned weights somewhat above one: scores of a few units
        s["q"] = _randn(g, T, c["Hq"] * c["d"], dtype=dt, scale=1.5)
        s["gate"] = _randn(g, T, c["Hq"] * c["d"], dtype=dt) if c["gate"] else None
        s["out"] = torch.zeros(T, c["Hq"] * c["d"], device=DEV, dtype=odt)
        if own:
            s["dims"] = gdn.make_attn_dims(c["Hq"], c["Hkv"], c["d"], dt, odt)
            s["cache"] = gdn.KvCache(s["k"], s["v"])
            s["ws"] = torch.zeros(gdn.gdn_attn_chunk_workspace_bytes(s["dims"], c["B"], T), device=DEV, dtype=torch.uint8)
    elif op == "share":
        ps, n, m = c["ps"], c["parents"], c["children"]
        lens, parent, take = _share_lens(c)
        held = [_cdiv(x, ps) for x in lens]
        pages = sum(held) + m + 20
        perm, at = torch.randperm(pages, generator=h).to(torch.int32), sum(held)
        # the parents lie anywhere among the sequences
        where = torch.randperm(n + m, generator=h).tolist()
        child = sorted(where[n:])
        table = torch.zeros(n + m, max(held) + 1, dtype=torch.int32)
        len_, held_, got = [0] * (n + m), [0] * (n + m), 0
        for i in range(n):
            table[where[i], :held[i]] = perm[got:got + held[i]]
            got += held[i]
            len_[where[i]], held_[where[i]] = lens[i], held[i]
        mixed = torch.randperm(m, generator=h).tolist()
        s["src"], s["dst"] = _i32([where[parent[i]] for i in mixed]), _i32(child)
        s["take"] = _i32([take[i] for i in mixed])
        s["table"], s["lens"], s["held"], s["keep"] = table.to(DEV), _i32(len_), _i32(held_), _i32(len_)
        s["free"] = torch.cat([perm[at:], torch.zeros(at, dtype=torch.int32)]).to(DEV)
        s["n_free"] = _i32([pages - at])
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["fork_src"], s["fork_dst"] = _empty(m), _empty(m)
        s["rel_src"], s["rel_dst"] = _empty(n + m), _empty(n + m)
    elif op == "compact":
        held, take = _compact_held(c)
        _, pages = _compact_pages(c)
        perm, at = torch.randperm(pages, generator=h).to(torch.int32), 0
        table = torch.zeros(c["B"], max(held) + 1, dtype=torch.int32)
        for b, x in enumerate(held):
            t = take.get(b, 0)
            table[b, :t] = table[b - 1, :t]
            table[b, t:x] = perm[at:at + x - t]
            at += x - t
        s["table"], s["held"], s["pages"] = table.to(DEV), _i32(held), pages
        s["table_out"] = s["table"].clone()
        s["refs"], s["free"], s["map"], s["n_free"], s["n_copy"] = _empty(pages), _empty(pages), _empty(pages), _empty(1), _empty(1)
        s["src"], s["dst"] = _empty(max(1, pages // 2)), _empty(max(1, pages // 2))
    else:
        dt = DT[c["dtype"]]
        s["k"], s["v"] = _cache(g, c["pages"], c, dt), _cache(g, c["pages"], c, dt)
        perm = torch.randperm(c["pages"], generator=h).to(torch.int32)
        src, dst = perm[:c["n"]].clone(), perm[c["n"]:2 * c["n"]].clone()
        gone = torch.randperm(c["n"], generator=h)[: c["n"] - int(c["n"] * (1 - c["skip"]))]
        src[gone] = -1
        dst[gone] = -1
        s["src"], s["dst"] = src.to(DEV), dst.to(DEV)
        if own:
            s["dims"] = gdn.make_attn_dims(c["Hkv"], c["Hkv"], c["d"], dt, dt)
            s["cache"] = gdn.KvCache(s["k"], s["v"])
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _OWN[op](s, s["gdn"])
    return _PLAIN[op](s)


def _own_chunk(s, gdn):
    gdn.gdn_attn_chunk(s["dims"], s["cache"], s["q"], s["cu"], s["table"], s["lens"], s["out"], gate=s["gate"], workspace=s["ws"])
    return s["out"]


def _shared(s):
    return {k: s[k] for k in ("table", "lens", "held", "free", "n_free", "refs", "fork_src", "fork_dst", "rel_src", "rel_dst")}


def _own_share(s, gdn):
    ps = s["c"]["ps"]
    gdn.gdn_kv_fork(ps, s["src"], s["dst"], s["take"], s["lens"], s["held"], s["table"], s["refs"], s["free"], s["n_free"],
                    s["fork_src"], s["fork_dst"])
    gdn.gdn_kv_release(ps, s["keep"], s["lens"], s["held"], s["table"], s["refs"], s["free"], s["n_free"], s["rel_src"],
                       s["rel_dst"])
    return _shared(s)


def _compacted(s):
    return {k: s[k] for k in ("table_out", "refs", "n_free", "map", "src", "dst", "n_copy", "free")}


def _own_compact(s, gdn):
    gdn.gdn_kv_compact(s["held"], s["table"], s["refs"], s["free"], s["n_free"], s["map"], s["src"], s["dst"], s["n_copy"],
                       block_table_out=s["table_out"])
    return _compacted(s)


def _own_copy(s, gdn):
    gdn.gdn_kv_copy_pages(s["dims"], s["cache"], s["src"], s["dst"])
    return {"k": s["k"], "v": s["v"]}


_OWN = {"chunk": _own_chunk, "share": _own_share, "compact": _own_compact, "copy": _own_copy}


def _plain_chunk(s):
    c = s["c"]
    Hq, Hkv, d, ps, at = c["Hq"], c["Hkv"], c["d"], c["ps"], 0
    G, out = Hq // Hkv, s["out"]
    for b, n in enumerate(s["new"]):
        if n == 0:
            continue
        L = s["host_lens"][b]
        j = torch.arange(L, device=DEV)
        page = s["table"].long()[b, j // ps]
        q = s["q"][at:at + n].float().view(n, Hkv, G, d)
        seen = j < (L - n + 1 + torch.arange(n, device=DEV))[:, None]                   # [n][L]
        for h in range(Hkv):
            k, v = s["k"][page, j % ps, h].float(), s["v"][page, j % ps, h].float()     # [L][d]
            sc = torch.matmul(q[:, h].transpose(0, 1), k.t()) * (1.0 / math.sqrt(d))    # [G][n][L]
            sc = torch.where(seen, sc, float("-inf"))
            m = sc.amax(-1, keepdim=True)
            e = torch.exp(sc - torch.where(m == float("-inf"), 0.0, m))
            z = e.sum(-1, keepdim=True)
            o = torch.matmul(e, v) / torch.where(z == 0, 1.0, z)                        # [G][n][d]
            del sc, e
            o = o.transpose(0, 1).reshape(n, G * d)
            if s["gate"] is not None:
                o = o / (1 + torch.exp(-s["gate"][at:at + n, h * G * d:(h + 1) * G * d].float()))
            out[at:at + n, h * G * d:(h + 1) * G * d] = o.to(out.dtype)
        at += n
    return out


def _plain_share(s):
    ps, table, refs, free = s["c"]["ps"], s["table"], s["refs"], s["free"]
    src, dst, take = s["src"].long(), s["dst"].long(), s["take"].long()
    i32, P = torch.int32, table.shape[1]
    col, n = torch.arange(P, device=DEV), s["n_free"].long()
    # forked: the full pages of the parent, a fresh page for what is left
    full, part = take // ps, (take % ps > 0).long()
    nth = part.cumsum(0) - part
    fresh = free[(n - 1 - nth).clamp(min=0)]
    old = table[src]
    shared = col < full[:, None]
    last = (col == full[:, None]) & (part[:, None] > 0)
    table[dst] = torch.where(shared, old, torch.where(last, fresh[:, None], table[dst]))
    refs.index_add_(0, old[shared].long(), torch.ones_like(old[shared]))
    s["fork_src"].copy_(torch.where(part > 0, old.gather(1, full[:, None])[:, 0], -1))
    s["fork_dst"].copy_(torch.where(part > 0, fresh, -1))
    s["lens"][dst] = take.to(i32)
    s["held"][dst] = (full + part).to(i32)
    s["n_free"].sub_(part.sum().to(i32))
    # released: every page past the new length loses a holder, and so does a kept one that is not full and not its own, which
    # a fresh page takes the place of; pages without a holder go back, the first in order on top
    keep, held, n = s["keep"].long(), s["held"].long(), s["n_free"].long()
    stay = (keep + ps - 1) // ps
    at = (keep // ps).clamp(max=P - 1)[:, None]
    kept = table.gather(1, at)[:, 0]
    own_page = ((keep % ps > 0) & (refs[kept.long()] > 0)).long()
    nth = own_page.cumsum(0) - own_page
    fresh = free[(n - 1 - nth).clamp(min=0)]
    s["rel_src"].copy_(torch.where(own_page > 0, kept, -1))
    s["rel_dst"].copy_(torch.where(own_page > 0, fresh, -1))
    gone = (col >= (stay - own_page)[:, None]) & (col < held[:, None])
    page = table[gone].long()                                                           # in order
    table.scatter_(1, at, torch.where(own_page > 0, fresh, kept)[:, None])
    n = n - own_page.sum()
    refs.index_add_(0, page, torch.full_like(page, -1, dtype=i32))
    order = torch.arange(page.numel(), device=DEV)
    first = torch.full((refs.numel(),), page.numel(), device=DEV).scatter_reduce_(0, page, order, "amin")
    back = page[(refs[page] < 0) & (first[page] == order)]
    refs.clamp_(min=0)
    free[n + back.numel() - 1 - torch.arange(back.numel(), device=DEV)] = back.to(i32)
    s["n_free"].copy_((n + back.numel()).to(i32))
    s["held"].copy_(stay.to(i32))
    s["lens"].copy_(keep.to(i32))
    return _shared(s)


def _plain_compact(s):
    table, N, i32 = s["table"], s["pages"], torch.int32
    held = torch.arange(table.shape[1], device=DEV) < s["held"].long()[:, None]
    count = torch.bincount(table[held].long(), minlength=N)
    used, page = count > 0, torch.arange(N, device=DEV)
    n_used = used.sum()
    hole, moves = page[~used & (page < n_used)], page[used & (page >= n_used)].flip(0)
    new = torch.where(used, page, -1)
    new[moves] = hole
    s["map"].copy_(new.to(i32))
    s["src"].fill_(-1)
    s["dst"].fill_(-1)
    s["src"][: moves.numel()] = moves.to(i32)
    s["dst"][: hole.numel()] = hole.to(i32)
    s["n_copy"].fill_(moves.numel())
    refs = torch.zeros(N, dtype=torch.int64, device=DEV)
    refs[new[used]] = count[used] - 1
    s["refs"].copy_(refs.to(i32))
    s["table_out"].copy_(torch.where(held, new[table.long()].to(i32), s["table_out"]))
    s["n_free"].copy_((N - n_used).to(i32))
    s["free"].copy_(torch.where(page < N - n_used, N - 1 - page, s["free"].long()).to(i32))
    return _compacted(s)


def _plain_copy(s):
    there = s["src"] >= 0
    src, dst = s["src"][there].long(), s["dst"][there].long()
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    return {"k": s["k"], "v": s["v"]}


_PLAIN = {"chunk": _plain_chunk, "share": _plain_share, "compact": _plain_compact, "copy": _plain_copy}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "chunk":
        d, ps, Hq, Hkv = c["d"], c["ps"], c["Hq"], c["Hkv"]
        G, T, at = Hq // Hkv, s["q"].shape[0], 0
        out = torch.zeros(T, Hq, d, dtype=torch.float64, device=DEV)
        lens, table = s["lens"].tolist(), s["table"].long()
        q = s["q"].view(T, Hq, d)
        for b, n in enumerate(s["new"]):
            L = lens[b]
            slot = (table[b, : _cdiv(L, ps), None] * ps + torch.arange(ps, device=DEV)).reshape(-1)[:L]
            for h in range(Hkv if n else 0):
                kh, vh = s["k"][slot // ps, slot % ps, h].double(), s["v"][slot // ps, slot % ps, h].double()
                step = max(1, int(2e8 / (8 * L * G)))
                for p in range(0, n, step):
                    m = min(step, n - p)
                    last = L - n + p + m                                   # keys that the last row of these sees
                    w = torch.einsum("pgd,jd->pgj", q[at + p:at + p + m, h * G:(h + 1) * G].double(), kh[:last]) / math.sqrt(d)
                    hide = torch.ones(m, last, dtype=torch.bool, device=DEV).triu(L - n + p + 1)
                    w = torch.softmax(w.masked_fill(hide[:, None], -math.inf), -1)
                    out[at + p:at + p + m, h * G:(h + 1) * G] = torch.einsum("pgj,jd->pgd", w, vh[:last])
            at += n
        out = out.view(T, -1)
        return out * torch.sigmoid(s["gate"].double()) if c["gate"] else out
    if op == "share":
        ps, n = c["ps"], int(s["n_free"])
        table, refs, free = s["table"].tolist(), s["refs"].tolist(), s["free"].tolist()
        lens, held = s["lens"].tolist(), s["held"].tolist()
        cs, cd = [], []
        for a, b, t in zip(s["src"].tolist(), s["dst"].tolist(), s["take"].tolist()):
            row = []
            for i in range(t // ps):
                row.append(table[a][i])
                refs[table[a][i]] += 1
            cs.append(-1)
            cd.append(-1)
            if t % ps:
                n -= 1
                row.append(free[n])
                cs[-1], cd[-1] = table[a][t // ps], free[n]
            table[b][:len(row)] = row
            lens[b], held[b] = t, len(row)
        given = []                         # pages without a holder, in the order in which their first holder gives them up
        children = set(s["dst"].tolist())
        left = {}
        for b in sorted(children):
            for g in table[b][:held[b]]:
                left.setdefault(g, refs[g] + 1)
                left[g] -= 1
            lens[b] = 0
        for g, x in left.items():
            refs[g] = max(0, x - 1)
            if x == 0:
                given.append(g)
        for b in children:
            held[b] = 0
        for g in reversed(given):
            free[n] = g
            n += 1
        none = [-1] * len(lens)
        out = {"table": table, "lens": lens, "held": held, "free": free, "n_free": [n], "refs": refs, "fork_src": cs, "fork_dst": cd,
               "rel_src": none, "rel_dst": none}
        return {k: np.array(v, dtype=np.int32) for k, v in out.items()}
    if op == "compact":
        table, held, N = s["table"].tolist(), s["held"].tolist(), s["pages"]
        out, count = s["table_out"].tolist(), [0] * N
        for b, x in enumerate(held):
            for g in table[b][:x]:
                count[g] += 1
        n = sum(x > 0 for x in count)
        move = {g: g for g in range(N) if count[g]}
        src, dst, high = [], [], N - 1
        for g in range(n):
            if count[g] == 0:              # the lowest hole takes the highest page
                while count[high] == 0:
                    high -= 1
                move[high] = g
                src.append(high)
                dst.append(g)
                high -= 1
        refs = [0] * N
        for g, to in move.items():
            refs[to] = count[g] - 1
        for b, x in enumerate(held):
            out[b][:x] = [move[g] for g in table[b][:x]]
        pad = [-1] * (s["src"].numel() - len(src))
        free = s["free"].tolist()
        free[: N - n] = range(N - 1, n - 1, -1)
        res = {"table_out": out, "refs": refs, "n_free": [N - n], "map": [move.get(g, -1) for g in range(N)], "src": src + pad,
               "dst": dst + pad, "n_copy": [len(src)], "free": free}
        return {k: np.array(v, dtype=np.int32) for k, v in res.items()}
    k, v = s["k"].clone(), s["v"].clone()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        if a >= 0:
            k[b].copy_(s["k"][a])
            v[b].copy_(s["v"][a])
    return {"k": k, "v": v}
