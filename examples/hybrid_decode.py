"""Two layers of a hybrid stack decoding together: a gated DeltaNet layer and a full-attention layer, each between its
norms, on random weights.

  python examples/hybrid_decode.py [--batch 8] [--steps 32] [--verify 3]

A step gives every sequence one token (or, with --verify K, K drafted tokens of which a random number is accepted):
page bookkeeping for the new tokens, the DeltaNet layer (norm, projections, recurrent step or verify walk, projection),
the attention layer (norm, projection, cache append, attention over the paged cache, projection), and after a verify the
commit of the state and the truncation of the cache.  Lengths, block tables and slots stay on the device, so the plain
decode step is captured once and replayed as a CUDA graph.

gdn_kv_extend packs the rows of the sequences that it gives tokens, while the other calls have row b*K + p for token p of
sequence b: the slots and positions are brought to those rows on the device, -1 where a sequence was refused (its table is
full, or the pages are out).  A refused sequence keeps its cache and, after a verify, its state; its outputs mean nothing,
`status` names it, and it has to leave the batch before the next step.  The others are not touched by it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_decode_gb300 as gdn  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class HybridDecoder:
    """Hidden size H; a DeltaNet layer of Hk/Hv heads; an attention layer of Hq/Hkv heads of D with a paged cache."""

    def __init__(self, B, K=1, H=2048, Hk=16, Hv=32, Hq=16, Hkv=2, D=256, rope=64, page_size=16, max_len=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s, scale=1.0, dt=BF: (torch.randn(*s, generator=g, device="cuda") * scale).to(dt)
        z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")
        self.B, self.K, self.T, self.H, self.ps = B, K, B * K, H, page_size
        T, C, inner, nq, nk = self.T, 128 * (2 * Hk + Hv), 128 * Hv, Hq * D, Hkv * D
        ones = lambda n: 1 + 0.1 * torch.randn(n, generator=g, device="cuda")
        # the DeltaNet layer
        self.gd = gdn.make_dims(Hk, Hv, BF, BF)
        self.w = gdn.make_weights(rn(C, 4, scale=0.25, dt=F32), rn(Hv, dt=F32), -torch.exp(rn(Hv, dt=F32)), ones(128))
        self.W_in = [rn(n, H, scale=H ** -0.5) for n in (C, inner, Hv, Hv)]
        self.W_out = rn(H, inner, scale=inner ** -0.5)
        self.conv, self.S = z(B, 3, C), z(B, Hv, 128, 128, dt=F32)
        if K > 1:
            self.conv_ck, self.S_ck = z(B, K, 3, C), z(B, K, Hv, 128, 128, dt=F32)
        self.x, self.z, self.a, self.b, self.y = z(T, C), z(T, inner), z(T, Hv), z(T, Hv), z(T, inner)
        # the attention layer: one projection for q, k, v and the output gate
        self.ad = gdn.make_attn_dims(Hq, Hkv, D, BF, BF, rope_dim=rope)
        self.W_qkvg, self.W_o = rn(2 * nq + 2 * nk, H, scale=H ** -0.5), rn(H, nq, scale=nq ** -0.5)
        self.q_w, self.k_w = ones(D), ones(D)
        ang = torch.arange(max_len, device="cuda").double()[:, None] * 1e7 ** (-2 * torch.arange(rope // 2, device="cuda").double() / rope)
        self.cos, self.sin = ang.cos().float(), ang.sin().float()
        per_seq = -(-max_len // page_size)
        pages = B * per_seq
        self.kv = gdn.KvCache(z(pages, page_size, Hkv, D), z(pages, page_size, Hkv, D))
        self.table, self.free = z(B, per_seq, dt=I32), torch.randperm(pages, generator=g, device="cuda").to(I32)
        self.n_free, self.lens, self.held = torch.full((1,), pages, dtype=I32, device="cuda"), z(B, dt=I32), z(B, dt=I32)
        self.n_new, self.cu = torch.full((B,), K, dtype=I32, device="cuda"), z(B + 1, dt=I32)
        # slots and positions as gdn_kv_extend packs them, with an entry T for rows that a sequence does not have; then by row b*K + p
        width = -(-(T + 1) // 4) * 4
        self.packed, self.by_row, self.at = z(2, width, dt=I32), z(2, width, dt=I32), torch.full((width,), T, dtype=I32, device="cuda")
        self.packed[0, T] = -1
        self.slots, self.pos = self.packed[0, :T], self.packed[1, :T]
        self.token, self.nowhere = torch.arange(K, dtype=I32, device="cuda"), self.at[T]
        self.qkvg, self.q, self.o, self.status = z(T, 2 * nq + 2 * nk), z(T, nq), z(T, nq), z(B, dt=I32)
        self.cuts = (nq, nq + nk, nq + 2 * nk)
        self.ws = z(gdn.gdn_attn_decode_workspace_bytes(self.ad, B, K), dt=torch.uint8)
        # residual stream and norms
        self.nd = gdn.make_norm_dims(H, BF, F32)
        self.pre = [ones(H) for _ in range(3)]
        self.hidden, self.h, self.xn, self.d = z(T, H), z(T, H, dt=F32), z(T, H), z(T, H)

    def step(self):
        """self.hidden [B*K][H] (the tokens' embeddings) -> self.xn (normed output of the two layers)."""
        nd, K = self.nd, self.K
        gdn.gdn_kv_extend(self.ps, self.n_new, self.lens, self.held, self.table, self.free, self.n_free, self.slots, self.pos,
                          self.cu, dev_status=self.status)
        row = self.cu[:-1, None] + self.token               # where sequence b's token p is in the packed rows, if it is
        torch.where(row < self.cu[1:, None], row, self.nowhere, out=self.at[:self.T].view(self.B, K))
        torch.index_select(self.packed, 1, self.at, out=self.by_row)
        self.h.copy_(self.hidden)
        gdn.gdn_norm_residual(nd, self.h, pre_w=self.pre[0], x=self.xn)
        gdn.gdn_in_proj(self.gd, self.xn, *self.W_in, self.x, self.z, self.a, self.b)
        if K == 1:
            gdn.gdn_decode_step(self.gd, self.w, self.x, self.z, self.a, self.b, self.conv, self.S, self.y)
        else:
            gdn.gdn_verify_k(self.gd, self.w, K, self.x, self.z, self.a, self.b, self.conv, self.S, self.conv_ck, self.S_ck, self.y)
        gdn.gdn_out_proj(self.gd, self.y, self.W_out, self.d)
        gdn.gdn_norm_residual(nd, self.h, self.h, y=self.d, pre_w=self.pre[1], x=self.xn)
        torch.matmul(self.xn, self.W_qkvg.t(), out=self.qkvg)
        a, b, c = self.cuts
        gdn.gdn_kv_append(self.ad, self.kv, self.qkvg[:, :a], self.qkvg[:, a:b], self.qkvg[:, b:c], self.by_row[1, :self.T],
                          self.by_row[0, :self.T], self.q, q_norm_w=self.q_w, k_norm_w=self.k_w, rope_cos=self.cos, rope_sin=self.sin)
        gdn.gdn_attn_decode(self.ad, self.kv, K, self.q, self.table, self.lens, self.o, gate=self.qkvg[:, c:], workspace=self.ws,
                            dev_status=self.status)
        torch.matmul(self.o, self.W_o.t(), out=self.d)
        gdn.gdn_norm_residual(nd, self.h, self.h, y=self.d, pre_w=self.pre[2], x=self.xn)

    def commit(self, accept):
        """After a step of K > 1: keep accept[b] of the drafted tokens, in the state and in the cache; a sequence that the step
        refused stays as it was."""
        added = self.cu.diff()
        accept = torch.minimum(accept, added)               # 0 leaves the state as it is
        gdn.gdn_commit(self.gd, self.K, accept, self.conv_ck, self.S_ck, self.conv, self.S)
        gdn.gdn_kv_truncate(self.ps, self.lens - (added - accept), self.lens, self.held, self.table, self.free, self.n_free,
                            dev_status=self.status)

    def capture(self):
        """The decode step as a graph (run once before, so that everything is loaded)."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--verify", type=int, default=1, help="drafted tokens a step")
    args = ap.parse_args()
    m = HybridDecoder(args.batch, args.verify)
    graph = None
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(args.steps):
        m.hidden.normal_()
        if i == 1:
            start.record()
        if graph:
            graph.replay()
        else:
            m.step()
        if args.verify > 1:
            m.commit(torch.randint(1, args.verify + 1, (args.batch,), device="cuda", dtype=I32))
        elif graph is None:
            graph = m.capture()   # a capture runs nothing
    end.record()
    torch.cuda.synchronize()
    assert int(m.status.max()) == 0 and bool(torch.isfinite(m.xn.float()).all())
    print(f"{args.batch} sequences, {args.steps} steps, lengths {int(m.lens.min())}..{int(m.lens.max())}: "
          f"{start.elapsed_time(end) / max(1, args.steps - 1) * 1000:.1f} us a step")


if __name__ == "__main__":
    main()
