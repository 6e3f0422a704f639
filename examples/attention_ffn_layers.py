"""Layers of attention and token-indexed FFN: trained for a few steps on packed
documents, then served from a paged key-value cache.

    python examples/attention_ffn_layers.py [--dtype bf16|f32] [--steps 20]

Training joins staple_attn_fwd and staple_attn_bwd with the FFN's calls in
torch's autograd.  Serving prefills prompts of different lengths into pages
(staple_kv_extend, staple_attn_fwd, staple_kv_append), decodes token by token
(staple_attn_decode_paged), forks a sequence into beams that share its pages
until they write, ends sequences, packs the pool and goes on decoding.  The
logits of every served token are checked against one pass over whole sequences.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import token_indexed_ffn_amd as st  # noqa: E402

LAYERS, D_MODEL, D_FF, VOCAB = 2, 256, 512, 1000
HEADS, KV_HEADS, HEAD_DIM = 4, 2, 64
MASK = dict(window=48, sinks=4)
PAGE = 16


class Attention(torch.autograd.Function):
    """q, k, v are slices of one projection, read in place; so are its gradient's."""

    @staticmethod
    def forward(ctx, qkv, cu):
        q, k, v = heads_of(qkv)
        out = st.staple_attn_fwd(q, k, v, cu, cu, **MASK)
        ctx.save_for_backward(qkv, cu, out["o"], out["lse"])
        return out["o"].view(len(qkv), -1)

    @staticmethod
    def backward(ctx, do):
        qkv, cu, o, lse = ctx.saved_tensors
        grad = torch.empty_like(qkv)
        dq, dk, dv = heads_of(grad)
        st.staple_attn_bwd(do.contiguous().view_as(o), *heads_of(qkv), o, lse, cu, cu,
                           out={"dq": dq, "dk": dk, "dv": dv}, **MASK)
        return grad, None


class TokenFFN(torch.autograd.Function):
    """Weights and the table's rows of the batch's unique tokens in fp32, products in x's type."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, rows, batch):
        w = [t.to(x.dtype) for t in (w_gate, w_up, w_down)]
        out = st.staple_ffn_fwd(x, *w, rows.to(x.dtype), batch["inv"], save=True)
        ctx.save_for_backward(x, *w, out["g"], out["u"], out["h"])
        ctx.batch, ctx.n_rows = batch, len(rows)
        return out["y"]

    @staticmethod
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, g, u, h = ctx.saved_tensors
        b = ctx.batch
        d = st.staple_ffn_bwd_table_grad(dy.contiguous(), x, w_gate, w_up, w_down, g, u, h, b["sorted_pos"],
                                         b["seg_start"], b["n_unique"], inv=b["inv"])
        return d["dx"], d["dw_gate"], d["dw_up"], d["dw_down"], d["d_rows"][:ctx.n_rows], None


def heads_of(qkv):
    t = qkv.view(len(qkv), HEADS + 2 * KV_HEADS, HEAD_DIM)
    return t[:, :HEADS], t[:, HEADS:HEADS + KV_HEADS], t[:, HEADS + KV_HEADS:]


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(dim=1, keepdim=True) + 1e-6)).to(x.dtype)


def offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


class Model:
    def __init__(self, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) * cols ** -0.5).cuda().requires_grad_()

        self.dtype = dtype
        self.embed = weight(VOCAB, D_MODEL)
        width = (HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.layers = [dict(qkv=weight(width, D_MODEL), o=weight(D_MODEL, HEADS * HEAD_DIM), gate=weight(D_FF, D_MODEL),
                            up=weight(D_FF, D_MODEL), down=weight(D_MODEL, D_FF), table=weight(VOCAB, D_FF))
                       for _ in range(LAYERS)]

    def parameters(self):
        return [self.embed] + [w for layer in self.layers for w in layer.values()]

    def forward(self, ids, cu):
        """Logits of packed sequences."""
        batch = st.staple_dedup(ids, VOCAB)
        uniq = batch["uniq"][:int(batch["n_unique"])].long()
        x = self.embed[ids.long()].to(self.dtype)
        for layer in self.layers:
            x = x + Attention.apply(norm(x) @ layer["qkv"].to(x.dtype).T, cu) @ layer["o"].to(x.dtype).T
            x = x + TokenFFN.apply(norm(x), layer["gate"], layer["up"], layer["down"], layer["table"][uniq], batch)
        return norm(x).float() @ self.embed.T


def train(model, steps):
    """Next-token loss on documents of odd lengths; the same documents every step."""
    lens = [130, 1, 77, 200, 33]
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(VOCAB, (sum(lens),), generator=gen, dtype=torch.int32).cuda()
    cu = offsets(lens)
    target = torch.roll(ids.long(), -1)
    target[cu[1:].long() - 1] = -100   # a document's last token has no next one
    adam = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        loss = torch.nn.functional.cross_entropy(model.forward(ids, cu), target, ignore_index=-100)
        adam.zero_grad()
        loss.backward()
        adam.step()
        losses.append(float(loss.detach()))
    return losses


class Server:
    """One pool of pages for all layers and one table row for each sequence."""

    def __init__(self, model, rows=8, pages=96, max_pages=16):
        self.model, t = model, model.dtype
        shape = (LAYERS, pages, KV_HEADS, PAGE, HEAD_DIM)
        self.k, self.v = torch.zeros(shape, dtype=t, device="cuda"), torch.zeros(shape, dtype=t, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.book = (self.refs, self.table, self.lens)
        # rows that the last growth left as they are: no new token of theirs is written
        self.refused = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.layers = []
        for layer in model.layers:
            w = {n: x.detach().to(t).contiguous() for n, x in layer.items()}
            if t == torch.bfloat16:   # the decode kernels' own order
                w["packed"] = st.staple_decode_pack_weights(w["gate"], w["up"], w["down"], d_model=D_MODEL, d_ff=D_FF)
            self.layers.append(w)

    def ffn(self, w, x, ids):
        if "packed" in w and len(ids) <= 64:
            return st.staple_ffn_fwd_packed(x, *w["packed"], w["table"], ids, d_ff=D_FF)["y"]
        return st.staple_ffn_fwd(x, w["gate"], w["up"], w["down"], w["table"], ids)["y"]

    def run(self, ids, attend):
        """Logits of new tokens; attend: (layer, q, k, v) -> o."""
        x = self.model.embed.detach()[ids.long()].to(self.model.dtype)
        for i, w in enumerate(self.layers):
            o = attend(i, *heads_of(norm(x) @ w["qkv"].T))
            x = x + o.reshape(len(ids), -1) @ w["o"].T
            x = x + self.ffn(w, norm(x), ids)
        return norm(x).float() @ self.model.embed.detach().T

    def prefill(self, seqs, prompts):
        lens = [len(p) for p in prompts]
        cu, rows = offsets(lens), torch.tensor(seqs, dtype=torch.int32, device="cuda")
        st.staple_kv_extend(*self.book, rows, torch.tensor(lens, dtype=torch.int32, device="cuda"), k_pages=self.k,
                            v_pages=self.v, refused=self.refused)

        def attend(i, q, k, v):
            st.staple_kv_append(k, v, self.k[i], self.v[i], self.table, self.lens, rows, cu, refused=self.refused)
            return st.staple_attn_fwd(q, k, v, cu, cu, **MASK)["o"]

        return self.run(torch.cat(prompts), attend)[cu[1:].long() - 1]

    def decode(self, seqs, ids):
        """One more token for each sequence."""
        rows = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        st.staple_kv_extend(*self.book, rows, k_pages=self.k, v_pages=self.v, refused=self.refused)

        def attend(i, q, k, v):
            return st.staple_attn_decode_paged(q, self.k[i], self.v[i], self.table, self.lens, seqs=rows, k_new=k, v_new=v,
                                               refused=self.refused, **MASK)["o"]

        return self.run(ids, attend)

    def fork(self, parents, children):
        st.staple_kv_fork(*self.book, torch.tensor(parents, dtype=torch.int32, device="cuda"),
                          torch.tensor(children, dtype=torch.int32, device="cuda"), page_size=PAGE, refused=self.refused)

    def free(self, seqs):
        st.staple_kv_free(*self.book, torch.tensor(seqs, dtype=torch.int32, device="cuda"), page_size=PAGE,
                          refused=self.refused)

    def compact(self):
        return int(st.staple_kv_compact(*self.book, self.k, self.v)["n_live"])


@torch.no_grad()
def serve(model, steps=20):
    """Greedy decoding of four prompts, then beams of the longest; returns the largest difference from a
    pass over the whole sequences, relative to the largest logit, and the pages in use at the end."""
    server = Server(model)
    gen = torch.Generator().manual_seed(2)
    text = {s: torch.randint(VOCAB, (n,), generator=gen, dtype=torch.int32).cuda() for s, n in enumerate((1, 47, 90, 16))}
    logits = {}   # of each sequence's next token

    def keep(seqs, out):
        logits.update(zip(seqs, out))

    def step(seqs, rank=lambda s: 0):
        """Each sequence goes on with its best token, or the one of that rank."""
        ids = torch.stack([logits[s].topk(rank(s) + 1).indices[-1] for s in seqs]).int()
        for s, t in zip(seqs, ids):
            text[s] = torch.cat((text[s], t.view(1)))
        keep(seqs, server.decode(seqs, ids))

    def worst():
        seqs = sorted(logits)
        cu = offsets([len(text[s]) for s in seqs])
        whole = model.forward(torch.cat([text[s] for s in seqs]), cu)[cu[1:].long() - 1]
        served = torch.stack([logits[s] for s in seqs])
        return float((served - whole).abs().max() / whole.abs().max())

    keep(list(text), server.prefill(list(text), list(text.values())))
    error = worst()
    for _ in range(steps):
        step(sorted(logits))
    error = max(error, worst())
    beams = [4, 5, 6]
    server.fork([2] * len(beams), beams)
    for b in beams:
        text[b], logits[b] = text[2], logits[2]
    step(beams, rank=lambda s: s - 4)   # a page of its own for each from here on
    gone = [0, 2]
    server.free(gone)
    for s in gone:
        del text[s], logits[s]
    live = server.compact()
    for _ in range(steps):
        step(sorted(logits))
    error = max(error, worst())
    if st.staple_get_device_error() != 0:
        raise RuntimeError("device error word set")
    return error, live


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args(argv)
    model = Model(torch.bfloat16 if args.dtype == "bf16" else torch.float32)
    losses = train(model, args.steps)
    print(f"training loss {losses[0]:.3f} -> {losses[-1]:.3f} in {args.steps} steps")
    error, live = serve(model)
    print(f"served logits within {error:.2e} of a whole pass, {live} pages in use after compaction")
    return losses, error, live


if __name__ == "__main__":
    main()
