"""The attention operators' measured cases: attention with a sliding window and sinks (forward and
backward), attention of one new token over a paged key-value cache, and the cache's page operations.

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, with the
framework's entry points.  The mask of all attention cases: a sequence's query i stands at position
p = i + Lk - Lq and sees key j when j <= p and (window == 0 or j > p - window or j < sinks).
"""
import math
import random

import numpy as np
import torch


own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"

# The drawn cases' bounds: score-matrix elements of the dense plain form, bytes of a page pool pair.
MOST_SCORES = 2.2e9
MOST_POOL = 2.2e9


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a step of a small fp32 model, the size of its unit workload: 512 tokens in ragged documents
        dict(name="train_f32_512tok", op="window", train=True, dtype="f32", seqs=5, q_lo=1, q_hi=250, past_lo=0,
             past_hi=0, heads=4, kv_heads=4, dim=64, window=100, sinks=4, ragged=1),
        # the serving table's prefill: 64 prompts of 256 tokens, 16 heads of 128 (a d_model of 2048)
        dict(name="prefill_64x256", op="window", train=False, dtype="bf16", seqs=64, q_lo=256, q_hi=256, past_lo=0,
             past_hi=0, heads=16, kv_heads=16, dim=128, window=0, sinks=0, ragged=0),
        # later chunks of long prompts: 2048 new tokens after up to 14000 cached ones, grouped heads
        dict(name="prefill_chunk_past", op="window", train=False, dtype="bf16", seqs=4, q_lo=1024, q_hi=2048,
             past_lo=2001, past_hi=14000, heads=32, kv_heads=8, dim=128, window=4096, sinks=4, ragged=2),
        # the training batch of 8 x 4096 tokens, 16 heads of 128, a window of a quarter of the sequence
        dict(name="train_8x4096_window", op="window", train=True, dtype="bf16", seqs=8, q_lo=4096, q_hi=4096,
             past_lo=0, past_hi=0, heads=16, kv_heads=16, dim=128, window=1024, sinks=4, ragged=0),
        # packed documents of odd lengths, full causal attention, grouped heads: the training step's largest work
        dict(name="train_ragged_causal", op="window", train=True, dtype="bf16", seqs=6, q_lo=700, q_hi=4096,
             past_lo=0, past_hi=0, heads=32, kv_heads=8, dim=128, window=0, sinks=0, ragged=4),
        # one user's next token early in a chat: latency alone
        dict(name="decode_1x37", op="decode", dtype="bf16", seqs=1, len_lo=37, len_hi=37, heads=16, kv_heads=16,
             dim=128, page=16, window=0, sinks=0, ragged=0),
        # the decode step of 64 sequences around a context of 256, 16 heads of 128
        dict(name="decode_64x256", op="decode", dtype="bf16", seqs=64, len_lo=192, len_hi=320, heads=16, kv_heads=16,
             dim=128, page=16, window=0, sinks=0, ragged=1),
        # the same batch deep in long chats, grouped heads, a window and sinks over scattered pages
        dict(name="decode_64_window", op="decode", dtype="bf16", seqs=64, len_lo=1, len_hi=8192, heads=32, kv_heads=8,
             dim=128, page=32, window=1024, sinks=4, ragged=2),
        # two very long contexts, everything visible: the cache is split along its length
        dict(name="decode_2x131071", op="decode", dtype="bf16", seqs=2, len_lo=100001, len_hi=131071, heads=32,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, ragged=3),
        # a beam step of 64 beams on 16 parents: the old beams freed, the parents forked, every beam one token longer
        dict(name="pages_beam_64", op="beam", dtype="bf16", parents=16, children=64, len_lo=129, len_hi=384, layers=4,
             kv_heads=16, dim=128, page=16, pages=2048, ragged=1),
        # prompts of a prefill chunk written into their pages
        dict(name="pages_append_64x256", op="append", dtype="bf16", seqs=64, new_lo=200, new_hi=300, past_lo=0,
             past_hi=64, kv_heads=16, dim=128, page=16, pages=2048, ragged=2),
        # a pool half empty after many requests have ended, packed to its low end
        dict(name="pages_compact_4096", op="compact", dtype="bf16", seqs=96, len_lo=1, len_hi=600, layers=4,
             kv_heads=16, dim=128, page=16, pages=4096, ragged=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "decode", "decode", "decode", "beam", "append", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, rng.randrange(8, 136, 8)])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 4, 8])
    ragged = rng.randrange(1, 1 << 30)
    if op == "window":
        most = work(max((c for c in listed() if c["op"] == "window"), key=lambda c: work(c)["flops"]))["flops"]
        while True:
            train = rng.random() < 0.5
            c = dict(op=op, train=train, dtype=dtype, seqs=_log(rng, 1, 64), q_lo=1, q_hi=_log(rng, 1, 4096), past_lo=0,
                     past_hi=0 if train or rng.random() < 0.5 else _log(rng, 1, 14000), heads=kv_heads * group,
                     kv_heads=kv_heads, dim=dim, window=rng.choice([0, _log(rng, 1, 4096)]),
                     sinks=rng.choice([0, 1, 4, rng.randrange(0, 80)]), ragged=ragged)
            c["q_lo"] = max(1, int(c["q_hi"] * rng.choice([0.05, 0.5, 1.0])))
            lq, lk = _window_lens(c)
            if c["seqs"] * c["heads"] * max(lq) * max(lk) > MOST_SCORES:
                continue
            w = work(c)
            if w["flops"] > (most if dtype == "bf16" else most / 16) or max(sum(lq), sum(lk)) > 65536:
                continue
            return c
    if op == "decode":
        while True:
            c = dict(op=op, dtype=dtype, seqs=_log(rng, 1, 256), len_lo=1, len_hi=_log(rng, 1, 131072),
                     heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                     window=rng.choice([0, 0, _log(rng, 1, 8192)]), sinks=rng.choice([0, 4, rng.randrange(0, 200)]),
                     ragged=ragged)
            c["len_lo"] = max(1, int(c["len_hi"] * rng.choice([0.01, 0.5, 1.0])))
            lens = _lens(c["seqs"], c["len_lo"], c["len_hi"], ragged)
            size = 4 if dtype == "f32" else 2
            if sum(lens) * 2 * kv_heads * dim * size > MOST_POOL / 2 or \
                    c["seqs"] * max(lens) * kv_heads * dim * 4 > 8e9:
                continue
            return c
    while True:
        page = rng.choice([16, 32, 64])
        size = 4 if dtype == "f32" else 2
        c = dict(op=op, dtype=dtype, kv_heads=kv_heads, dim=dim, page=page, ragged=ragged)
        if op == "append":
            c.update(seqs=_log(rng, 1, 256), new_lo=1, new_hi=_log(rng, 1, 1024), past_lo=0, past_hi=_log(rng, 1, 512))
            need = sum(-(-(a + b) // page) for a, b in zip(*_append_lens(c)))
            layers = 1
        elif op == "beam":
            c.update(parents=_log(rng, 1, 32), len_lo=1, len_hi=_log(rng, 16, 2000), layers=rng.randrange(1, 7))
            c["children"] = c["parents"] * rng.randrange(1, 5)
            need = sum(-(-n // page) for n in _lens(c["parents"], 1, c["len_hi"], ragged)) + c["children"] * 2
            layers = c["layers"]
        else:
            c.update(seqs=_log(rng, 1, 256), len_lo=1, len_hi=_log(rng, 16, 2000), layers=rng.randrange(1, 7))
            need = sum(-(-n // page) for n in _lens(c["seqs"], 1, c["len_hi"], ragged)) * 2
            layers = c["layers"]
        c["pages"] = need + rng.randrange(1, 2 * need + 16)
        if 2 * layers * c["pages"] * kv_heads * page * dim * size <= MOST_POOL / 2:
            return c


def _lens(n, lo, hi, ragged):
    r = random.Random(ragged * 7919 + n)
    return [r.randint(lo, hi) for _ in range(n)]


def _window_lens(c):
    lq = _lens(c["seqs"], c["q_lo"], c["q_hi"], c["ragged"])
    past = _lens(c["seqs"], c["past_lo"], c["past_hi"], c["ragged"] + 1)
    return lq, [a + b for a, b in zip(lq, past)]


def _append_lens(c):
    return (_lens(c["seqs"], c["new_lo"], c["new_hi"], c["ragged"]),
            _lens(c["seqs"], c["past_lo"], c["past_hi"], c["ragged"] + 1))


def _visible(p, window, sinks):
    """Visible keys of a query at position p (0-based), summed by the caller."""
    if window == 0 or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


# ---------------------------------------------------------------------------------------- prepare
def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pool(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _tables(lens, page, width, pages, rng):
    """A table of scattered pages (-1 past a sequence's last page) and the pages' reference counts."""
    ids = rng.permutation(pages)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(lens):
        k = -(-n // page)
        table[i, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(pages, dtype=np.int32)
    refs[ids[:at]] = 1
    return torch.from_numpy(table).to(DEV), torch.from_numpy(refs).to(DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[c["dtype"]]
    s = {"c": c}
    if c["op"] == "window":
        lq, lk = _window_lens(c)
        s["max_q"], s["max_k"] = max(lq), max(lk)
        s["cu_q"], s["cu_k"] = _cu(lq), _cu(lk)
        s["q"] = _normal((sum(lq), c["heads"], c["dim"]), dt, gen)
        s["k"] = _normal((sum(lk), c["kv_heads"], c["dim"]), dt, gen)
        s["v"] = _normal((sum(lk), c["kv_heads"], c["dim"]), dt, gen)
        if c["train"]:
            s["do"] = _normal((sum(lq), c["heads"], c["dim"]), dt, gen)
    elif c["op"] == "decode":
        lens = _lens(c["seqs"], c["len_lo"], c["len_hi"], c["ragged"])
        width = -(-max(lens) // c["page"])
        pages = sum(-(-n // c["page"]) for n in lens) + 3
        s["max_len"] = max(lens)
        s["table"], _ = _tables(lens, c["page"], width, pages, rng)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["k"] = _pool((pages, c["kv_heads"], c["page"], c["dim"]), dt, gen)
        s["v"] = _pool((pages, c["kv_heads"], c["page"], c["dim"]), dt, gen)
        s["q"] = _normal((c["seqs"], c["heads"], c["dim"]), dt, gen)
        s["k_new"] = _normal((c["seqs"], c["kv_heads"], c["dim"]), dt, gen)
        s["v_new"] = _normal((c["seqs"], c["kv_heads"], c["dim"]), dt, gen)
    elif c["op"] == "append":
        new, past = _append_lens(c)
        lens = [a + b for a, b in zip(new, past)]
        s["table"], _ = _tables(lens, c["page"], -(-max(lens) // c["page"]), c["pages"], rng)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["seqs"] = torch.arange(c["seqs"], dtype=torch.int32, device=DEV)
        s["cu"] = _cu(new)
        shape = (c["pages"], c["kv_heads"], c["page"], c["dim"])
        s["k"], s["v"] = _pool(shape, dt, gen), _pool(shape, dt, gen)
        s["k_new"] = _normal((sum(new), c["kv_heads"], c["dim"]), dt, gen)
        s["v_new"] = _normal((sum(new), c["kv_heads"], c["dim"]), dt, gen)
    else:
        n = c["parents"] if c["op"] == "beam" else c["seqs"]
        lens = _lens(n, c["len_lo"], c["len_hi"], c["ragged"])
        rows = n + (c["children"] if c["op"] == "beam" else 0)
        width = -(-(max(lens) + 1) // c["page"])
        lens = lens + [0] * (rows - n)
        s["table"], s["refs"] = _tables(lens, c["page"], width, c["pages"], rng)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        shape = (c["layers"], c["pages"], c["kv_heads"], c["page"], c["dim"])
        s["k"], s["v"] = _pool(shape, dt, gen), _pool(shape, dt, gen)
        if c["op"] == "beam":
            s["children"] = torch.arange(n, rows, dtype=torch.int32, device=DEV)
            s["parents"] = torch.from_numpy(rng.integers(0, n, rows - n).astype(np.int32)).to(DEV)
        else:  # the packed pool's own table and counts: steps in flight still read the old ones
            s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    return s


# ------------------------------------------------------------------------------------- plain forms
def _masked(lq, lk, max_q, max_k, window, sinks):
    """[B, max_q, max_k] truth values of the visible pairs of a padded batch."""
    i = torch.arange(max_q, device=DEV)[None, :, None]
    j = torch.arange(max_k, device=DEV)[None, None, :]
    p = i + (lk - lq)[:, None, None]
    see = (j <= p) & (i < lq[:, None, None])
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def _softmax(scores, see):
    """Probabilities (zero where nothing is visible) and the log of the sums, of scores changed in place."""
    scores.masked_fill_(~see, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return p.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _pad(x, cu, most, groups):
    """[T, H, D] of packed sequences -> [B, H / groups, groups, most, D] in 32 bits, zeros past a sequence's end."""
    at = cu[:-1, None].long() + torch.arange(most, device=DEV)[None]
    fine = at < cu[1:, None]
    y = x.float()[torch.where(fine, at, 0)] * fine[..., None, None]
    b, _, h, d = y.shape
    return y.view(b, most, h // groups, groups, d).permute(0, 2, 3, 1, 4).contiguous(), at[fine], fine


def _unpad(y, fine):
    """The inverse: [B, H, G, most, D] -> [T, H G, D]."""
    b, h, g, most, d = y.shape
    return y.permute(0, 3, 1, 2, 4).reshape(b, most, h * g, d)[fine]


def _plain_window(s):
    c, dt, scale = s["c"], s["q"].dtype, s["c"]["dim"] ** -0.5
    group = c["heads"] // c["kv_heads"]
    q, _, fine_q = _pad(s["q"], s["cu_q"], s["max_q"], group)
    k, _, fine_k = _pad(s["k"], s["cu_k"], s["max_k"], 1)
    v, _, _ = _pad(s["v"], s["cu_k"], s["max_k"], 1)
    see = _masked(s["cu_q"].diff(), s["cu_k"].diff(), s["max_q"], s["max_k"], c["window"], c["sinks"])[:, None, None]
    b, h = q.shape[:2]
    flat = lambda x: x.reshape(b, h, group * s["max_q"], -1)
    grouped = lambda x: x.view(b, h, group, s["max_q"], -1)
    p, lse = _softmax(grouped(torch.matmul(flat(q), k.squeeze(2).mT)).mul_(scale), see)
    o = grouped(torch.matmul(flat(p), v.squeeze(2)))
    out = {"o": _unpad(o, fine_q).to(dt), "lse": _unpad(lse[..., None], fine_q).squeeze(-1)}
    if c["train"]:
        do, _, _ = _pad(s["do"], s["cu_q"], s["max_q"], group)
        dv = torch.matmul(flat(p).mT, flat(do))
        ds = grouped(torch.matmul(flat(do), v.squeeze(2).mT))
        ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq = grouped(torch.matmul(flat(ds), k.squeeze(2)))
        dk = torch.matmul(flat(ds).mT, flat(q))
        out["dq"] = _unpad(dq, fine_q).to(dt)
        out["dk"], out["dv"] = _unpad(dk[:, :, None], fine_k).to(dt), _unpad(dv[:, :, None], fine_k).to(dt)
    return out


def _plain_decode(s):
    c, group = s["c"], s["c"]["heads"] // s["c"]["kv_heads"]
    b, page, dim = c["seqs"], c["page"], c["dim"]
    last = (s["lens"] - 1).long()
    own_page = s["table"].long().gather(1, (last // page)[:, None]).squeeze(1)
    s["k"][own_page, :, last % page] = s["k_new"]
    s["v"][own_page, :, last % page] = s["v_new"]
    at = s["table"].long().clamp(min=0)
    rows = lambda pool: pool[at].permute(0, 2, 1, 3, 4).float().reshape(b, c["kv_heads"], -1, dim)
    j = torch.arange(at.shape[1] * page, device=DEV)[None]
    see = j <= last[:, None]
    if c["window"]:
        see &= (j > last[:, None] - c["window"]) | (j < c["sinks"])
    k, v = rows(s["k"]), rows(s["v"])
    q = s["q"].float().view(b, c["kv_heads"], group, dim)
    p, lse = _softmax(torch.matmul(q, k.mT).mul_(dim ** -0.5), see[:, None, None])
    o = torch.matmul(p, v)
    return {"o": o.view(b, -1, dim).to(s["q"].dtype), "lse": lse.view(b, -1), "k": s["k"], "v": s["v"]}


def _plain_append(s):
    page, cu = s["c"]["page"], s["cu"].long()
    t = torch.arange(s["k_new"].shape[0], device=DEV)
    i = torch.searchsorted(cu[1:], t, right=True)
    pos = s["lens"].long()[i] - cu[i + 1] + t
    at = s["table"].long()[i, pos // page]
    s["k"][at, :, pos % page] = s["k_new"]
    s["v"][at, :, pos % page] = s["v_new"]
    return {"k": s["k"], "v": s["v"]}


def _plain_beam(s):
    page, refs, table, lens = s["c"]["page"], s["refs"], s["table"], s["lens"]
    col = torch.arange(table.shape[1], device=DEV)[None]
    kids, parents = s["children"].long(), s["parents"].long()
    # the old beams' pages freed
    held = col < -(-lens[kids] // page)[:, None]
    refs.index_add_(0, table[kids][held].long(), -torch.ones_like(table[kids][held]))
    table[kids] = torch.where(held, -1, table[kids])
    lens[kids] = 0
    # the parents forked
    held = col < -(-lens[parents] // page)[:, None]
    refs.index_add_(0, table[parents][held].long(), torch.ones_like(table[parents][held]))
    table[kids] = torch.where(held, table[parents], table[kids])
    lens[kids] = lens[parents]
    # one token more: a page of its own where the last one is shared and not full, or where it is full
    old = lens[kids]
    part = old % page != 0
    last = table[kids, (old // page).clamp(max=table.shape[1] - 1).long()].long()
    cow = part & (refs[last.clamp(min=0)] > 1)
    need = cow | ~part
    fresh = torch.nonzero(refs == 0).squeeze(1)[:int(need.sum())]
    src, dst = last[cow], fresh[(need.cumsum(0) - 1)[cow]]
    keep = (torch.arange(page, device=DEV)[None] < (old % page)[cow][:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(keep, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(keep, s["v"][:, src], s["v"][:, dst])
    refs.index_add_(0, src, -torch.ones_like(src, dtype=torch.int32))
    refs[fresh] = 1
    table[kids[need], (old // page).long()[need]] = fresh.int()
    lens[kids] = old + 1
    return {"table": table, "refs": refs, "lens": lens, "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    page, refs, table = s["c"]["page"], s["refs"], s["table"]
    live = refs > 0
    n_live = int(live.sum())
    at = torch.arange(refs.numel(), device=DEV)
    src, dst = at[live & (at >= n_live)], at[~live & (at < n_live)]
    to = at.int()
    to[src] = dst.int()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    held = torch.arange(table.shape[1], device=DEV)[None] < -(-s["lens"] // page)[:, None]
    s["table_out"].copy_(torch.where(held, to[table.clamp(min=0).long()], table))
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    return {"table": s["table_out"], "refs": s["refs_out"], "n_live": torch.full((1,), n_live, dtype=torch.int32, device=DEV),
            "k": s["k"], "v": s["v"]}


# --------------------------------------------------------------------------------------------- run
def run(state):
    s, c = state, state["c"]
    if not own:
        return {"window": _plain_window, "decode": _plain_decode, "append": _plain_append, "beam": _plain_beam,
                "compact": _plain_compact}[c["op"]](s)
    import token_indexed_ffn_amd as st
    if c["op"] == "window":
        how = dict(window=c["window"], sinks=c["sinks"])
        out = st.staple_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], **how)
        if c["train"]:
            out.update(st.staple_attn_bwd(s["do"], s["q"], s["k"], s["v"], out["o"], out["lse"], s["cu_q"], s["cu_k"],
                                          **how))
        return out
    if c["op"] == "decode":
        out = st.staple_attn_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], k_new=s["k_new"],
                                          v_new=s["v_new"], max_len=s["max_len"], window=c["window"],
                                          sinks=c["sinks"])
        return {"o": out["o"], "lse": out["lse"], "k": s["k"], "v": s["v"]}
    if c["op"] == "append":
        st.staple_kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], s["seqs"], s["cu"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "beam":
        st.staple_kv_free(s["refs"], s["table"], s["lens"], s["children"], page_size=c["page"])
        st.staple_kv_fork(s["refs"], s["table"], s["lens"], s["parents"], s["children"], page_size=c["page"])
        st.staple_kv_extend(s["refs"], s["table"], s["lens"], s["children"], k_pages=s["k"], v_pages=s["v"])
        return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "k": s["k"], "v": s["v"]}
    out = st.staple_kv_compact(s["refs"], s["table"], s["lens"], s["k"], s["v"],
                               out={"refs": s["refs_out"], "table": s["table_out"]})
    return {"table": out["table"], "refs": out["refs"], "n_live": out["n_live"], "k": s["k"], "v": s["v"]}


# -------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "window":
        lq, lk = _window_lens(c)
        pairs = sum(_visible(p, c["window"], c["sinks"]) for a, b in zip(lq, lk) for p in range(b - a, b))
        q, kv = sum(lq) * c["heads"] * c["dim"] * size, sum(lk) * c["kv_heads"] * c["dim"] * size
        lse = sum(lq) * c["heads"] * 4
        if c["train"]:  # two products forward, five backward; do read, dq, dk and dv written
            return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * c["dim"] * c["heads"] * pairs}
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * c["dim"] * c["heads"] * pairs}
    row = c["kv_heads"] * c["dim"] * size
    if c["op"] == "decode":
        lens = _lens(c["seqs"], c["len_lo"], c["len_hi"], c["ragged"])
        seen = sum(_visible(n - 1, c["window"], c["sinks"]) for n in lens)
        small = c["seqs"] * (2 * row + c["heads"] * (2 * c["dim"] * size + 4) + 4)
        return {"bytes": 2 * seen * row + small, "flops": 4 * c["dim"] * c["heads"] * seen}
    if c["op"] == "append":
        new, _ = _append_lens(c)
        return {"bytes": 4 * sum(new) * row, "flops": 0}
    if c["op"] == "beam":
        lens = _lens(c["parents"], c["len_lo"], c["len_hi"], c["ragged"])
        part = sum(n % c["page"] for n in lens) * c["children"] / c["parents"]
        held = sum(-(-n // c["page"]) for n in lens) * c["children"] / c["parents"]
        return {"bytes": int(4 * c["layers"] * part * row + 3 * 8 * held), "flops": 0}
    lens = _lens(c["seqs"], c["len_lo"], c["len_hi"], c["ragged"])
    held = sum(-(-n // c["page"]) for n in lens)
    moved = held * (1 - held / c["pages"])  # the expected number of live pages past n_live
    return {"bytes": int(4 * c["layers"] * moved * c["page"] * row + 8 * (held + c["pages"])), "flops": 0}


# ------------------------------------------------------------------------------------------- exact
def _exact_pairs(lq, lk, window, sinks):
    p = torch.arange(lk - lq, lk, device=DEV)[:, None]
    j = torch.arange(lk, device=DEV)[None]
    hidden = j > p
    if window:
        hidden |= (p - j >= window) & (j >= sinks)
    return hidden


def _exact_window(s):
    c = s["c"]
    group, scale = c["heads"] // c["kv_heads"], 1.0 / math.sqrt(c["dim"])
    f = {n: s[n].double() for n in ("q", "k", "v", "do") if n in s}
    out = {"o": torch.zeros_like(f["q"]), "lse": torch.zeros(f["q"].shape[:2], dtype=torch.float64, device=DEV)}
    if c["train"]:
        out.update(dq=torch.zeros_like(f["q"]), dk=torch.zeros_like(f["k"]), dv=torch.zeros_like(f["v"]))
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for a, b, x, y in zip(cq, cq[1:], ck, ck[1:]):
        if a == b:
            continue
        hidden = _exact_pairs(b - a, y - x, c["window"], c["sinks"])
        for h in range(c["heads"]):
            q, k, v = f["q"][a:b, h], f["k"][x:y, h // group], f["v"][x:y, h // group]
            w = (scale * (q @ k.T)).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(w, -1)
            w = torch.exp(w - lse[:, None])
            out["o"][a:b, h], out["lse"][a:b, h] = w @ v, lse
            if c["train"]:
                do = f["do"][a:b, h]
                g = do @ v.T
                g = scale * w * (g - (w * g).sum(-1, keepdim=True))
                out["dq"][a:b, h] = g @ k
                out["dk"][x:y, h // group] += g.T @ q
                out["dv"][x:y, h // group] += w.T @ do
    return out


def _exact_decode(s):
    c = s["c"]
    page, group, dim = c["page"], c["heads"] // c["kv_heads"], c["dim"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        seen = [j for j in range(n) if not c["window"] or j >= n - c["window"] or j < c["sinks"]]
        at = torch.tensor(seen, device=DEV)
        ids = s["table"][i].long()[at // page]
        k, v = s["k"][ids, :, at % page].double(), s["v"][ids, :, at % page].double()
        k[-1], v[-1] = s["k_new"][i].double(), s["v_new"][i].double()
        q = s["q"][i].double().view(c["kv_heads"], group, dim)
        w = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(dim)
        lse[i] = torch.logsumexp(w, -1).reshape(-1)
        o[i] = torch.matmul(torch.softmax(w, -1), v.permute(1, 0, 2)).reshape(-1, dim)
    return {"o": o, "lse": lse, "k": None, "v": None}


def exact(case, seed):
    if case["op"] not in ("window", "decode"):
        return None  # moved rows and whole numbers: nothing is computed
    return (_exact_window if case["op"] == "window" else _exact_decode)(prepare(case, seed))
