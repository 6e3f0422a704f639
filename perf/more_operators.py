"""Measured cases of the operators at a model's two ends and around its blocks: the embedding lookup
with its gradient, the norms before and after a block with its gate and residual sum, the loss of a
vocabulary's logits with its gradient, and sampling of the next token.

`run` computes a case in elementary torch operations in 32 bits (long sums, and what decides a token, in
64), or, where `own` is true, with the framework's entry points.

Embedding      y_i = scale E[t_i];   dE_t = scale sum of dy_i over the positions i of token t
Norms          b = z / rms(z) w_post (or z),  r = x + scale gate b,  h = r / rms(r) w_pre,
               rms(v) = sqrt(mean(v^2) + eps)
Loss           lse_i = log sum_j exp l_ij,  loss_i = lse_i - l_i[t_i],  dl_ij = g_i (exp(l_ij - lse_i) - [j = t_i]);
               rows with a negative target have a loss and a gradient of zero
Sampling       w_j = exp((l_j - max l) / T).  In the order of falling l_j, ties by rising j, a token is kept while it
               is among the first k, the sum of the kept ones before it is less than p times the sum of the first k,
               and w_j >= min_p; the token is the first j, in the order of j, at which the sum of the kept w passes
               u times the sum of all of them.  T = 0: the largest l_j.  logprob: log of its share of the kept sum.
               A row with nothing but -inf has token -1 and logprob -inf.
"""
import math

import numpy as np
import torch


own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the decode step's 64 tokens looked up in a table of 100352 rows: latency alone
        dict(name="embed_decode_64", op="embed", train=False, dtype="bf16", out="bf16", tokens=64, vocab=100352,
             dim=2048, zipf=1.1, scale=1.0, into="rows"),
        # the training batch of 32768 tokens: lookup, and the gradient of the rows of its unique tokens
        dict(name="embed_train_32k", op="embed", train=True, dtype="bf16", out="bf16", tokens=32768, vocab=100352,
             dim=2048, zipf=1.1, scale=1.0, into="rows"),
        # fp32 master weights looked up in bf16 and scaled, odd sizes, the gradient in the whole table's rows
        dict(name="embed_train_odd_f32", op="embed", train=True, dtype="f32", out="bf16", tokens=8191, vocab=50021,
             dim=1111, zipf=1.3, scale=32.0, into="table"),
        # a decode step's 64 rows between two blocks: norm after the one, residual sum, norm before the next
        dict(name="norm_decode_64", op="norm", train=False, dtype="bf16", residual="bf16", weights="bf16", rows=64,
             dim=2048, post=True, pre=True, gate="none", scale=1.0),
        # the same seam in the training step of 32768 tokens, with a learned gate, and its gradients
        dict(name="norm_train_32k", op="norm", train=True, dtype="bf16", residual="bf16", weights="f32", rows=32768,
             dim=2048, post=True, pre=True, gate="vector", scale=1.0),
        # 16384 tokens of 4096: the residual stream in fp32 beside bf16 blocks, norm before the block only
        dict(name="norm_train_16k_f32_stream", op="norm", train=True, dtype="bf16", residual="f32", weights="f32",
             rows=16384, dim=4096, post=False, pre=True, gate="none", scale=0.5),
        # odd sizes in fp32, every token with a gate of its own
        dict(name="norm_train_odd_f32", op="norm", train=True, dtype="f32", residual="f32", weights="f32", rows=4099,
             dim=1111, post=True, pre=True, gate="rows", scale=0.25),
        # the small fp32 model's unit workload: 512 tokens over 4096 classes, a tenth of the targets left out
        dict(name="xent_train_f32_512", op="xent", train=True, dtype="f32", rows=512, vocab=4096, ignored=0.1),
        # a training micro-batch over the whole vocabulary, padded documents, with the gradient of the logits
        dict(name="xent_train_8k", op="xent", train=True, dtype="bf16", rows=8192, vocab=100352, ignored=0.05),
        # one user's next token, all three limits
        dict(name="sample_1", op="sample", dtype="bf16", rows=1, vocab=100352, limits="kpm", masked=0.0),
        # the decode batch of 64: each row with a temperature and limits of its own, some of the vocabulary ruled out
        dict(name="sample_64_mixed", op="sample", dtype="f32", rows=64, vocab=100352, limits="kpm", masked=0.3),
        # many rollouts at once: temperature alone, a vocabulary of odd size
        dict(name="sample_509_free", op="sample", dtype="bf16", rows=509, vocab=50021, limits="", masked=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "norm", "xent", "sample"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "embed":
            c = dict(op=op, train=rng.random() < 0.6, dtype=dtype, out=rng.choice([dtype, "bf16", "f32"]),
                     tokens=_log(rng, 1, 40000), vocab=_log(rng, 10, 110000), dim=_log(rng, 8, 8192),
                     zipf=rng.choice([0.0, 1.1, 2.0]), scale=rng.choice([1.0, 0.125, 32.0]),
                     into=rng.choice(["rows", "table"]))
            if rng.random() < 0.5:
                c["dim"] = max(8, c["dim"] // 64 * 64)
            if c["vocab"] * c["dim"] * 4 > 4e9:
                continue
        elif op == "norm":
            c = dict(op=op, train=rng.random() < 0.6, dtype=dtype, residual=rng.choice([dtype, "f32"]),
                     weights=rng.choice([dtype, "f32"]), rows=_log(rng, 1, 40000), dim=_log(rng, 8, 16384),
                     post=rng.random() < 0.6, pre=rng.random() < 0.8, gate=rng.choice(["none", "vector", "rows"]),
                     scale=rng.choice([1.0, 0.5, 0.125]))
            if rng.random() < 0.5:
                c["dim"] = max(8, c["dim"] // 64 * 64)
        elif op == "xent":
            c = dict(op=op, train=rng.random() < 0.7, dtype=dtype, rows=_log(rng, 1, 33000), vocab=_log(rng, 2, 260000),
                     ignored=rng.choice([0.0, 0.1, 0.9]))
        else:
            c = dict(op=op, dtype=dtype, rows=_log(rng, 1, 512), vocab=_log(rng, 2, 260000),
                     limits=rng.choice(["", "k", "p", "m", "kp", "kpm"]), masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
        if work(c)["bytes"] <= most:
            return c


# ---------------------------------------------------------------------------------------- prepare
def _normal(shape, gen, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _weight(dim, gen, dtype):
    return (1 + 0.1 * torch.randn(dim, generator=gen, device=DEV)).to(dtype)


def _tokens(n, vocab, exponent, gen):
    """Token IDs with the frequencies of text: rank ~ Zipf, the ranks' IDs shuffled."""
    share = torch.arange(1, vocab + 1, device=DEV, dtype=torch.float64) ** -exponent
    cdf = share.cumsum(0) / share.sum()
    rank = torch.searchsorted(cdf, torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)).clamp(max=vocab - 1)
    return torch.randperm(vocab, generator=gen, device=DEV)[rank].int()


def _logits(rows, vocab, gen, dtype):
    """Logits over tokens whose frequencies fall like text's, the row's own preferences on top."""
    usual = -1.1 * torch.log1p(torch.randperm(vocab, generator=gen, device=DEV).float())
    out = torch.empty(rows, vocab, dtype=dtype, device=DEV)
    for a in range(0, rows, 1024):
        b = min(a + 1024, rows)
        out[a:b] = _normal((b - a, vocab), gen, std=2.0).add_(usual)
    return out


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c}
    if c["op"] == "embed":
        n, dim = c["tokens"], c["dim"]
        s["ids"] = _tokens(n, c["vocab"], c["zipf"], gen)
        s["table"] = _normal((c["vocab"], dim), gen, DTYPES[c["dtype"]], 0.02)
        if c["train"]:
            s["dy"] = _normal((n, dim), gen, DTYPES[c["out"]], 1e-2)
            # the batch's unique tokens, found once a batch for every table that it reads
            uniq, inv, count = torch.unique(s["ids"], return_inverse=True, return_counts=True)
            s["uniq"], s["inv"] = uniq, inv.int()
            s["sorted_pos"] = torch.sort(inv, stable=True).indices.int()
            s["seg_start"] = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
            s["seg_start"][1:len(uniq) + 1] = count.cumsum(0)
            s["n_unique"] = torch.full((1,), len(uniq), dtype=torch.int32, device=DEV)
            # as many rows as there could be: how many there are is known on the device
            s["grad"] = torch.zeros(c["vocab"] if c["into"] == "table" else min(n, c["vocab"]), dim, device=DEV)
    elif c["op"] == "norm":
        shape, dt, wt = (c["rows"], c["dim"]), DTYPES[c["dtype"]], DTYPES[c["weights"]]
        # a residual stream has grown over the layers, a few of its channels far more than the rest
        s["x"] = (_normal(shape, gen, std=2.0) * (1 + 20 * (torch.rand(c["dim"], generator=gen, device=DEV) < 0.01))).to(
            DTYPES[c["residual"]])
        s["z"] = _normal(shape, gen, dt, 0.7)
        s["w_post"] = _weight(c["dim"], gen, wt) if c["post"] else None
        s["w_pre"] = _weight(c["dim"], gen, wt) if c["pre"] else None
        s["gate"] = None
        if c["gate"] == "vector":
            s["gate"] = _weight(c["dim"], gen, wt)
        elif c["gate"] == "rows":
            s["gate"] = _normal(shape, gen, dt)
        if c["train"]:
            s["dr"] = _normal(shape, gen, DTYPES[c["residual"]], 1e-2)
            s["dh"] = _normal(shape, gen, dt, 1e-2) if c["pre"] else None
    elif c["op"] == "xent":
        n, v = c["rows"], c["vocab"]
        s["logits"] = _logits(n, v, gen, DTYPES[c["dtype"]])
        # half of the targets are what the model would say
        t = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.5, s["logits"].argmax(1),
                        torch.randint(v, (n,), generator=gen, device=DEV))
        left_out = torch.rand(n, generator=gen, device=DEV) < c["ignored"]
        s["targets"] = torch.where(left_out, -100, t).int()
        s["g"] = torch.full((n,), 1.0 / max(1, n - int(left_out.sum())), device=DEV)
    else:
        n, v = c["rows"], c["vocab"]
        s["logits"] = _logits(n, v, gen, DTYPES[c["dtype"]])
        if c["masked"]:  # tokens that a grammar rules out
            hidden = torch.rand(n, v, generator=gen, device=DEV) < c["masked"]
            hidden &= torch.rand(n, 1, generator=gen, device=DEV) < 0.5
            s["logits"].masked_fill_(hidden, -math.inf)
        unit = lambda: torch.rand(n, generator=gen, device=DEV)
        s["u"] = unit()
        s["temperature"] = torch.where(unit() < 0.1, 0.0, 0.3 + 1.2 * unit())
        on = lambda letter: (unit() < 0.7) if n > 1 else torch.ones(1, dtype=torch.bool, device=DEV)
        s["top_k"] = torch.where(on("k"), 1 + (200 * unit()).int(), 0).int() if "k" in c["limits"] else None
        s["top_p"] = torch.where(on("p"), 0.8 + 0.19 * unit(), 1.0) if "p" in c["limits"] else None
        s["min_p"] = torch.where(on("m"), 0.2 * unit(), 0.0) if "m" in c["limits"] else None
    return s


# ------------------------------------------------------------------------------------- plain forms
def _plain_embed(s):
    c = s["c"]
    out = {"y": (s["table"][s["ids"].long()].float() * c["scale"]).to(DTYPES[c["out"]])}
    if c["train"]:
        # in 64 bits: added one by one, a frequent token's thousands of rows
        total = torch.zeros(len(s["uniq"]), c["dim"], dtype=torch.float64, device=DEV)
        total.index_add_(0, s["inv"].long(), s["dy"].double())
        rows = (total * c["scale"]).float()
        if c["into"] == "table":
            s["grad"][s["uniq"].long()] = rows
        else:
            s["grad"][:len(rows)] = rows
        out["grad"] = s["grad"]
    return out


def _normed(v):
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * rstd, rstd


def _norm_grad(dy, hat, rstd):
    return rstd * (dy - hat * (dy * hat).mean(-1, keepdim=True))


def _columns(t):
    return t.sum(0)


def _plain_norm(s):
    c, dt, rt = s["c"], s["z"].dtype, s["x"].dtype
    f = {n: s[n].float() for n in ("x", "z", "w_post", "w_pre", "gate", "dr", "dh") if s.get(n) is not None}
    z_hat, z_rstd = _normed(f["z"]) if c["post"] else (f["z"], None)
    b = z_hat * f["w_post"] if c["post"] else z_hat
    r = f["x"] + c["scale"] * (f["gate"] * b if "gate" in f else b)
    out = {"r": r.to(rt)}
    if c["pre"]:
        r_hat, r_rstd = _normed(r)
        out["h"] = (r_hat * f["w_pre"]).to(dt)
    if c["train"]:
        g = f["dr"]
        if c["pre"]:
            out["dw_pre"] = _columns(f["dh"] * r_hat)
            g = g + _norm_grad(f["dh"] * f["w_pre"], r_hat, r_rstd)
        out["dx"] = g.to(rt)
        g = c["scale"] * g
        if "gate" in f:
            dgate = g * b
            out["dgate"] = _columns(dgate) if c["gate"] == "vector" else dgate.to(dt)
            g = g * f["gate"]
        if c["post"]:
            out["dw_post"] = _columns(g * z_hat)
            g = _norm_grad(g * f["w_post"], z_hat, z_rstd)
        out["dz"] = g.to(dt)
    return out


def _plain_xent(s):
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = x.sub(top).exp_()
    total = e.sum(1, keepdim=True)
    lse = total.log().add_(top).squeeze(1)
    counts = s["targets"] >= 0
    at = s["targets"].clamp(min=0).long()[:, None]
    out = {"loss": torch.where(counts, lse - x.gather(1, at).squeeze(1), 0.0), "lse": lse}
    if s["c"]["train"]:
        e.div_(total).scatter_add_(1, at, -torch.ones_like(total))
        out["d_logits"] = e.mul_(torch.where(counts, s["g"], 0.0)[:, None]).to(s["logits"].dtype)
    return out


def _plain_sample(s):
    l = s["logits"].double()
    n, v = l.shape
    t = s["temperature"].double()[:, None]
    greedy = t.squeeze(1) <= 0
    sorted_l, order = torch.sort(l, dim=1, descending=True, stable=True)
    top = sorted_l[:, :1]
    empty = top.squeeze(1) == -math.inf
    w = ((sorted_l - torch.where(empty[:, None], 0.0, top)) / torch.where(t > 0, t, 1.0)).exp()
    rank = torch.arange(v, device=DEV)[None]
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        p, sums = s["top_p"].double()[:, None], (w * keep).cumsum(1)
        before = torch.cat((torch.zeros_like(top), sums[:, :-1]), 1)
        keep &= (before < p * sums[:, -1:]) | (p >= 1) | (rank == 0)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(l).scatter_(1, order, w * keep)
    sums = kept.cumsum(1)
    total = sums[:, -1:]
    token = (sums <= s["u"].double()[:, None] * total).sum(1).clamp(max=v - 1)
    logprob = (kept.gather(1, token[:, None]) / total).log().squeeze(1)
    token = torch.where(empty, -1, torch.where(greedy, order[:, 0], token))
    logprob = torch.where(empty, -math.inf, torch.where(greedy, 0.0, logprob))
    return {"token": token.int(), "logprob": logprob.float()}


# --------------------------------------------------------------------------------------------- run
def run(state):
    s, c = state, state["c"]
    if not own:
        return {"embed": _plain_embed, "norm": _plain_norm, "xent": _plain_xent, "sample": _plain_sample}[c["op"]](s)
    import token_indexed_ffn_amd as st
    if c["op"] == "embed":
        out = {"y": st.staple_embed_fwd(s["table"], s["ids"], scale=c["scale"], out_dtype=DTYPES[c["out"]])}
        if c["train"]:
            out["grad"] = st.staple_embed_bwd(s["dy"], s["sorted_pos"], s["seg_start"], s["n_unique"], inv=s["inv"],
                                              uniq=s["uniq"] if c["into"] == "table" else None, scale=c["scale"],
                                              out=s["grad"])
        return out
    if c["op"] == "norm":
        how = dict(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], pre=c["pre"], post=c["post"], scale=c["scale"],
                   eps=EPS)
        f = st.staple_norm_fwd(s["x"], s["z"], save=c["train"], **how)
        out = {n: f[n] for n in ("r", "h") if f[n] is not None}
        if c["train"]:
            # a sum stored in bf16 is formed again from what it is made of, one in fp32 is read
            b = st.staple_norm_bwd(s["dr"], s["dh"], s["x"], s["z"], f["rstd_r"], f["rstd_z"],
                                   r=f["r"] if c["residual"] == "f32" else None, **how)
            out.update({n: t for n, t in b.items() if t is not None})
        return out
    if c["op"] == "xent":
        return st.staple_xent_fwd(s["logits"], s["targets"], g=s["g"] if c["train"] else None)
    return st.staple_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"])


# -------------------------------------------------------------------------------------------- work
def _distinct(n, vocab, exponent):
    """The expected number of distinct tokens among n."""
    share = np.arange(1, vocab + 1, dtype=np.float64) ** -exponent
    return int(round(float(-np.expm1(n * np.log1p(-np.minimum(share / share.sum(), 1 - 1e-12))).sum())))


def work(case):
    c = case
    if c["op"] == "embed":
        n, dim, rows = c["tokens"], c["dim"], _distinct(c["tokens"], c["vocab"], c["zipf"])
        moved = rows * dim * SIZE[c["dtype"]] + n * dim * SIZE[c["out"]] + 4 * n
        if c["train"]:
            moved += n * dim * SIZE[c["out"]] + rows * dim * 4 + 8 * n
        return {"bytes": moved, "flops": n * dim * (2 if c["train"] else 1)}
    if c["op"] == "norm":
        n = c["rows"] * c["dim"]
        size, stream = SIZE[c["dtype"]], SIZE[c["residual"]]
        gate = size if c["gate"] == "rows" else 0
        moved = n * (2 * stream + size + gate + (size if c["pre"] else 0))
        if c["train"]:  # the gradients of r and h read, those of x, z and the gate written
            moved += n * (2 * stream + size + gate + (size if c["pre"] else 0))
        return {"bytes": moved, "flops": n * (30 if c["train"] else 10)}
    n = c["rows"] * c["vocab"]
    if c["op"] == "xent":
        return {"bytes": n * SIZE[c["dtype"]] * (2 if c["train"] else 1) + 16 * c["rows"], "flops": n * (6 if c["train"] else 4)}
    return {"bytes": n * SIZE[c["dtype"]] + 28 * c["rows"], "flops": 5 * n}


# ------------------------------------------------------------------------------------------- exact
def _exact_embed(s):
    c = s["c"]
    out = {"y": torch.stack([s["table"][t].double() for t in s["ids"].tolist()]) * c["scale"]}
    if c["train"]:
        grad = torch.zeros(s["grad"].shape, dtype=torch.float64, device=DEV)
        ids = s["ids"].tolist()
        at = {}
        for i, t in enumerate(ids):
            at.setdefault(t, []).append(i)
        for u, t in enumerate(sorted(at)):
            grad[t if c["into"] == "table" else u] = s["dy"][at[t]].double().sum(0) * c["scale"]
        out["grad"] = grad
    return out


def _exact_norm(s):
    """Gradients by differentiation of the definition."""
    c = s["c"]
    leaf = {n: s[n].double().requires_grad_() for n in ("x", "z", "w_post", "w_pre", "gate") if s[n] is not None}
    b = leaf["z"]
    if c["post"]:
        b = leaf["w_post"] * b / (b.pow(2).sum(1, keepdim=True) / c["dim"] + EPS).sqrt()
    if "gate" in leaf:
        b = leaf["gate"] * b
    r = leaf["x"] + c["scale"] * b
    out, ends = {"r": r.detach()}, [r]
    if c["pre"]:
        h = leaf["w_pre"] * r / (r.pow(2).sum(1, keepdim=True) / c["dim"] + EPS).sqrt()
        out["h"] = h.detach()
        ends.append(h)
    if c["train"]:
        torch.autograd.backward(ends, [s["dr"].double()] + ([s["dh"].double()] if c["pre"] else []))
        name = {"x": "dx", "z": "dz", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
        out.update({name[n]: t.grad for n, t in leaf.items()})
    return out


def _exact_xent(s):
    n = s["c"]["rows"]
    out = {"loss": torch.zeros(n, dtype=torch.float64, device=DEV), "lse": torch.zeros(n, dtype=torch.float64, device=DEV)}
    if s["c"]["train"]:
        out["d_logits"] = torch.zeros(s["logits"].shape, dtype=torch.float64, device=DEV)
    for a in range(0, n, 512):
        at = slice(a, min(a + 512, n))
        x = s["logits"][at].double()
        out["lse"][at] = torch.logsumexp(x, 1)
        t = s["targets"][at].long()
        i = torch.nonzero(t >= 0).squeeze(1)
        out["loss"][at][i] = out["lse"][at][i] - x[i, t[i]]
        if s["c"]["train"]:
            d = torch.softmax(x[i], 1)
            d[torch.arange(len(i), device=DEV), t[i]] -= 1
            out["d_logits"][at][i] = d * s["g"][at][i].double()[:, None]
    return out


def _exact_sample(s):
    tokens, logprobs = [], []
    host = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    for i, l in enumerate(s["logits"].float().cpu().numpy().astype(np.float64)):
        if l.max() == -math.inf or host["temperature"][i] <= 0:
            tokens.append(-1 if l.max() == -math.inf else int(l.argmax()))
            logprobs.append(-math.inf if l.max() == -math.inf else 0.0)
            continue
        order = np.lexsort((np.arange(len(l)), -l))
        w = np.exp((l[order] - l[order[0]]) / host["temperature"][i])
        count = len(l)
        if host["top_k"] is not None and host["top_k"][i] > 0:
            count = min(count, int(host["top_k"][i]))
        if host["top_p"] is not None and host["top_p"][i] < 1:
            sums = np.cumsum(w[:count])
            count = min(count, 1 + int(np.searchsorted(sums, host["top_p"][i] * sums[-1], side="left")))
        if host["min_p"] is not None:
            count = min(count, int((w >= host["min_p"][i]).sum()))
        at = np.sort(order[:count])
        w = np.exp((l[at] - l.max()) / host["temperature"][i])
        sums = np.cumsum(w)
        j = min(int(np.searchsorted(sums, host["u"][i] * sums[-1], side="right")), count - 1)
        tokens.append(int(at[j]))
        logprobs.append(math.log(w[j] / sums[-1]))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device=DEV),
            "logprob": torch.tensor(logprobs, dtype=torch.float64, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "xent": _exact_xent, "sample": _exact_sample}[case["op"]](s)
