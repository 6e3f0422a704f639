"""CPU oracle of the embedding, the norms around a block, the loss and sampling.

TEST INFRASTRUCTURE ONLY, like staple_oracle: plain float64 numpy, sharing no code with the
library.
"""
from __future__ import annotations

import numpy as np


def f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


# ------------------------------------------------------------------------------------- embedding
def embed(table, ids, scale):
    return scale * f64(table)[np.asarray(ids)]


def embed_grad(dy, ids, scale):
    """{token: scale * the sum of its positions' rows}."""
    dy, out = f64(dy), {}
    for i, t in enumerate(np.asarray(ids).tolist()):
        out[t] = out.get(t, 0.0) + scale * dy[i]
    return out


# ----------------------------------------------------------------------------------------- norms
def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def norm(x, z, *, w_pre=None, w_post=None, gate=None, pre=True, post=False, scale=1.0, eps=1e-6):
    """r, h and 1 / rms of both; None for what there is not."""
    x, z, w_pre, w_post, gate = map(f64, (x, z, w_pre, w_post, gate))
    out = {"r": x, "h": None, "rstd_r": None, "rstd_z": None}
    if z is not None:
        b = z
        if post:
            out["rstd_z"] = rstd(z, eps)
            b = z * out["rstd_z"][:, None] * (1.0 if w_post is None else w_post)
        b = scale * b * (1.0 if gate is None else gate)
        out["r"] = b if x is None else x + b
    if pre:
        out["rstd_r"] = rstd(out["r"], eps)
        out["h"] = out["r"] * out["rstd_r"][:, None] * (1.0 if w_pre is None else w_pre)
    return out


def norm_grad(dr, dh, r, z, rstd_r, rstd_z, *, w_pre=None, w_post=None, gate=None, pre=True, post=False, scale=1.0):
    """Gradients from the stored r and the stored 1 / rms; dgate a row each."""
    dr, dh, r, z, rstd_r, rstd_z, w_pre, w_post, gate = map(f64, (dr, dh, r, z, rstd_r, rstd_z, w_pre, w_post, gate))
    g = np.zeros_like(r) if dr is None else dr
    out = {}
    if pre:
        hat = r * rstd_r[:, None]
        t = dh * (1.0 if w_pre is None else w_pre)
        g = g + rstd_r[:, None] * (t - hat * (t * hat).mean(axis=1, keepdims=True))
        out["dw_pre"] = (dh * hat).sum(axis=0)
    out["dx"] = g
    if z is None:
        return out
    hat = z * rstd_z[:, None] if post else z
    w = 1.0 if w_post is None else w_post
    q = scale * g
    if gate is not None:
        out["dgate"] = q * hat * (w if post else 1.0)
        q = q * gate
    if post:
        out["dw_post"] = (q * hat).sum(axis=0)
        q = q * w
        q = rstd_z[:, None] * (q - hat * (q * hat).mean(axis=1, keepdims=True))
    out["dz"] = q
    return out


# ------------------------------------------------------------------------------------------ loss
def xent(logits, targets, g=None):
    """loss, lse, p and with g d_logits."""
    l, targets = f64(logits), np.asarray(targets)
    n = len(l)
    out = {"loss": np.zeros(n), "lse": np.zeros(n), "p": np.zeros_like(l), "d_logits": np.zeros_like(l)}
    for i in range(n):
        top = l[i].max()
        with np.errstate(invalid="ignore", divide="ignore"):
            out["lse"][i] = top
            if not np.isinf(top):
                # p without the logarithm: far from 0 the sum is nothing beside the logits
                e = np.exp(l[i] - top)
                out["lse"][i] += np.log(e.sum())
                out["p"][i] = e / e.sum()
            t = targets[i]
            if t < 0:
                continue
            out["loss"][i] = np.inf if l[i, t] == -np.inf else out["lse"][i] - l[i, t]
            if g is not None and top != -np.inf:
                d = out["p"][i].copy()
                d[t] -= 1.0
                out["d_logits"][i] = float(g[i]) * d
    return out


# -------------------------------------------------------------------------------------- sampling
def whole(w):
    """A weight as a whole number of 2^-200."""
    num, den = float(w).as_integer_ratio()
    return (num << 200) // den


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """token and logprob of each row.  Sums and their shares are exact (of the weights in 64 bits): equal
    logits make sums that meet a border exactly."""
    logits = f64(logits)
    tokens, logprobs = [], []
    for i, l in enumerate(logits):
        l = np.minimum(np.where(np.isnan(l), -np.inf, l), float(np.finfo(np.float32).max))
        top = l.max()
        t = 1.0 if temperature is None else float(temperature[i])
        if top == -np.inf:
            tokens.append(-1)
            logprobs.append(-np.inf)
            continue
        if not t > 0.0:
            tokens.append(int(np.argmax(l)))
            logprobs.append(0.0)
            continue
        d = np.where(l == -np.inf, 0.0, l - top) / t
        w = np.where(l == -np.inf, 0.0, np.exp(d))
        order = sorted(range(len(l)), key=lambda j: (-l[j], j))
        kept = order
        if top_k is not None and 0 < int(top_k[i]) < len(l):
            kept = kept[:int(top_k[i])]
        if top_p is not None and float(top_p[i]) < 1.0:
            num, den = max(float(top_p[i]), 0.0).as_integer_ratio()
            want = num * sum(whole(w[j]) for j in kept)
            out, total = [], 0
            for j in kept:
                if out and total * den >= want:
                    break
                out.append(j)
                total += whole(w[j])
            kept = out
        if min_p is not None and float(min_p[i]) > 0.0:
            kept = [j for j in kept if w[j] >= min(float(min_p[i]), 1.0)]
        kept = sorted(j for j in kept if w[j] > 0.0)
        total = w[kept].sum()
        r = float(u[i])
        num, den = (min(r, 1.0) if r > 0.0 else 0.0).as_integer_ratio()
        target, sums = num * sum(whole(w[j]) for j in kept), 0
        for at, j in enumerate(kept):
            sums += whole(w[j])
            if sums * den > target:
                break
        tokens.append(kept[at])
        logprobs.append(d[kept[at]] - np.log(total))
    return np.array(tokens), np.array(logprobs)
