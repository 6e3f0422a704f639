"""Error bounds of the embedding, the norms and the loss, element by element, from the formulas.

u is the unit roundoff of a stored type (2^-8 in bf16, 2^-24 in fp32), E that of fp32.  A sum of
terms of one sign in fp32 is off by at most E times the longest chain of additions that a term goes
through, relative to it; of terms of both signs by as much of the sum of their magnitudes.

A row's sum (norms): a lane adds up to 16 terms, a wave's lanes join in 6 steps, up to 16
waves in turn: chains of CHAIN = 40 and fewer.  1 / rms: half of the sum's error, the division by
d, eps, and the reciprocal square root, 2 units in the last place: CHAIN / 2 + 8 roundings.
A sum over rows or positions counts one rounding a term and 32 for the joining of parts.
Nothing here comes from a run.
"""
import numpy as np

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": E}
CHAIN = 40
RSTD = (CHAIN / 2 + 8) * E


def one(v):
    return 1.0 if v is None else np.abs(v)


def embed(y, out):
    return (U[out] + 2 * E) * np.abs(y)


def embed_grad(dy, ids, scale):
    """{token: bound}."""
    total, count = {}, {}
    for i, t in enumerate(np.asarray(ids).tolist()):
        total[t] = total.get(t, 0.0) + np.abs(scale * dy[i])
        count[t] = count.get(t, 0) + 1
    return {t: (count[t] + 34) * E * total[t] for t in total}


def norm(ref, x, z, dtype, r_dtype, *, w_pre=None, w_post=None, gate=None, pre=True, post=False, scale=1.0, **_):
    """Bounds of r, h, rstd_r, rstd_z for the oracle's values."""
    b = {"rstd_z": None if ref["rstd_z"] is None else RSTD * ref["rstd_z"]}
    r = ref["r"]
    if z is not None:
        part = np.abs(r if x is None else r - x)       # |scale gate b|
        part = np.maximum(part, 0.0)
        e_r = (RSTD + 6 * E) * part + E * np.abs(r)     # of the sum before it is stored
    else:
        e_r = np.zeros_like(r)
    b["sum"] = e_r
    b["r"] = e_r + U[r_dtype] * np.abs(r)
    if pre:
        size = np.sqrt((r * r).sum(axis=1))
        moved = np.sqrt((e_r * e_r).sum(axis=1)) / np.where(size == 0, 1.0, size)
        b["rstd_r"] = (RSTD + moved) * ref["rstd_r"]
        inv = ref["rstd_r"][:, None]
        b["h"] = one(w_pre) * inv * (e_r + np.abs(r) * (RSTD + 3 * E + moved[:, None])) + U[dtype] * np.abs(ref["h"])
    return b


def norm_grad(ref, dr, dh, r, z, rstd_r, rstd_z, dtype, r_dtype, *, w_pre=None, w_post=None, gate=None, pre=True,
              post=False, scale=1.0, e_r=0.0, **_):
    """Bounds of the gradients from r (off by e_r) and the stored 1 / rms."""
    n, d = r.shape
    rows = (n + 36) * E
    b = {}
    e_g = E * (0.0 if dr is None else np.abs(dr))
    if pre:
        inv = rstd_r[:, None]
        hat, t = np.abs(r * inv), np.abs(dh) * one(w_pre)
        e_hat = inv * e_r
        mean = (t * hat).mean(axis=1, keepdims=True)
        e_mean = (CHAIN + 12) * E * mean + (t * e_hat).mean(axis=1, keepdims=True)
        e_g = e_g + inv * (6 * E * t + hat * e_mean + e_hat * mean) + E * np.abs(ref["dx"])
        b["dw_pre"] = rows * (np.abs(dh) * hat).sum(axis=0) + (np.abs(dh) * e_hat).sum(axis=0)
    e_g = e_g + np.zeros_like(r)
    b["dx"] = e_g + U[r_dtype] * np.abs(ref["dx"])
    if z is None:
        return b
    hat = np.abs(z * (rstd_z[:, None] if post else 1.0))
    w = one(w_post) if post else 1.0
    e_q = abs(scale) * e_g
    q = np.abs(scale * ref["dx"])
    if gate is not None:
        e_gate = hat * w * e_q + 6 * E * q * hat * w
        b["dgate_sum"] = (e_gate + rows * q * hat * w).sum(axis=0)
        b["dgate"] = e_gate + U[dtype] * np.abs(ref["dgate"])
        e_q, q = np.abs(gate) * e_q, q * np.abs(gate)
    e_q = e_q + 3 * E * q
    if post:
        b["dw_post"] = (hat * e_q + rows * q * hat).sum(axis=0)
        e_q, q = w * e_q + E * w * q, q * w
        e_mean = (hat * e_q + (CHAIN + 6) * E * q * hat).mean(axis=1, keepdims=True)
        mean = (q * hat).mean(axis=1, keepdims=True)
        e_q = rstd_z[:, None] * (e_q + 4 * E * q + hat * (e_mean + 6 * E * mean))
    b["dz"] = e_q + U[dtype] * np.abs(ref["dz"]) + E * np.abs(ref["dz"])
    return b


def xent(ref, logits, targets, g, dtype, chain, from_lse=False):
    """A term exp(l - m) is off by 2 |l - m| + 4 units (the difference, its product with log2 e, the
    exponential), a row's sum by `chain` additions and changes of reference; the loss by that,
    the logarithm (2 units) and the last sums.  The gradient of a forward divides by the sum,
    staple_xent_bwd goes by the stored lse."""
    top = logits.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(logits), np.abs(logits - np.where(np.isfinite(top), top, 0.0)), 0.0)
    term = (2 * far + 6) * E
    total = (ref["p"] * term).sum(axis=1) + chain * E
    fine = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
    span = np.log(logits.shape[1]) + 1.0
    e_lse = total + 3 * E * span + 2 * E * np.abs(fine)
    b = {"lse": e_lse, "loss": e_lse + E * np.where(np.isfinite(ref["loss"]), np.abs(ref["loss"]), 0.0)}
    if g is not None:
        share = term + (e_lse if from_lse else total)[:, None] + 4 * E + \
            (2 * E * (np.abs(fine)[:, None] + far) if from_lse else 0.0)
        scale = np.abs(np.asarray(g, dtype=np.float64))[:, None]
        b["d_logits"] = scale * ref["p"] * share + (2 * E + U[dtype]) * np.abs(ref["d_logits"])
    return b
