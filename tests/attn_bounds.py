"""Error bounds of the attention outputs, element by element, from the formulas.

u is the unit roundoff of the stored type (2^-8 in bf16, 2^-24 in fp32), e that
of fp32.  A fp32 sum of n products is off by at most n e times the sum of their
magnitudes, whatever its order.

scores     s = scale q.k          off by  es = (D + 4) e scale |q|.|k|  (plus one rounding of s)
P          exp(s - lse), rounded to the stored type as the next product's operand:
                                  relative  ep + u,  ep = 2 max es + 16 e (1 + max|s|)
o          sum P v                (u + ep + n e) sum P|v|  + u |o|
lse                               max es + 8 e (1 + |lse|) + n e
delta      sum do o, from the stored o:   sum |do| (err o) + D e sum |do||o|
dS         P (dP - delta), rounded:  (u + ep + 4 e)|dS| + P (D e |do|.|v| + err delta + 4 e |delta|)
dq         scale sum dS k         scale sum (err dS)|k| + (n e) scale sum |dS||k| + u |dq|;  dk likewise
dv         sum P do               (u + ep + n e) sum P|do| + u |dv|

Sums over the heads of a group add their bounds.  2 u stands for u where a value
and the operand it is made from are both rounded.  Nothing here comes from a run.
"""
import numpy as np

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def bounds(dtype, q, k, v, out, see, scale, do=None):
    """`out`: the oracle's values of one head."""
    u = U[dtype]
    d, n = q.shape[1], see.shape[1]
    aq, ak, av = np.abs(q), np.abs(k), np.abs(v)
    es = np.where(see, (d + 4) * E * abs(scale) * (aq @ ak.T), 0.0).max(axis=1, initial=0.0)
    top = np.where(see, np.abs(scale * (q @ k.T)), 0.0).max(axis=1, initial=0.0)
    lse = np.where(np.isfinite(out["lse"]), out["lse"], 0.0)
    ep = 2 * es + 16 * E * (1 + top + np.abs(lse))
    p = out["p"]
    rel = u + ep + n * E
    b = {"lse": es + 8 * E * (1 + np.abs(lse)) + n * E,
         "o": rel[:, None] * (p @ av) + u * np.abs(out["o"])}
    if do is not None:
        ado = np.abs(do)
        delta = (do * out["o"]).sum(axis=1)
        e_delta = (ado * b["o"]).sum(axis=1) + d * E * (ado * np.abs(out["o"])).sum(axis=1)
        ds = np.abs(out["ds"])
        e_ds = (rel + 4 * E)[:, None] * ds + p * (d * E * (ado @ av.T) + (e_delta + 4 * E * np.abs(delta))[:, None])
        s = abs(scale)
        b["dq"] = s * (e_ds @ ak) + n * E * s * (ds @ ak) + u * np.abs(out["dq"])
        m = see.shape[0]
        b["dk"] = s * (e_ds.T @ aq) + m * E * s * (ds.T @ aq)
        b["dv"] = (p * (rel + m * E)[:, None]).T @ ado
        b["dk_round"], b["dv_round"] = u, u   # times |the group's sum|, added by the caller
    return b


def check(got, ref, bound, name):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), f"{name}: finite in other places"
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), f"{name}: infinities"
    over = np.abs(got[fine] - ref[fine]) / (bound[fine] + 1e-30)
    worst = float(over.max()) if over.size else 0.0
    print(f"  {name}: error at most {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound"
