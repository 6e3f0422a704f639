"""The oracle of embedding, norms, loss and sampling: gradients against differences, tokens against
their definition drawn out."""
import numpy as np
import pytest

from oracle import model_oracle as M


def differences(f, a, step=1e-6):
    """Central differences of the number f(a) by every element of a."""
    d = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + step
        up = f(a)
        a[i] = keep - step
        d[i] = (up - f(a)) / (2 * step)
        a[i] = keep
    return d


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "vector", "rows"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_gradients_are_differences(pre, post, gate, residual):
    rng = np.random.default_rng(3)
    n, d, scale, eps = 3, 5, 0.75, 1e-3
    leaf = {"x": rng.normal(size=(n, d)) if residual else None, "z": rng.normal(size=(n, d)),
            "w_pre": 1 + rng.normal(size=d) / 3 if pre else None, "w_post": 1 + rng.normal(size=d) / 3 if post else None,
            "gate": None if gate is None else rng.normal(size=d if gate == "vector" else (n, d))}
    dr, dh = rng.normal(size=(n, d)), rng.normal(size=(n, d))
    how = dict(pre=pre, post=post, scale=scale)

    def forward(**change):
        f = {**leaf, **change}
        return M.norm(f["x"], f["z"], w_pre=f["w_pre"], w_post=f["w_post"], gate=f["gate"], eps=eps, **how)

    def loss(**change):
        o = forward(**change)
        return (dr * o["r"]).sum() + ((dh * o["h"]).sum() if pre else 0.0)

    o = forward()
    got = M.norm_grad(dr, dh if pre else None, o["r"], leaf["z"], o["rstd_r"], o["rstd_z"], w_pre=leaf["w_pre"],
                      w_post=leaf["w_post"], gate=leaf["gate"], **how)
    if gate == "vector":
        got["dgate"] = got["dgate"].sum(axis=0)
    for name, grad in (("x", "dx"), ("z", "dz"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        if leaf[name] is not None:
            want = differences(lambda a: loss(**{name: a}), leaf[name].copy())
            np.testing.assert_allclose(got[grad], want, rtol=1e-6, atol=1e-8)


def test_norm_alone_is_the_same_without_a_block():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(4, 6))
    a, b = M.norm(x, None), M.norm(None, x)
    np.testing.assert_array_equal(a["h"], b["h"])
    np.testing.assert_allclose((a["h"] ** 2).mean(axis=1), 1.0, rtol=1e-4)


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(5)
    ids = np.array([4, 1, 4, 0, 4])
    table, dy = rng.normal(size=(6, 3)), rng.normal(size=(5, 3))
    want = differences(lambda t: (dy * M.embed(t, ids, 2.0)).sum(), table.copy())
    got = np.zeros_like(table)
    for t, row in M.embed_grad(dy, ids, 2.0).items():
        got[t] = row
    np.testing.assert_allclose(got, want, atol=1e-8)


def test_loss_gradient_is_differences():
    rng = np.random.default_rng(6)
    l, t, g = rng.normal(size=(4, 7)), np.array([3, -1, 0, 6]), rng.normal(size=4)
    want = differences(lambda a: (g * M.xent(a, t)["loss"]).sum(), l.copy())
    np.testing.assert_allclose(M.xent(l, t, g)["d_logits"], want, atol=1e-8)


def test_loss_of_impossible_classes():
    inf = np.inf
    l = np.array([[0.0, -inf, 1.0], [-inf, -inf, -inf], [0.0, -inf, 1.0]])
    o = M.xent(l, [0, 1, 1], [1.0, 1.0, 1.0])
    assert np.isfinite(o["loss"][0]) and o["loss"][1] == inf and o["loss"][2] == inf
    assert o["d_logits"][0, 1] == 0 and not o["d_logits"][1].any()
    assert o["d_logits"][2, 1] == -1


def test_sampling_follows_the_kept_shares():
    """Over an even grid of random numbers a token comes up as often as its share says."""
    l = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    n = 1000
    u = (np.arange(n) + 0.5) / n
    share = lambda **k: np.bincount(M.sample(np.repeat(l, n, 0), u, **{a: np.full(n, b) for a, b in k.items()})[0],
                                    minlength=4) / n
    np.testing.assert_allclose(share(), [0.1, 0.4, 0.2, 0.3], atol=1e-3)
    np.testing.assert_allclose(share(top_k=2), [0, 4 / 7, 0, 3 / 7], atol=1e-3)
    np.testing.assert_allclose(share(top_p=0.75), [0, 4 / 9, 2 / 9, 3 / 9], atol=1.1e-3)
    np.testing.assert_allclose(share(top_p=0.69), [0, 4 / 7, 0, 3 / 7], atol=1e-3)
    np.testing.assert_allclose(share(min_p=0.49), [0, 4 / 9, 2 / 9, 3 / 9], atol=1.1e-3)
    np.testing.assert_allclose(share(top_k=3, top_p=0.5), [0, 4 / 7, 0, 3 / 7], atol=1e-3)
    np.testing.assert_allclose(share(temperature=0.5), np.array([1, 16, 4, 9]) / 30, atol=1e-3)
    np.testing.assert_array_equal(share(temperature=0.0), [0, 1, 0, 0])
    np.testing.assert_array_equal(share(top_p=0.0), [0, 1, 0, 0])


def test_sampling_ties_and_ruled_out_tokens():
    inf = np.inf
    l = np.array([[1.0, 2.0, 2.0, 2.0, -inf]])
    assert M.sample(l, [0.99], top_k=[2])[0] == [2]      # the first two of three
    assert M.sample(l, [0.0], top_k=[1])[0] == [1]
    assert M.sample(l, [0.999999])[0] == [3]
    assert M.sample(l, [0.0])[0] == [0]
    token, logprob = M.sample(np.full((1, 3), -inf), [0.5])
    assert token == [-1] and logprob == [-inf]
    token, logprob = M.sample(np.array([[np.nan, 0.0]]), [0.0])
    assert token == [1] and logprob == [0.0]
    token, logprob = M.sample(np.array([[0.0, inf, inf]]), [0.6], temperature=[0.7])
    assert token == [2] and logprob == pytest.approx(-np.log(2))
