"""The attention oracle against closed forms, torch in float64, and differences."""
import numpy as np
import pytest

from oracle import attn_oracle as A


@pytest.mark.parametrize("lq,lk,window,sinks", [(1, 1, 0, 0), (7, 7, 3, 2), (5, 12, 4, 0), (6, 4, 0, 0),
                                                (9, 9, 1, 0), (9, 9, 1, 30), (0, 3, 0, 0), (3, 0, 2, 2)])
def test_visible_against_the_definition(lq, lk, window, sinks):
    see = A.visible(lq, lk, window, sinks)
    for i in range(lq):
        for j in range(lk):
            p = i + lk - lq
            assert see[i, j] == (j <= p and (window == 0 or j > p - window or j < sinks))


@pytest.mark.parametrize("lq,lk,window,sinks", [(6, 6, 0, 0), (5, 9, 3, 2), (7, 4, 0, 0)])
def test_against_torch_autograd(lq, lk, window, sinks):
    import torch
    rng = np.random.default_rng(lq * 10 + lk)
    q, k, v, do = (rng.standard_normal((n, 8)) for n in (lq, lk, lk, lq))
    see = A.visible(lq, lk, window, sinks)
    out = A.attend(q, k, v, see, 0.3, do)
    tq, tk, tv = (torch.tensor(a, requires_grad=True) for a in (q, k, v))
    rows = see.any(axis=1)
    s = (0.3 * tq @ tk.T).masked_fill(~torch.tensor(see), -np.inf)[torch.tensor(rows)]
    o = torch.softmax(s, -1) @ tv
    o.backward(torch.tensor(do)[torch.tensor(rows)])
    assert np.allclose(out["o"][rows], o.detach().numpy(), atol=1e-12)
    assert np.allclose(out["lse"][rows], torch.logsumexp(s, -1).detach().numpy(), atol=1e-12)
    assert np.all(out["o"][~rows] == 0) and np.all(out["lse"][~rows] == -np.inf)
    for name, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        assert np.allclose(out[name], t.grad.numpy(), atol=1e-12), name


def test_gradients_against_central_differences():
    rng = np.random.default_rng(3)
    q, k, v, do = (rng.standard_normal((5, 4)) for _ in range(4))
    see = A.visible(5, 5, 2, 1)
    out = A.attend(q, k, v, see, 0.5, do)
    f = lambda: float((A.attend(q, k, v, see, 0.5)["o"] * do).sum())
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(x)
        for at in np.ndindex(*x.shape):
            h, x0 = 1e-5, x[at]
            x[at] = x0 + h
            up = f()
            x[at] = x0 - h
            num[at] = (up - f()) / (2 * h)
            x[at] = x0
        assert np.allclose(out[name], num, atol=1e-8), name


def test_hidden_rows_have_no_part():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((6, 4)) for _ in range(3))
    see = A.visible(6, 6, 2, 0)
    ref = A.attend(q, k, v, see, 0.5)
    k[1], v[1] = np.inf, np.nan
    out = A.attend(q, k, v, see, 0.5)
    rows = ~see[:, 1]
    assert np.allclose(out["o"][rows], ref["o"][rows], rtol=0, atol=1e-13)


def test_equal_scores_average_the_visible_values():
    v = np.arange(12.0).reshape(6, 2)
    out = A.attend(np.zeros((6, 2)), np.ones((6, 2)), v, A.visible(6, 6, 3, 1), 1.0)
    assert np.allclose(out["o"][5], v[[0, 3, 4, 5]].mean(axis=0)) and np.isclose(out["lse"][5], np.log(4))


def test_pages_keep_every_sequence_through_fork_extend_free_and_compact():
    rng = np.random.default_rng(5)
    pages, page = 40, 4
    c = A.Pages(np.zeros(pages), -np.ones((8, 6)), np.zeros(8), np.zeros((2, pages, 1, page, 1)),
                np.zeros((2, pages, 1, page, 1)))
    text = {}

    def write(s, n):
        assert c.extend([s], [n])
        rows = rng.standard_normal((2, n, 1, 1))
        for layer in (0, 1):
            c.append([s], [rows[layer]], [-rows[layer]], layer)
        text[s] = np.concatenate([text.get(s, np.zeros((2, 0, 1, 1))), rows], axis=1)

    def intact():
        for s, t in text.items():
            for layer in (0, 1):
                assert np.array_equal(c.rows(c.k, s, layer), t[layer])
                assert np.array_equal(c.rows(c.v, s, layer), -t[layer])
        held = [int(p) for s in text for p in c.table[s, :c.held(s)]]
        assert np.array_equal(np.bincount(held, minlength=pages), c.refs)

    write(0, 9)
    write(1, 4)
    c.fork([0, 0, 1], [2, 3, 4])
    for a, b in ((0, 2), (0, 3), (1, 4)):
        text[b] = text[a]
    intact()
    for s, n in ((2, 1), (0, 3), (3, 7), (4, 1)):
        write(s, n)
        intact()
    c.free([0, 1])
    del text[0], text[1]
    intact()
    n = c.compact()
    assert np.all(c.refs[n:] == 0) and np.all(c.refs[:n] > 0)
    intact()
    before = c.refs.copy()
    assert not c.extend([2], [100]) and np.array_equal(c.refs, before)   # past the table's width
    c.refs[n:] = 1
    assert not c.extend([2, 3], [2, 20 - int(c.lens[3])])                # no page is free
