"""Attention over inputs that hold NaN in every row: what a training step is made
of once it has diverged.  Exactly what the formulas make NaN is NaN, at the speed
of a sound step."""
import numpy as np
import pytest

from attn_bounds import check
from helpers import to_np
from oracle import attn_oracle as A
from test_gpu_attn import cu, oracle_window, rand, run_window, st  # noqa: F401

pytestmark = pytest.mark.gpu

NAN = float("nan")
DIM = 3   # the element that is NaN in every row
CASES = [   # lens, keys before them, heads, kv heads, dim, window, sinks
    ([200, 40, 70, 1], [0, 100, -20, 5], 4, 2, 72, 33, 2),
    ([300], [0], 8, 1, 128, 0, 0),
    ([1100], [0], 1, 1, 64, 0, 0),       # keys and queries in parts
    ([9], [2400], 4, 2, 128, 0, 0),      # keys in parts, most of them before the queries
]


def sights(lq, lk, window, sinks):
    """Queries that see a key, keys that some query sees, and the pairs of each sequence."""
    see = [A.visible(a, b, window, sinks) for a, b in zip(lq, lk)]
    return np.concatenate([s.any(axis=1) for s in see]), np.concatenate([s.any(axis=0) for s in see]), see


def compare(got, ref, bound, nan, name):
    """NaN where `nan` says, the others within their bounds."""
    assert np.array_equal(np.isnan(got), nan), f"{name}: NaN in other places"
    check(np.where(nan, 0.0, got), np.where(nan, 0.0, ref), bound, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"q{sum(c[0])}-h{c[2]}_{c[3]}-d{c[4]}-w{c[5]}")
def test_nan_in_one_element_of_every_row(st, dtype, which, case):
    lq, past, h, hk, d, window, sinks = case
    print(case, dtype, which, flush=True)
    ops = [rand((n, m, d), dtype, 400 + i) for i, (n, m) in
           enumerate(((sum(lq), h), (sum(lq) + sum(past), hk), (sum(lq) + sum(past), hk), (sum(lq), h)))]
    lk = [a + b for a, b in zip(lq, past)]
    ref, bound = oracle_window(dtype, ops, lq, lk, h, hk, window, sinks, d ** -0.5)
    sees, seen, _ = sights(lq, lk, window, sinks)
    bad = [t.clone() for t in ops]
    bad["q k v do".split().index(which)][:, :, DIM] = NAN
    _, _, got = run_window(st, dtype, lq, past, h, hk, d, window, sinks, qkv=bad)
    rows = lambda x, n: np.broadcast_to(x[:, None, None], (len(x), n, d))
    one = np.arange(d) == DIM
    none_q, none_k = np.zeros((len(sees), h, d), bool), np.zeros((len(seen), hk, d), bool)
    scores = which in ("q", "k")   # a NaN in every score: everything that sees or is seen
    nan = {"o": rows(sees, h) if scores else rows(sees, h) & one if which == "v" else none_q,
           "dq": rows(sees, h), "dk": rows(seen, hk),
           "dv": rows(seen, hk) if scores else rows(seen, hk) & one if which == "do" else none_k}
    nan["lse"] = np.broadcast_to(sees[:, None], (len(sees), h)) if scores else np.zeros((len(sees), h), bool)
    fine = np.isfinite(ref["lse"])
    assert np.array_equal(got["lse"][~fine], ref["lse"][~fine])   # -inf where nothing is seen
    compare(np.where(fine, got["lse"], 0), np.where(fine, ref["lse"], 0), bound["lse"], nan["lse"], "lse")
    for n in ("o", "dq", "dk", "dv"):
        compare(got[n], ref[n], bound[n], nan[n], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_a_nan_of_its_own_does_not_hide_what_a_row_does_not_see(st, dtype, bad):
    """Beside the NaN of every row, one key (one query) holds nothing finite: rows that do not see
    it keep every other element."""
    lens, h, hk, d, window, sinks = [230], 4, 2, 128, 25, 1
    ops = [rand((230, n, d), dtype, 410 + i) for i, n in enumerate((h, hk, hk, h))]
    ref, bound = oracle_window(dtype, ops, lens, lens, h, hk, window, sinks, d ** -0.5)
    see = A.visible(230, 230, window, sinks)
    others = np.arange(d) != DIM
    for where in (77, 190):
        print(dtype, bad, where, flush=True)
        q, k, v, do = (t.clone() for t in ops)
        v[:, :, DIM] = NAN
        v[where] = bad
        _, _, got = run_window(st, dtype, lens, [0], h, hk, d, window, sinks, qkv=(q, k, v, do))
        far = ~see[:, where]
        assert np.isnan(got["o"][far][:, :, DIM]).all() and not np.isfinite(got["o"][~far]).any()
        check(got["o"][far][:, :, others], ref["o"][far][:, :, others], bound["o"][far][:, :, others], "o")
        check(got["dv"], ref["dv"], bound["dv"], "dv")
        q, k, v, do = (t.clone() for t in ops)
        do[:, :, DIM] = NAN
        do[where] = bad
        _, _, got = run_window(st, dtype, lens, [0], h, hk, d, window, sinks, qkv=(q, k, v, do))
        far = ~see[where]
        assert np.isnan(got["dv"][far][:, :, DIM]).all() and not np.isfinite(got["dv"][~far]).any()
        check(got["dv"][far][:, :, others], ref["dv"][far][:, :, others], bound["dv"][far][:, :, others], "dv")
        check(got["o"], ref["o"], bound["o"], "o")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["q", "k", "v", "do", "all"])
def test_a_diverged_step_takes_no_longer(st, dtype, which):
    """Each row done again one key at a time would take a thousand times as long."""
    import torch
    c = cu([1024] * 4)
    ops = [rand((4096, n, 128), dtype, 420 + i) for i, n in enumerate((8, 2, 2, 8))]

    def step(q, k, v, do):
        f = st.staple_attn_fwd(q, k, v, c, c)
        st.staple_attn_bwd(do, q, k, v, f["o"], f["lse"], c, c)

    def fastest(x):
        best = float("inf")
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            step(*x)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    bad = [t.clone() for t in ops]
    for n, t in zip("q k v do".split(), bad):
        if which in (n, "all"):
            t[:, :, DIM] = NAN
    sound, diverged = fastest(ops), fastest(bad)
    print(f"  {dtype} {which}: {1e3 * sound:.0f} us sound, {1e3 * diverged:.0f} diverged", flush=True)
    assert diverged <= 4 * sound


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hk,d", [(4, 2, 72), (1, 1, 128), (2, 2, 64)])
def test_no_keys_and_no_queries_at_all(st, dtype, h, hk, d):
    """Sequences without a single key (o = 0, lse = -inf, dq = 0), and without a single query (dk =
    dv = 0), whatever the other side holds."""
    import torch
    n, mask = 150, dict(window=20, sinks=3)
    c, none = cu([100, 0, 50]), cu([0, 0, 0])
    rows, keys = torch.full_like(rand((n, h, d), dtype, 430), NAN), torch.full_like(rand((n, hk, d), dtype, 431), NAN)
    print(dtype, h, hk, d, "no keys", flush=True)
    f = st.staple_attn_fwd(rows, keys[:0], keys[:0], c, none, **mask)
    b = st.staple_attn_bwd(rows, rows, keys[:0], keys[:0], f["o"], f["lse"], c, none, **mask)
    assert (f["o"] == 0).all() and (f["lse"] == -float("inf")).all() and (b["dq"] == 0).all() and b["dk"].numel() == 0
    print(dtype, h, hk, d, "no queries", flush=True)
    f = st.staple_attn_fwd(rows[:0], keys, keys, none, c, **mask)
    assert f["o"].numel() == 0 and f["lse"].numel() == 0
    b = st.staple_attn_bwd(rows[:0], rows[:0], keys, keys, f["o"], f["lse"], none, c, **mask)
    assert (b["dk"] == 0).all() and (b["dv"] == 0).all() and b["dq"].numel() == 0
    assert st.staple_get_device_error() == 0
