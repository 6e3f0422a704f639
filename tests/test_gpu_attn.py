"""Attention over packed sequences, decode attention over pages, and the page
operations on the GPU against the float64 oracle."""
import numpy as np
import pytest

from attn_bounds import bounds, check
from helpers import to_np
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

TORCH = {"bf16": "bfloat16", "f32": "float32"}


@pytest.fixture(scope="module")
def st():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import token_indexed_ffn_amd as st
    st.lib()
    return st


def rand(shape, dtype, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(getattr(torch, TORCH[dtype])).cuda()


def ints(values):
    import torch
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def cu(lens):
    return ints([0] + list(np.cumsum(lens)))


# lens of queries, cached keys before them (negative: fewer keys than queries), heads, kv heads, dim, window, sinks
WINDOW_CASES = [
    ([1], [0], 1, 1, 8, 0, 0),
    ([1, 1, 1], [0, 5, 100], 4, 2, 64, 3, 1),
    ([0, 1, 31, 32, 33, 0], [0] * 6, 2, 2, 128, 0, 0),
    ([63, 64, 65, 129], [0] * 4, 4, 4, 128, 0, 0),
    ([127, 200], [0, 0], 8, 2, 64, 17, 3),
    ([130, 5], [70, 300], 6, 1, 72, 50, 0),
    ([40, 70, 3], [-13, -70, -3], 2, 1, 64, 9, 2),
    ([90], [0], 3, 3, 40, 1, 0),
    ([150], [0], 2, 2, 128, 1000, 1000),
    ([260], [0], 2, 1, 96, 33, 200),
    ([700], [0], 2, 2, 128, 100, 70),
    ([513, 300], [100, 0], 4, 1, 128, 0, 0),
    ([300], [900], 16, 2, 128, 256, 4),
    ([33] * 20, [0] * 20, 8, 8, 64, 0, 0),
]


def run_window(st, dtype, lq, past, h, hk, d, window, sinks, seed=0, qkv=None, scale=None):
    import torch
    lk = [max(0, a + b) for a, b in zip(lq, past)]
    q, k, v, do = qkv or [rand((sum(n), m, d), dtype, seed + i) for i, (n, m) in
                          enumerate(((lq, h), (lk, hk), (lk, hk), (lq, h)))]
    cq, ck = cu(lq), cu(lk)
    fwd = st.staple_attn_fwd(q, k, v, cq, ck, window=window, sinks=sinks, scale=scale)
    bwd = st.staple_attn_bwd(do, q, k, v, fwd["o"], fwd["lse"], cq, ck, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    assert st.staple_get_device_error() == 0
    return (q, k, v, do), lk, {n: to_np(t) for n, t in (fwd | bwd).items()}


def oracle_window(dtype, operands, lq, lk, h, hk, window, sinks, scale):
    """Values and bounds of a packed batch."""
    q, k, v, do = (to_np(t) for t in operands)
    group = h // hk
    ref = {n: np.zeros(s) for n, s in (("o", q.shape), ("lse", q.shape[:2]), ("dq", q.shape), ("dk", k.shape),
                                       ("dv", v.shape))}
    bound = {n: np.zeros(a.shape) for n, a in ref.items()}
    a = x = 0
    for nq, nk in zip(lq, lk):
        see = A.visible(nq, nk, window, sinks)
        rq, rk = slice(a, a + nq), slice(x, x + nk)
        for i in range(h):
            ops = q[rq, i], k[rk, i // group], v[rk, i // group]
            out = A.attend(*ops, see, scale, do[rq, i])
            b = bounds(dtype, *ops, out, see, scale, do[rq, i])
            for n in ("o", "lse", "dq"):
                ref[n][rq, i], bound[n][rq, i] = out[n], b[n]
            for n in ("dk", "dv"):
                ref[n][rk, i // group] += out[n]
                bound[n][rk, i // group] += b[n]
        a, x = a + nq, x + nk
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for n in ("dk", "dv"):
        bound[n] += u * np.abs(ref[n]) + group * 2.0 ** -24 * np.abs(ref[n])
    return ref, bound


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", WINDOW_CASES, ids=lambda c: f"q{sum(c[0])}x{len(c[0])}-h{c[2]}_{c[3]}-d{c[4]}-w{c[5]}-s{c[6]}")
def test_window_attention_and_its_gradients(st, dtype, case):
    lq, past, h, hk, d, window, sinks = case
    print(case, dtype, flush=True)
    ops, lk, got = run_window(st, dtype, lq, past, h, hk, d, window, sinks)
    ref, bound = oracle_window(dtype, ops, lq, lk, h, hk, window, sinks, d ** -0.5)
    for n in ref:
        check(got[n], ref[n], bound[n], n)


# few queries of many keys: the keys in parts
LONG_CASES = [
    ([1], [599], 1, 1, 64, 0, 0),
    ([7], [2993], 2, 1, 128, 0, 0),
    ([33, 1, 0, 2], [1500, 40, 300, 2100], 4, 2, 72, 0, 0),
    ([20], [2500], 2, 2, 128, 1000, 300),
    ([150], [1200], 1, 1, 128, 700, 64),
    ([130, 40], [-100, 1800], 2, 1, 40, 0, 0),
    ([1100], [0], 1, 1, 64, 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", LONG_CASES, ids=lambda c: f"q{sum(c[0])}x{len(c[0])}-p{max(c[1])}-h{c[2]}_{c[3]}-d{c[4]}-w{c[5]}-s{c[6]}")
def test_window_attention_few_queries_of_many_keys(st, dtype, case):
    lq, past, h, hk, d, window, sinks = case
    print(case, dtype, flush=True)
    ops, lk, got = run_window(st, dtype, lq, past, h, hk, d, window, sinks, seed=20)
    ref, bound = oracle_window(dtype, ops, lq, lk, h, hk, window, sinks, d ** -0.5)
    for n in ref:
        check(got[n], ref[n], bound[n], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_few_queries_never_read_a_hidden_key(st, dtype):
    """Keys before the window and after the query hold NaN and infinities in parts of their own
    and at the edges of others."""
    import torch
    lk, lq, h, d, window, sinks = 2600, 5, 2, 64, 900, 40
    q, k, v = rand((lq, h, d), dtype, 60), rand((lk, 1, d), dtype, 61), rand((lk, 1, d), dtype, 62)
    cq, ck = cu([lq]), cu([lk])
    ref, bound = oracle_window(dtype, (q, k, v, torch.zeros_like(q)), [lq], [lk], h, 1, window, sinks, d ** -0.5)
    want = st.staple_attn_fwd(q, k, v, cq, ck, window=window, sinks=sinks)
    k[sinks:lk - lq + 1 - window], v[sinks:lk - lq + 1 - window] = float("nan"), float("inf")
    got = st.staple_attn_fwd(q, k, v, cq, ck, window=window, sinks=sinks)
    assert torch.equal(got["lse"], want["lse"])
    for n in ("o", "lse"):
        check(to_np(got[n]), ref[n], bound[n], n)
    k[lk - 2], v[lk - 2] = float("nan"), float("nan")   # the last two queries see it, the others don't
    got = st.staple_attn_fwd(q, k, v, cq, ck, window=window, sinks=sinks)
    assert torch.isfinite(got["o"][:3]).all() and torch.isnan(got["o"][3:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_gradients_in_parts_never_read_a_hidden_row(st, dtype):
    """One head of 1100 tokens: a late key holds NaN, which no earlier query's dq may take; an
    early query's gradient does, which no later key's dk, dv may take."""
    n, h, d = 1100, 1, 64
    ops, lk, _ = run_window(st, dtype, [n], [0], h, h, d, 0, 0, seed=80)
    q, k, v, do = ops
    ref, bound = oracle_window(dtype, ops, [n], lk, h, h, 0, 0, d ** -0.5)
    c = cu([n])
    fwd = st.staple_attn_fwd(q, k, v, c, c)
    bad_k, bad_v, bad_do = k.clone(), v.clone(), do.clone()
    bad_k[1090], bad_v[1090], bad_do[5] = float("nan"), float("inf"), float("nan")
    late = st.staple_attn_bwd(do, q, bad_k, bad_v, fwd["o"], fwd["lse"], c, c)
    check(to_np(late["dq"])[:1090], ref["dq"][:1090], bound["dq"][:1090], "dq")
    early = st.staple_attn_bwd(bad_do, q, k, v, fwd["o"], fwd["lse"], c, c)
    for name in ("dk", "dv"):
        check(to_np(early[name])[6:], ref[name][6:], bound[name][6:], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_in_a_graph(st, dtype):
    """Forward and backward, split and not, captured once and replayed on new inputs."""
    import torch
    for lens, window, sinks in (([700], 0, 0), ([40, 130], 33, 2)):
        c, n = cu(lens), sum(lens)
        q, k, v, do = (rand((n, 2, 64), dtype, 90 + i) for i in range(4))

        def step():
            f = st.staple_attn_fwd(q, k, v, c, c, window=window, sinks=sinks)
            return f | st.staple_attn_bwd(do, q, k, v, f["o"], f["lse"], c, c, window=window, sinks=sinks)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for i in range(4):
            for j, t in enumerate((q, k, v, do)):
                t.copy_(rand(t.shape, dtype, 100 + 10 * i + j))
            want = step()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for name in want:
                assert torch.equal(held[name], want[name]), (i, name)
        assert st.staple_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_peaked_scores(st, dtype):
    """Scores of a few hundred: softmax rows that one key takes whole."""
    lq, h, d = [200], 2, 64
    ops = [rand((200, h, d), dtype, 50 + i, s) for i, s in enumerate((6.0, 6.0, 1.0, 1.0))]
    ops, lk, got = run_window(st, dtype, lq, [0], h, h, d, 60, 2, qkv=ops, scale=1.0)
    ref, bound = oracle_window(dtype, ops, lq, lk, h, h, 60, 2, 1.0)
    for n in ref:
        check(got[n], ref[n], bound[n], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_of_one_key_is_its_value(st, dtype):
    """A window of one key, and scores far from zero: the weight is 1 in the stored type too."""
    import torch
    lens, h, hk, d = [1, 70, 200], 4, 2, 72
    q, k, v = (rand((271, n, d), dtype, 70 + i, s) for i, (n, s) in enumerate(((h, 3.0), (hk, 3.0), (hk, 1.0))))
    c = cu(lens)
    got = st.staple_attn_fwd(q, k, v, c, c, window=1)
    want = v.repeat_interleave(h // hk, dim=1)
    if dtype == "bf16":
        assert torch.equal(got["o"], want)
    else:   # an exponential of at most (d + 4) 2^-24 |s| from zero over a sum of itself
        assert ((got["o"] - want).abs() <= 2.0 ** -22 * want.abs()).all()


def test_window_attention_negative_and_zero_scale(st):
    for scale in (-0.2, 0.0):
        ops, lk, got = run_window(st, "bf16", [140], [0], 2, 1, 64, 0, 0, seed=3, scale=scale)
        ref, bound = oracle_window("bf16", ops, [140], lk, 2, 1, 0, 0, scale)
        for n in ref:
            check(got[n], ref[n], bound[n], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_reads_and_writes_strided_views(st, dtype):
    """q, k, v as slices of one fused projection, gradients into slices of its gradient."""
    import torch
    lq, h, hk, d = [77, 120], 4, 2, 64
    fused = rand((197, h + 2 * hk, d), dtype, 9)
    q, k, v = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
    do = rand((h, 197, d), dtype, 10).transpose(0, 1)   # heads first
    c = cu(lq)
    plain = [t.contiguous() for t in (q, k, v, do)]
    grad = torch.full_like(fused, float("nan"))
    o = torch.full((h, 197, d), float("nan"), dtype=fused.dtype, device="cuda").transpose(0, 1)
    lse = torch.empty(197, h, device="cuda")
    st.staple_attn_fwd(q, k, v, c, c, window=50, sinks=2, out={"o": o, "lse": lse})
    st.staple_attn_bwd(do, q, k, v, o, lse, c, c, window=50, sinks=2,
                       out={"dq": grad[:, :h], "dk": grad[:, h:h + hk], "dv": grad[:, h + hk:]})
    f = st.staple_attn_fwd(*plain[:3], c, c, window=50, sinks=2)
    b = st.staple_attn_bwd(plain[3], *plain[:3], f["o"], f["lse"], c, c, window=50, sinks=2)
    assert torch.equal(o, f["o"]) and torch.equal(lse, f["lse"])
    assert torch.equal(grad, torch.cat([b["dq"], b["dk"], b["dv"]], dim=1))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", [70, 3, 190])
def test_window_attention_hidden_rows_do_not_matter(st, dtype, bad, where):
    """A key with non-finite rows, and a query with a non-finite gradient: everything that
    does not see them keeps its value."""
    lq, h, hk, d, window, sinks = [200], 4, 2, 128, 20, 2
    ops = [rand((200, n, d), dtype, 20 + i) for i, n in enumerate((h, hk, hk, h))]
    ref, bound = oracle_window(dtype, ops, lq, lq, h, hk, window, sinks, d ** -0.5)
    see = A.visible(200, 200, window, sinks)
    hit_q = see[:, where]                       # queries that see the bad key
    hit_k = see[hit_q].any(axis=0)              # keys that those queries see
    q, k, v, do = (t.clone() for t in ops)
    v[where] = bad
    _, _, got = run_window(st, dtype, lq, [0], h, hk, d, window, sinks, qkv=(q, k, v, do))
    for n in ("o", "dq"):
        check(got[n][~hit_q], ref[n][~hit_q], bound[n][~hit_q], f"{n}, bad v")
    for n in ("dk", "dv"):
        check(got[n][~hit_k], ref[n][~hit_k], bound[n][~hit_k], f"{n}, bad v")
    check(got["lse"], ref["lse"], bound["lse"], "lse, bad v")
    q, k, v, do = (t.clone() for t in ops)
    k[where] = bad
    _, _, got = run_window(st, dtype, lq, [0], h, hk, d, window, sinks, qkv=(q, k, v, do))
    for n in ("o", "lse", "dq"):
        check(got[n][~hit_q], ref[n][~hit_q], bound[n][~hit_q], f"{n}, bad k")
    for n in ("dk", "dv"):
        check(got[n][~hit_k], ref[n][~hit_k], bound[n][~hit_k], f"{n}, bad k")
    q, k, v, do = (t.clone() for t in ops)
    do[where] = bad
    _, _, got = run_window(st, dtype, lq, [0], h, hk, d, window, sinks, qkv=(q, k, v, do))
    rows = np.arange(200) != where
    check(got["dq"][rows], ref["dq"][rows], bound["dq"][rows], "dq, bad do")
    keys = ~see[where]
    for n in ("dk", "dv"):
        check(got[n][keys], ref[n][keys], bound[n][keys], f"{n}, bad do")


def test_window_attention_rows_in_no_sequence_stay_out(st):
    """Rows before, between and past the sequences are neither read into results nor written."""
    import torch
    h, d = 2, 64
    q, k, v, do = (rand((100, h, d), "bf16", 30 + i) for i in range(4))
    off = ints([10, 50, 83])
    for t in (q, k, v, do):
        t[:10] = float("nan")
        t[83:] = float("nan")
    nan = lambda: torch.full((100, h, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = {"o": nan(), "lse": torch.full((100, h), 7.0, device="cuda")}
    grads = {n: nan() for n in ("dq", "dk", "dv")}
    st.staple_attn_fwd(q, k, v, off, off, window=20, sinks=1, out=out)
    st.staple_attn_bwd(do, q, k, v, out["o"], out["lse"], off, off, window=20, sinks=1, out=grads)
    for t in [out["o"], *grads.values()]:
        assert torch.isnan(t[:10]).all() and torch.isnan(t[83:]).all() and torch.isfinite(t[10:83]).all()
    assert (out["lse"][:10] == 7).all() and (out["lse"][83:] == 7).all()


def test_window_attention_offsets_past_32_bits(st):
    """Rows more than 2^32 bytes apart."""
    import torch
    n, h, d, stride = 70, 2, 64, (1 << 26) + 64
    buf = torch.empty(n * stride + h * d, dtype=torch.bfloat16, device="cuda")
    wide = buf.as_strided((n, h, d), (stride, d, 1))
    q, k, v, do = (rand((n, h, d), "bf16", 40 + i) for i in range(4))
    c = cu([n])
    f = st.staple_attn_fwd(q, k, v, c, c)
    b = st.staple_attn_bwd(do, q, k, v, f["o"], f["lse"], c, c)
    for name, x in (("q", q), ("k", k), ("v", v), ("do", do)):
        wide.copy_(x)
        ops = {"q": q, "k": k, "v": v, "do": do, name: wide}
        f2 = st.staple_attn_fwd(ops["q"], ops["k"], ops["v"], c, c)
        b2 = st.staple_attn_bwd(ops["do"], ops["q"], ops["k"], ops["v"], f2["o"], f2["lse"], c, c)
        for m in ("o", "lse"):
            assert torch.equal(f[m], f2[m]), (name, m)
        for m in ("dq", "dk", "dv"):
            assert torch.equal(b[m], b2[m]), (name, m)
    out = {m: wide if m == "dk" else torch.empty_like(t) for m, t in b.items()}
    st.staple_attn_bwd(do, q, k, v, f["o"], f["lse"], c, c, out=out)
    assert torch.equal(wide.contiguous(), b["dk"])


def test_window_attention_bad_offsets_set_the_error_word(st):
    import torch
    q = rand((40, 2, 64), "bf16", 1)
    for off in ([0, 30, 20], [0, 20, 41], [-1, 20, 40]):
        o = torch.full_like(q, 5.0)
        st.staple_attn_fwd(q, q, q, ints(off), ints(off), out={"o": o, "lse": torch.empty(40, 2, device="cuda")})
        assert st.staple_get_device_error() == -5
    f = st.staple_attn_fwd(q, q, q, cu([40]), cu([40]))
    assert st.staple_get_device_error() == 0 and torch.isfinite(f["o"]).all()


def test_window_attention_on_another_stream_and_repeated_is_identical(st):
    import torch
    ops = [rand((333, n, 128), "bf16", 60 + i) for i, n in enumerate((8, 2, 2, 8))]
    _, _, first = run_window(st, "bf16", [300, 33], [0, 0], 8, 2, 128, 90, 3, qkv=ops)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, _, again = run_window(st, "bf16", [300, 33], [0, 0], 8, 2, 128, 90, 3, qkv=ops)
    for n in first:
        assert np.array_equal(first[n], again[n]), n


# ------------------------------------------------------------------------------------------ decode
def make_cache(dtype, lens, hk, d, page, seed, width=None, spare=5, layers=None):
    """Scattered pages; every slot that no sequence uses holds NaN."""
    import torch
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in lens]
    width = width or max(1, max(held, default=1))
    pages = sum(held) + spare
    ids = rng.permutation(pages)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    shape = ((layers or 1), pages, hk, page, d)
    k, v = (rand(shape, dtype, seed + i) for i in (1, 2))
    used = np.zeros((pages, page), dtype=bool)
    at = 0
    for s, n in enumerate(lens):
        table[s, :held[s]] = ids[at:at + held[s]]
        for j in range(n):
            used[table[s, j // page], j % page] = True
        at += held[s]
    hole = torch.from_numpy(~used).cuda()[None, :, None, :, None]
    k, v = (torch.where(hole, float("nan"), t.float()).to(t.dtype) for t in (k, v))
    refs = np.zeros(pages, dtype=np.int32)
    refs[ids[:at]] = 1
    if layers is None:
        k, v = k[0], v[0]
    return k, v, torch.from_numpy(table).cuda(), ints(lens), torch.from_numpy(refs).cuda()


DECODE_CASES = [   # lens, heads, kv heads, dim, page, window, sinks
    ([1], 1, 1, 8, 16, 0, 0),
    ([37], 16, 16, 128, 16, 0, 0),
    ([0, 1, 15, 16, 17, 31, 32, 33, 0, 64, 65], 4, 2, 64, 16, 0, 0),
    ([200, 1, 129, 300], 8, 8, 128, 32, 0, 0),
    ([200, 1, 129, 300], 32, 8, 128, 64, 50, 4),
    ([77, 500], 16, 1, 128, 16, 0, 0),
    ([77, 500], 40, 1, 96, 128, 100, 3),
    ([300, 2], 3, 3, 72, 16, 1, 0),
    ([300, 2], 6, 2, 64, 256, 1, 70),
    ([90, 400], 4, 4, 40, 1024, 33, 1000),
    ([5000], 8, 2, 128, 16, 0, 0),
    ([5000, 17], 8, 2, 64, 64, 0, 0),
    ([9001, 4097, 3, 0], 4, 4, 128, 32, 3000, 100),
]


def decode_ref(dtype, q, k, v, table, lens, window, sinks, scale, rows=None):
    q, k, v, table, lens = (to_np(t) for t in (q, k, v, table, lens))
    n, h, d = q.shape
    page, hk = k.shape[2], k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros((n, h))
    bo, bl = np.zeros(q.shape), np.zeros((n, h))
    for i in range(n):
        s = i if rows is None else rows[i]
        m = int(lens[s])
        j = np.arange(m)
        ks, vs = k[table[s, j // page], :, j % page], v[table[s, j // page], :, j % page]
        see = A.visible(1, m, window, sinks) if m else np.zeros((1, 0), dtype=bool)
        for x in range(h):
            ops = q[i:i + 1, x], ks[:, x // (h // hk)].reshape(m, d), vs[:, x // (h // hk)].reshape(m, d)
            out = A.attend(*ops, see, scale)
            b = bounds(dtype, *ops, out, see, scale)
            o[i, x], lse[i, x], bo[i, x], bl[i, x] = out["o"][0], out["lse"][0], b["o"][0], b["lse"][0]
    return (o, lse), (bo, bl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", DECODE_CASES, ids=lambda c: f"n{len(c[0])}-len{max(c[0])}-h{c[1]}_{c[2]}-d{c[3]}-p{c[4]}-w{c[5]}-s{c[6]}")
def test_decode_attention(st, dtype, case):
    lens, h, hk, d, page, window, sinks = case
    print(case, dtype, flush=True)
    k, v, table, ln, _ = make_cache(dtype, lens, hk, d, page, 70)
    q = rand((len(lens), h, d), dtype, 71)
    got = st.staple_attn_decode_paged(q, k, v, table, ln, window=window, sinks=sinks, max_len=max(lens))
    (o, lse), (bo, bl) = decode_ref(dtype, q, k, v, table, ln, window, sinks, d ** -0.5)
    assert st.staple_get_device_error() == 0
    check(to_np(got["o"]), o, bo, "o")
    check(to_np(got["lse"]), lse, bl, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 40])
def test_decode_attention_writes_the_new_token(st, dtype, window):
    """With k_new, v_new: the cache and the result of an append and a plain call; rows by number."""
    import torch
    lens, h, hk, d, page = [33, 700, 1, 16, 128, 2000], 8, 4, 128, 16
    k, v, table, ln, _ = make_cache(dtype, lens, hk, d, page, 80)
    rows = ints([5, 0, 2, 3, 1])
    fused = rand((5, h + 2 * hk, d), dtype, 81)
    q, kn, vn = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
    k2, v2 = k.clone(), v.clone()
    st.staple_kv_append(kn, vn, k2, v2, table, ln, rows)
    ref = st.staple_attn_decode_paged(q, k2, v2, table, ln, seqs=rows, window=window, sinks=2)
    got = st.staple_attn_decode_paged(q, k, v, table, ln, seqs=rows, k_new=kn, v_new=vn, window=window, sinks=2)
    assert st.staple_get_device_error() == 0
    assert torch.equal(k.nan_to_num(7), k2.nan_to_num(7)) and torch.equal(v.nan_to_num(7), v2.nan_to_num(7))
    (o, lse), (bo, bl) = decode_ref(dtype, q, k2, v2, table, ln, window, 2, d ** -0.5, [5, 0, 2, 3, 1])
    for r in (ref, got):
        check(to_np(r["o"]), o, bo, "o")
        check(to_np(r["lse"]), lse, bl, "lse")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_attention_hidden_keys_do_not_matter(st, bad):
    import torch
    lens, h, hk, d, page, window, sinks = [300, 90], 8, 2, 128, 32, 45, 3
    k, v, table, ln, _ = make_cache("bf16", lens, hk, d, page, 90)
    q = rand((2, h, d), "bf16", 91)
    ref = st.staple_attn_decode_paged(q, k, v, table, ln, window=window, sinks=sinks)
    for s, n in enumerate(lens):
        for j in range(sinks, n - window):
            k[int(table[s, j // page]), :, j % page] = bad
            v[int(table[s, j // page]), :, j % page] = bad
    got = st.staple_attn_decode_paged(q, k, v, table, ln, window=window, sinks=sinks)
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["lse"], ref["lse"])


def test_decode_attention_pages_past_32_bits(st):
    """Pages whose offsets pass 2^32 bytes."""
    import torch
    hk, page, d, n = 8, 64, 128, 36000
    pools = [torch.empty((n, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens = [130, 64]
    k, v, table, ln, _ = make_cache("bf16", lens, hk, d, page, 95, spare=1)
    high = torch.where(table >= 0, n - 1 - table, table)
    for small, big in ((k, pools[0]), (v, pools[1])):
        big[n - small.shape[0]:] = small.flip(0)
    q = rand((2, 16, d), "bf16", 96)
    ref = st.staple_attn_decode_paged(q, k, v, table, ln)
    got = st.staple_attn_decode_paged(q, pools[0], pools[1], high, ln)
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["lse"], ref["lse"])
    kn, vn = rand((2, hk, d), "bf16", 97), rand((2, hk, d), "bf16", 98)
    st.staple_attn_decode_paged(q, pools[0], pools[1], high, ln, k_new=kn, v_new=vn)
    st.staple_kv_append(kn, vn, k, v, table, ln)
    for small, big in ((k, pools[0]), (v, pools[1])):
        assert torch.equal(big[n - small.shape[0]:].flip(0).nan_to_num(7), small.nan_to_num(7))


def test_decode_attention_bad_state_sets_the_error_word(st):
    import torch
    lens = [40, 40]
    k, v, table, ln, _ = make_cache("bf16", lens, 2, 64, 16, 99)
    q = rand((2, 4, 64), "bf16", 99)
    ref = st.staple_attn_decode_paged(q, k, v, table, ln)
    for broken in ("page -1", "page past the pool", "row", "length"):
        t, l, rows = table.clone(), ln.clone(), ints([0, 1])
        if broken == "page -1":
            t[1, 1] = -1
        elif broken == "page past the pool":
            t[1, 2] = k.shape[0]
        elif broken == "row":
            rows[1] = 2
        else:
            l[1] = 4000
        got = st.staple_attn_decode_paged(q, k, v, t, l, seqs=rows)
        assert st.staple_get_device_error() == -5, broken
        assert torch.equal(got["o"][0], ref["o"][0]), broken
    assert st.staple_get_device_error() == 0


def test_decode_step_in_a_graph(st):
    """extend, append and attention captured once and replayed as the sequences grow."""
    import torch
    h, hk, d, page = 8, 4, 64, 16
    lens = [30, 14, 1, 47]
    k, v, table, ln, refs = make_cache("bf16", lens, hk, d, page, 110, width=6, spare=20)
    rows = ints(range(4))
    q, kn, vn = (rand((4, n, d), "bf16", 111 + i) for i, n in enumerate((h, hk, hk)))
    state = [k, v, table, ln, refs]
    saved = [t.clone() for t in state]
    out = {"o": torch.empty_like(q), "lse": torch.empty(4, h, device="cuda")}
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        st.staple_kv_extend(refs, table, ln, rows, k_pages=k[None], v_pages=v[None], workspace=ws)
        st.staple_attn_decode_paged(q, k, v, table, ln, k_new=kn, v_new=vn, out=out, workspace=ws)

    inputs = [[rand(t.shape, "bf16", 120 + 3 * n + i) for i, t in enumerate((q, kn, vn))] for n in range(5)]
    eager = []
    for x in inputs:
        for t, y in zip((q, kn, vn), x):
            t.copy_(y)
        step()
        eager.append((out["o"].clone(), out["lse"].clone()))
    after = [t.clone() for t in state]
    for t, y in zip(state, saved):
        t.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, y in zip(state, saved):
        t.copy_(y)
    for x, want in zip(inputs, eager):
        for t, y in zip((q, kn, vn), x):
            t.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["o"], want[0]) and torch.equal(out["lse"], want[1])
    for t, y in zip(state, after):
        assert torch.equal(t.float().nan_to_num(7), y.float().nan_to_num(7))
    assert st.staple_get_device_error() == 0


# ------------------------------------------------------------------------------------------- pages
def same(c, refs, table, lens, k, v):
    assert np.array_equal(to_np(refs), c.refs) and np.array_equal(to_np(lens), c.lens)
    assert np.array_equal(to_np(table), c.table)
    for a, b in ((k, c.k), (v, c.v)):
        assert np.array_equal(np.nan_to_num(to_np(a), nan=7), np.nan_to_num(b, nan=7))


@pytest.mark.parametrize("dtype,layers,hk,d,page", [("bf16", 1, 1, 8, 16), ("bf16", 3, 2, 72, 32), ("f32", 2, 4, 64, 16)])
def test_pages_through_many_steps(st, dtype, layers, hk, d, page):
    """A random run of forks, growth, appends, ends and packing, every step against the oracle."""
    import torch
    rng = np.random.default_rng(layers)
    rows, width = 24, 9
    lens = [int(n) for n in rng.integers(1, 4 * page, 8)] + [0] * (rows - 8)
    k, v, table, ln, refs = make_cache(dtype, lens, hk, d, page, 130, width=width, spare=90, layers=layers)
    c = A.Pages(*(to_np(t) for t in (refs, table, ln, k, v)))
    for step in range(30):
        live = [s for s in range(rows) if c.lens[s] > 0]
        empty = [s for s in range(rows) if c.lens[s] == 0]
        what = ["fork", "extend", "free", "compact", "extend"][step % 5]
        print(step, what, flush=True)
        if what == "fork":
            kids = empty[:int(rng.integers(1, 6))]
            parents = [int(s) for s in rng.choice(live, len(kids))]
            c.fork(parents, kids)
            st.staple_kv_fork(refs, table, ln, ints(parents), ints(kids), page_size=page)
        elif what == "extend":
            seqs = [int(s) for s in rng.permutation(live)]
            n_new = [int(n) for n in rng.choice([0, 1, 2, page, page + 3], len(seqs))]
            n_new = [n if c.lens[s] + n <= width * page else 0 for s, n in zip(seqs, n_new)]
            assert c.extend(seqs, n_new)
            st.staple_kv_extend(refs, table, ln, ints(seqs), ints(n_new), k_pages=k, v_pages=v)
            new = [[rand((layers, sum(n_new), hk, d), dtype, 1000 * step + i)][0] for i in range(2)]
            at = np.cumsum([0] + n_new)
            for layer in range(layers):
                if sum(n_new):
                    st.staple_kv_append(new[0][layer], new[1][layer], k[layer], v[layer], table, ln, ints(seqs), cu(n_new))
                a, b = to_np(new[0][layer]), to_np(new[1][layer])
                c.append(seqs, [a[x:y] for x, y in zip(at, at[1:])], [b[x:y] for x, y in zip(at, at[1:])], layer)
        elif what == "free":
            seqs = [int(s) for s in rng.permutation(live)[:len(live) // 2]]
            c.free(seqs)
            st.staple_kv_free(refs, table, ln, ints(seqs), page_size=page)
        else:
            before = [t.clone() for t in (refs, table, k, v)]
            n = c.compact()
            if step % 2:
                out = st.staple_kv_compact(refs, table, ln, k, v)
            else:
                out = st.staple_kv_compact(refs, table, ln, k, v, out={n: torch.full_like(t, 99) for n, t in
                                                                      (("refs", refs), ("table", table))})
                # the old table still reads the same rows
                assert torch.equal(refs, before[0]) and torch.equal(table, before[1])
                held = torch.arange(width, device="cuda")[None] < -(-ln // page)[:, None]
                at = table[held].long()
                assert torch.equal(k[:, at].nan_to_num(7), before[2][:, at].nan_to_num(7))
                refs, table = out["refs"], out["table"]
            assert int(out["n_live"]) == n
        same(c, refs, table, ln, k, v)
    assert st.staple_get_device_error() == 0


@pytest.mark.parametrize("pages,n", [(20000, 700), (9000, 4096), (5, 1)])
def test_extend_and_compact_many(st, pages, n):
    """Pools and lists larger than one pass of the ranking workgroup."""
    rng = np.random.default_rng(n)
    page, width = 16, 4
    lens = np.zeros(n, dtype=np.int64)
    refs = np.zeros(pages, dtype=np.int64)
    refs[rng.permutation(pages)[:pages // 3]] = 1     # held elsewhere
    pool = np.zeros((1, pages, 1, page, 8), dtype=np.float32)
    pool[0, :, 0, :, 0] = np.arange(pages)[:, None]
    c = A.Pages(refs, -np.ones((n, width)), lens, pool, -pool)
    import torch
    tr, tt, tl = (torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in (c.refs, c.table, c.lens))
    k, v = torch.from_numpy(c.k).cuda(), torch.from_numpy(c.v).cuda()
    for n_new in (rng.integers(0, 30 if pages > 3 * n else 17, n), rng.integers(0, 2, n)):
        n_new = [int(x) for x in n_new]
        assert c.extend(range(n), n_new)
        st.staple_kv_extend(tr, tt, tl, ints(range(n)), ints(n_new), k_pages=k, v_pages=v)
        same(c, tr, tt, tl, k, v)
    gone = [int(s) for s in np.nonzero(rng.integers(0, 2, n))[0]]
    if gone:
        c.free(gone)
        st.staple_kv_free(tr, tt, tl, ints(gone), page_size=page)
    live = c.compact()
    assert int(st.staple_kv_compact(tr, tt, tl, k, v)["n_live"]) == live
    same(c, tr, tt, tl, k, v)
    assert st.staple_get_device_error() == 0


def test_extend_refuses_whole_when_pages_run_out(st):
    import torch
    lens = [16, 5, 30]
    k, v, table, ln, refs = make_cache("bf16", lens, 1, 8, 16, 140, width=3, spare=2)
    k, v = k[None], v[None]
    state = [refs, table, ln, k, v]
    before = [t.clone() for t in state]
    intact = lambda: all(torch.equal(a.float().nan_to_num(7), b.float().nan_to_num(7)) for a, b in zip(state, before))
    for n_new, why in (([17, 12, 0], "three pages of two"), ([0, 44, 0], "past the row's width"), ([1 << 30, 0, 0], "far past")):
        st.staple_kv_extend(refs, table, ln, ints(range(3)), ints(n_new), k_pages=k, v_pages=v)
        assert st.staple_get_device_error() == -8, why
        assert intact(), why
    st.staple_kv_extend(refs, table, ln, ints([0, 7, 1]), ints([0, 5, 0]), k_pages=k, v_pages=v)   # row 7
    assert st.staple_get_device_error() == -5 and intact()
    st.staple_kv_extend(refs, table, ln, ints(range(3)), ints([17, 11, 2]), k_pages=k, v_pages=v)
    assert st.staple_get_device_error() == 0 and ln.tolist() == [33, 16, 32]


def test_fork_free_and_copy_refuse_bad_rows(st):
    import torch
    lens = [16, 5, 0]
    k, v, table, ln, refs = make_cache("bf16", lens, 1, 8, 16, 150, width=3)
    before = [t.clone() for t in (refs, table, ln)]
    for parents, kids in (([0], [1]), ([0], [3]), ([-1], [2]), ([2], [2])):
        st.staple_kv_fork(refs, table, ln, ints(parents), ints(kids), page_size=16)
        assert st.staple_get_device_error() == -5, (parents, kids)
    st.staple_kv_free(refs, table, ln, ints([3, -1]), page_size=16)
    assert st.staple_get_device_error() == -5
    for a, b in zip((refs, table, ln), before):
        assert torch.equal(a, b)
    k2 = k.clone()
    st.staple_kv_copy_pages(k, v, ints([0, 99]), ints([-1, 1]))
    assert st.staple_get_device_error() == -5 and torch.equal(k.nan_to_num(7), k2.nan_to_num(7))
    st.staple_kv_copy_pages(k, v, ints([0, 2]), ints([3, 1]))
    assert torch.equal(k[[3, 1]].nan_to_num(7), k2[[0, 2]].nan_to_num(7)) and st.staple_get_device_error() == 0


def test_append_refuses_rows_that_do_not_fit(st):
    import torch
    lens = [16, 5]
    k, v, table, ln, _ = make_cache("bf16", lens, 1, 8, 16, 160)
    new = rand((20, 1, 8), "bf16", 161)
    k2 = k.clone()
    st.staple_kv_append(new[:6], new[:6], k, v, table, ln, ints([1]), cu([6]))   # six new tokens of five
    assert st.staple_get_device_error() == -5
    k2[int(table[1, 0]), :, :5] = new[1:6].transpose(0, 1)
    assert torch.equal(k.nan_to_num(7), k2.nan_to_num(7))
    st.staple_kv_append(new[:1], new[:1], k, v, table, ln, ints([2]))
    assert st.staple_get_device_error() == -5 and torch.equal(k.nan_to_num(7), k2.nan_to_num(7))
