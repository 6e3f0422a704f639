"""Embedding, norms around a block, loss and sampling on the GPU against the float64 oracle."""
import numpy as np
import pytest

import model_bounds as B
from attn_bounds import check
from helpers import to_np
from oracle import model_oracle as M
from test_gpu_attn import TORCH, ints, rand, st  # noqa: F401

pytestmark = pytest.mark.gpu


def floats(values):
    import torch
    return torch.tensor(list(values), dtype=torch.float32, device="cuda")


def strided(t, pad):
    """The same rows with `pad` more elements between them, NaN in those."""
    import torch
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def fine(st):
    import torch
    torch.cuda.synchronize()
    assert st.staple_get_device_error() == 0


# ------------------------------------------------------------------------------------- embedding
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,vocab,d,pad", [(1, 1, 1, 0), (1, 5, 2048, 0), (64, 1000, 2048, 0), (37, 9, 63, 0), (300, 50, 513, 3),
                                           (130, 77, 4096, 8), (5000, 300, 2056, 0), (4100, 11, 8, 0), (33, 4, 1111, 1)])
def test_embedding(st, dtype, out, n, vocab, d, pad):
    import torch
    print(dtype, out, n, vocab, d, pad, flush=True)
    table = rand((vocab, d), dtype, 1)
    ids = torch.from_numpy(np.random.default_rng(2).integers(0, vocab, n).astype(np.int32)).cuda()
    to = None
    if pad:
        to = strided(torch.zeros(n, d, dtype=getattr(torch, TORCH[out]), device="cuda"), pad)
    y = st.staple_embed_fwd(table, ids, scale=1.7, out_dtype=getattr(torch, TORCH[out]), out=to)
    fine(st)
    ref = M.embed(to_np(table), ids.cpu().numpy(), float(np.float32(1.7)))
    check(to_np(y), ref, B.embed(ref, out), "y")
    if pad:
        assert bool(torch.isnan(y._base[:, d:]).all())


def test_embedding_of_ids_out_of_range(st):
    table = rand((10, 24), "f32", 3)
    y = st.staple_embed_fwd(table, ints([3, -1, 10, 2 ** 31 - 1, 9]))
    assert st.staple_get_device_error() == -5 and st.staple_get_device_error() == 0
    want = table[[3, 0, 0, 0, 9]].clone()
    want[1:4] = 0
    assert bool((y == want).all())
    assert st.staple_embed_fwd(table, ints([])).shape == (0, 24)
    fine(st)


def id_patterns():
    rng = np.random.default_rng(7)
    zipf = np.minimum(rng.zipf(1.3, 3000), 400) - 1
    return {"one": [4], "same": [3] * 1000, "distinct": rng.permutation(700), "zipf": zipf, "two": [5] * 32 + [1] * 32,
            "borders": np.repeat(np.arange(6), [31, 33, 32, 64, 65, 1]), "31": np.arange(31) % 7, "33": np.arange(33) % 2,
            "64": [0] * 63 + [1], "long": rng.permutation(np.repeat([9, 2, 300], [5000, 1, 40]))}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pattern", list(id_patterns()))
@pytest.mark.parametrize("d,pad", [(8, 0), (512, 0), (1111, 0), (200, 8), (2048, 0), (70, 3)])
def test_embedding_gradient(st, dtype, pattern, d, pad):
    import torch
    print(dtype, pattern, d, pad, flush=True)
    ids = np.asarray(id_patterns()[pattern]).astype(np.int32)
    n, vocab, scale = len(ids), 701, 0.375
    dy = rand((n, d), dtype, 8)
    if pad:
        dy = strided(dy, pad)
    dd = st.staple_dedup(torch.from_numpy(ids).cuda(), vocab)
    maps = dict(inv=dd["inv"], scale=scale)
    three = (dd["sorted_pos"], dd["seg_start"], dd["n_unique"])
    rows = st.staple_embed_bwd(dy, *three, out=torch.full((n, d), float("nan"), device="cuda"), **maps)
    fine(st)
    host = to_np(dy)
    ref, bound = M.embed_grad(host, ids, scale), B.embed_grad(host, ids, scale)
    uniq = sorted(ref)
    u = len(uniq)
    check(to_np(rows[:u]), np.array([ref[t] for t in uniq]), np.array([bound[t] for t in uniq]), "rows")
    assert bool(torch.isnan(rows[u:]).all())
    # the whole table's gradient: the same sums in other places, other rows left as they were
    table = st.staple_embed_bwd(dy, *three, uniq=dd["uniq"], out=torch.full((vocab, d), 7.0, device="cuda"), **maps)
    want = torch.full((vocab, d), 7.0, device="cuda")
    want[torch.tensor(uniq, device="cuda").long()] = rows[:u]
    assert torch.equal(table, want)
    # added to
    more = st.staple_embed_bwd(dy, *three, uniq=dd["uniq"], accumulate=True, out=torch.full((vocab, d), 7.0, device="cuda"), **maps)
    want = torch.full((vocab, d), 7.0, device="cuda")
    want[torch.tensor(uniq, device="cuda").long()] += rows[:u]
    # scale and sum in one rounding or in two
    assert float((more - want).abs().max()) <= 2 * B.E * float(want.abs().max() + rows[:u].abs().max())
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [2048, 2047])
def test_embedding_gradient_of_many_tokens(st, dtype, d):
    """A training batch: wide chunks, tokens that hold thousands of positions."""
    import torch
    n, vocab = 33100, 3000
    ids = np.minimum(np.random.default_rng(12).zipf(1.2, n), vocab).astype(np.int32) - 1
    dy = rand((n, d), dtype, 13)
    dd = st.staple_dedup(torch.from_numpy(ids).cuda(), vocab)
    rows = st.staple_embed_bwd(dy, dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], scale=2.0, max_unique=vocab)
    fine(st)
    host = to_np(dy[:, ::73])
    ref, bound = M.embed_grad(host, ids, 2.0), B.embed_grad(host, ids, 2.0)
    uniq = sorted(ref)
    check(to_np(rows[:len(uniq)][:, ::73]), np.array([ref[t] for t in uniq]), np.array([bound[t] for t in uniq]), "rows")
    # every column against a sum in another order
    total = torch.zeros(vocab, d, dtype=torch.float64, device="cuda").index_add_(0, torch.from_numpy(ids).cuda().long(), dy.double())
    size = torch.zeros(vocab, d, dtype=torch.float64, device="cuda").index_add_(0, torch.from_numpy(ids).cuda().long(), dy.double().abs())
    at = torch.tensor(uniq, device="cuda")
    most = 2 * B.E * size[at] * (34 + torch.bincount(torch.from_numpy(ids).cuda().long(), minlength=vocab)[at, None])
    assert bool(((rows[:len(uniq)].double() - 2 * total[at]).abs() <= most).all())


def test_embedding_gradient_of_one_row_for_all(st):
    """A gradient that is the same for all positions, given by one row."""
    import torch
    ids = ints([1, 1, 0, 1])
    dd = st.staple_dedup(ids, 2)
    dy = rand((1, 24), "bf16", 9)
    got = st.staple_embed_bwd(dy.expand(4, 24), dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], max_unique=2)
    assert torch.equal(got, dy.float() * torch.tensor([[1.0], [3.0]], device="cuda"))
    fine(st)


def test_embedding_gradient_with_bad_maps(st):
    """Nothing out of range is read or written, and the error word says so."""
    import torch
    ids = np.repeat(np.arange(5), 20).astype(np.int32)
    n, d = len(ids), 72
    dy = rand((n, d), "f32", 10)
    dd = st.staple_dedup(torch.from_numpy(ids).cuda(), 5)
    arrays = {k: dd[k].clone() for k in ("sorted_pos", "inv", "seg_start", "n_unique", "uniq")}

    def call(max_unique=5, **change):
        a = {k: v.clone() for k, v in arrays.items()}
        for k, (at, value) in change.items():
            a[k][at] = value
        big = torch.full((7, d), 7.0, device="cuda")
        st.staple_embed_bwd(dy, a["sorted_pos"], a["seg_start"], a["n_unique"], inv=a["inv"], max_unique=max_unique,
                            out=big[1:6])
        assert bool((big[0] == 7).all()) and bool((big[6] == 7).all())
        return st.staple_get_device_error(), big[1:6]

    assert call()[0] == 0
    status, grad = call(max_unique=4)
    assert status == -5 and bool((grad == 7).all())
    for bad in (-1, n, 2 ** 31 - 1, -2 ** 31):
        assert call(sorted_pos=(30, bad))[0] == -5
    for bad in (-1, 5, 2 ** 31 - 1):
        assert call(inv=(int(arrays["sorted_pos"][30]), bad))[0] == -5
    for bad in (-1, 5, 2 ** 31 - 1):
        a = arrays["uniq"].clone()
        a[2] = bad
        big = torch.full((7, d), 7.0, device="cuda")
        st.staple_embed_bwd(dy, arrays["sorted_pos"], arrays["seg_start"], arrays["n_unique"], inv=arrays["inv"], uniq=a,
                            max_unique=5, out=big[1:6])
        assert st.staple_get_device_error() == -5
        assert bool((big[0] == 7).all()) and bool((big[6] == 7).all()) and bool((big[3] == 7).all())
    assert call(seg_start=(2, 2 ** 31 - 1))[0] == -5
    assert call(seg_start=(2, -5))[0] in (0, -5)


@pytest.mark.parametrize("each", [20, 90])
def test_embedding_gradient_with_bad_segments(st, each):
    """Every entry of seg_start that is out of range, or that its neighbours' positions contradict, sets the error
    word; tokens within a workgroup's positions and across them."""
    import torch
    tokens, d = 5, 72
    ids = torch.from_numpy(np.repeat(np.arange(tokens), each).astype(np.int32)).cuda()
    n = len(ids)
    dy = rand((n, d), "f32", 11)
    dd = st.staple_dedup(ids, tokens)
    right = each * np.arange(tokens + 1)

    def call(at, value):
        seg = dd["seg_start"].clone()
        seg[at] = value
        big = torch.full((tokens + 2, d), 7.0, device="cuda")
        st.staple_embed_bwd(dy, dd["sorted_pos"], seg, dd["n_unique"], inv=dd["inv"], max_unique=tokens, out=big[1:-1])
        assert bool((big[0] == 7).all()) and bool((big[-1] == 7).all())
        return st.staple_get_device_error()

    for at in range(tokens + 1):
        print(each, at, flush=True)
        assert call(at, int(right[at])) == 0
        for bad in (-5, -1, right[at] - 1, right[at] + 1, n + 1, 2 ** 31 - 1, -2 ** 31):
            assert call(at, int(bad)) == -5, (at, bad)


# ----------------------------------------------------------------------------------------- norms
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "f32"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16")]
DIMS = [(5, 1), (3, 7), (9, 8), (4, 64), (7, 512), (6, 520), (5, 1000), (5, 1111), (4, 2048), (3, 2056), (3, 4096), (2, 5001),
        (2, 8192), (2, 16384), (700, 264), (1, 2048), (1500, 33), (37, 65), (50, 128), (21, 129), (11, 255),
        (3, 4097), (2, 8191), (2, 8200), (2, 12291), (2, 16383),
        # more rows than there are places for them at once
        (9000, 40), (4000, 300), (3000, 1000), (1500, 2048), (1300, 4096), (600, 5001), (530, 16384),
        (20000, 64), (9000, 127), (1100, 2047), (300, 8193)]


def run_norm(st, n, d, dtype, r_dtype, w_dtype, pre, post, gate, residual, scale, pad, seed, x=None):
    how = dict(pre=pre, post=post, scale=scale, eps=1e-6)
    ops = {"x": rand((n, d), r_dtype, seed, 2.0) if x is None else x, "z": rand((n, d), dtype, seed + 1, 0.7)}
    w = lambda i: (1 + rand((d,), "f32", seed + i, 0.2)).to(rand((1,), w_dtype, 0).dtype)
    if pre:
        how["w_pre"] = w(2)
    if post:
        how["w_post"] = w(3)
    if gate:
        how["gate"] = w(4) if gate == "vector" else rand((n, d), dtype, seed + 4)
    grads = {"dr": rand((n, d), r_dtype, seed + 5), "dh": rand((n, d), dtype, seed + 6) if pre else None}
    if pad:
        ops = {k: strided(t, pad) for k, t in ops.items()}
        grads = {k: t if t is None else strided(t, pad) for k, t in grads.items()}
    if not residual:
        ops["x"] = None
    f = st.staple_norm_fwd(ops["x"], ops["z"], save=True, **how)
    both = [st.staple_norm_bwd(grads["dr"], grads["dh"], ops["x"], ops["z"], f["rstd_r"], f["rstd_z"], r=r, **how)
            for r in (None, f["r"])]
    fine(st)
    return ops, grads, how, f, both


def check_norm(ops, grads, how, f, both, dtype, r_dtype):
    """The gradients from r formed again, and from the stored one."""
    h = {k: to_np(v) if hasattr(v, "dtype") else v for k, v in how.items()}
    h["scale"] = float(np.float32(h["scale"]))
    h["eps"] = float(np.float32(h["eps"]))
    o = {k: None if t is None else to_np(t) for k, t in ops.items()}
    r_dtype = dtype if ops["x"] is None else r_dtype
    ref = M.norm(o["x"], o["z"], **h)
    bound = B.norm(ref, o["x"], o["z"], dtype, r_dtype, **h)
    for k in ("r", "h", "rstd_r", "rstd_z"):
        assert (f[k] is None) == (ref[k] is None)
        if f[k] is not None:
            check(to_np(f[k]), ref[k], bound[k], k)
    g = {k: None if t is None else to_np(t) for k, t in grads.items()}
    saved = [None if f[k] is None else to_np(f[k]) for k in ("rstd_r", "rstd_z")]
    del h["eps"]
    for b, r, e_r in ((both[0], ref["r"], bound["sum"]), (both[1], to_np(f["r"]), 0.0)):
        want = M.norm_grad(g["dr"], g["dh"], r, o["z"], *saved, **h)
        most = B.norm_grad(want, g["dr"], g["dh"], r, o["z"], *saved, dtype, r_dtype, e_r=e_r, **h)
        if "gate" in h and h["gate"].ndim == 1:
            want["dgate"], most["dgate"] = want["dgate"].sum(axis=0), most["dgate_sum"]
        for k, t in b.items():
            if t is not None:
                check(to_np(t), want[k], most[k], k)
        assert (b["dx"] is None) == (ops["x"] is None) and b["dz"] is not None


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("n,d", DIMS)
def test_norms_and_their_gradients(st, types, n, d):
    dtype, r_dtype, w_dtype = types
    print(types, n, d, flush=True)
    made = run_norm(st, n, d, *types, True, True, "vector", True, 0.75, 0, 20)
    check_norm(*made, dtype, r_dtype)


@pytest.mark.parametrize("types", TYPES[1:4], ids="-".join)
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "vector", "rows"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_combinations(st, types, pre, post, gate, residual):
    dtype, r_dtype, w_dtype = types
    if not residual:
        types = (dtype, dtype, w_dtype)   # r has the block's type then
    for n, d, pad in ((6, 136, 0), (3, 90, 1), (2, 2048, 8)):
        print(types, pre, post, gate, residual, n, d, pad, flush=True)
        made = run_norm(st, n, d, *types, pre, post, gate, residual, -1.25, pad, 30)
        check_norm(*made, dtype, types[1])


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,d", [(1, 64), (9, 2048), (5, 333)])
def test_a_norm_alone(st, dtype, out, n, d):
    """Without a block: r is x; its gradient with and without one from elsewhere."""
    import torch
    x, w = rand((n, d), dtype, 40, 3.0), 1 + rand((d,), "f32", 41, 0.2)
    f = st.staple_norm_fwd(x, w_pre=w, dtype=getattr(torch, TORCH[out]), save=True)
    assert f["r"] is None and f["rstd_z"] is None
    dh, dr = rand((n, d), out, 42), rand((n, d), dtype, 43)
    for more in (None, dr):
        b = st.staple_norm_bwd(more, dh, x, None, f["rstd_r"], w_pre=w)
        fine(st)
        assert b["dz"] is None and b["dgate"] is None and b["dw_post"] is None
        xs, ws, dhs, drs = to_np(x), to_np(w), to_np(dh), None if more is None else to_np(more)
        ref = M.norm(xs, None, w_pre=ws, eps=float(np.float32(1e-6)))
        bound = B.norm(ref, xs, None, out, dtype, w_pre=ws)
        check(to_np(f["h"]), ref["h"], bound["h"], "h")
        r = to_np(f["rstd_r"])
        ref = M.norm_grad(drs, dhs, xs, None, r, None, w_pre=ws)
        bound = B.norm_grad(ref, drs, dhs, xs, None, r, None, out, dtype, w_pre=ws)
        for k in ("dx", "dw_pre"):
            check(to_np(b[k]), ref[k], bound[k], k)


@pytest.fixture
def two_passes(monkeypatch):
    """Chains of sums where the backward reads rows twice: a lane adds up to 32 terms (16384 columns in 512 lanes), a wave's
    lanes join in 6 steps, 8 waves in turn, and the second mean is two sums' difference, each of whose terms has 6
    roundings: 52 and the 6 that the bounds add to CHAIN."""
    monkeypatch.setattr(B, "CHAIN", 52)


@pytest.mark.parametrize("types", TYPES[1:4], ids="-".join)
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "vector", "rows"])
@pytest.mark.parametrize("residual", [True, False])
def test_wide_norm_combinations(st, two_passes, types, pre, post, gate, residual):
    """Widths whose backward takes two passes: past 4096 with r in fp32, past 8192 in bf16."""
    dtype, r_dtype, w_dtype = types
    if not residual:
        types = (dtype, dtype, w_dtype)
    for n, d, pad in ((3, 4104, 0), (2, 8201, 1), (5, 8208, 8), (2, 16384, 0)):
        print(types, pre, post, gate, residual, n, d, pad, flush=True)
        made = run_norm(st, n, d, *types, pre, post, gate, residual, -1.25, pad, 35)
        check_norm(*made, dtype, types[1])


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,d", [(3, 4104), (2, 8201), (5, 16384)])
def test_a_wide_norm_alone(st, two_passes, dtype, out, n, d):
    test_a_norm_alone(st, dtype, out, n, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(300, 264), (5, 8201), (300, 8208)])
@pytest.mark.parametrize("residual", [True, False])
def test_gates_gradients_in_place(st, dtype, n, d, residual):
    """A gate a row, whose gradient takes its place, and the others' theirs."""
    import torch
    x, z, gate, dr, dh = (rand((n, d), dtype, 57 + i) for i in range(5))
    x = x if residual else None
    w = 1 + rand((d,), "f32", 62, 0.2)
    how = dict(w_pre=w, w_post=w, post=True, scale=0.5)
    f = st.staple_norm_fwd(x, z, gate=gate, save=True, **how)
    want = st.staple_norm_bwd(dr, dh, x, z, f["rstd_r"], f["rstd_z"], gate=gate, **how)
    out = {"dz": z, "dgate": gate, **({"dx": x} if residual else {})}
    got = st.staple_norm_bwd(dr, dh, x, z, f["rstd_r"], f["rstd_z"], gate=gate, out=out, **how)
    fine(st)
    for k, t in got.items():
        assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,d", [(3, 7), (9, 63), (20, 264), (3, 2048), (2, 4104), (2, 8201), (2, 8208)])
def test_gradients_that_need_nothing_of_a_block(st, dtype, r_dtype, n, d):
    """A norm after the block whose gradients nobody asks for: z and its 1 / rms are not read, and need not be given."""
    import torch
    print(dtype, r_dtype, n, d, flush=True)
    x, z = rand((n, d), r_dtype, 46, 2.0), rand((n, d), dtype, 47)
    dr, dh = rand((n, d), r_dtype, 48), rand((n, d), dtype, 49)
    w = 1 + rand((d,), "f32", 56, 0.2)
    how = dict(w_pre=w, post=True, scale=0.5)
    f = st.staple_norm_fwd(x, z, save=True, **how)
    room = lambda: {"dx": torch.full_like(x, 7.0), "dw_pre": torch.full((d,), 7.0, device="cuda")}
    want = st.staple_norm_bwd(dr, dh, x, z, f["rstd_r"], f["rstd_z"], r=f["r"], out=room(), **how)
    for block in (z, None):   # without z the sum takes x's place
        got = st.staple_norm_bwd(dr, dh, x if block is not None else f["r"], block, f["rstd_r"], r=f["r"], out=room(), **how)
        fine(st)
        for k, t in want.items():
            assert torch.equal(got[k], t), k
    # without the norm before the next block the sum's gradient is the residual stream's
    got = st.staple_norm_bwd(dr, None, x, z, out={"dx": torch.empty_like(x)}, pre=False, post=True)
    fine(st)
    assert torch.equal(got["dx"], dr)


def test_norms_without_weights_and_of_extreme_rows(st):
    import torch
    x = torch.zeros(4, 128, device="cuda")
    x[1] = 1e15
    x[2, 5] = 1e-30
    x[3] = torch.arange(128, device="cuda") - 64.0
    f = st.staple_norm_fwd(x, save=True)
    h = to_np(f["h"])
    assert not h[0].any() and np.allclose(h[1], 1.0, rtol=1e-5) and abs(h[2, 5] - 1e-27) < 1e-32
    b = st.staple_norm_bwd(None, torch.ones_like(x), x, None, f["rstd_r"], out={"dx": torch.empty_like(x)})
    assert bool(torch.isfinite(b["dx"]).all())
    assert st.staple_norm_fwd(x[:0], x[:0])["r"].shape == (0, 128)
    empty = st.staple_norm_bwd(x[:0], x[:0], x[:0], None, f["rstd_r"][:0], w_pre=torch.ones(128, device="cuda"))
    assert not bool(empty["dw_pre"].any())   # a sum of no rows
    fine(st)


def test_nan_and_infinity_stay_in_their_row(st):
    x, z = rand((6, 264), "bf16", 44), rand((6, 264), "bf16", 45)
    want = st.staple_norm_fwd(x, z, post=True)
    x[2, 7], z[4, 0] = float("nan"), float("inf")
    got = st.staple_norm_fwd(x, z, post=True)
    import torch
    for k in ("r", "h"):
        rows = [0, 1, 3, 5]
        assert torch.equal(got[k][rows], want[k][rows])
        assert bool(torch.isnan(got[k][2]).any()) and bool(torch.isnan(got[k][4]).any())


@pytest.mark.parametrize("n,d", [(70, 1024), (333, 63), (90, 1111), (600, 2047), (40, 8191), (33, 16384), (31, 16383)])
def test_norms_in_place(st, n, d):
    """Outputs that take the place of inputs of their type."""
    import torch
    x, z, dr, dh = (rand((n, d), "bf16", 50 + i) for i in range(4))
    w = 1 + rand((d,), "f32", 55, 0.2)
    how = dict(w_pre=w, w_post=w, post=True, scale=0.5)
    f = st.staple_norm_fwd(x, z, save=True, **how)
    b = st.staple_norm_bwd(dr, dh, x, z, f["rstd_r"], f["rstd_z"], **how)
    x2, z2 = x.clone(), z.clone()
    g = st.staple_norm_fwd(x2, z2, out={"r": x2, "h": z2}, **how)
    assert torch.equal(g["r"], f["r"]) and torch.equal(g["h"], f["h"]) and g["r"] is x2
    dr2, dh2 = dr.clone(), dh.clone()
    c = st.staple_norm_bwd(dr2, dh2, x, z, f["rstd_r"], f["rstd_z"], out={"dx": dr2, "dz": dh2}, **how)
    assert torch.equal(c["dx"], b["dx"]) and torch.equal(c["dz"], b["dz"])
    x3, z3 = x.clone(), z.clone()
    c = st.staple_norm_bwd(dr, dh, x3, z3, f["rstd_r"], f["rstd_z"], out={"dx": x3, "dz": z3}, **how)
    assert torch.equal(c["dx"], b["dx"]) and torch.equal(c["dz"], b["dz"])
    fine(st)


# ------------------------------------------------------------------------------------------ loss
def run_xent(st, logits, targets, g, dtype, chain):
    import torch
    n, v = logits.shape
    t, gd = ints(targets), floats(g)
    one = st.staple_xent_fwd(logits, t)
    both = st.staple_xent_fwd(logits, t, g=gd)
    later = st.staple_xent_bwd(gd, logits, t, one["lse"])
    torch.cuda.synchronize()
    for k in ("loss", "lse"):
        assert torch.equal(one[k].view(torch.int32), both[k].view(torch.int32))
    host, g = to_np(logits), np.asarray(g, dtype=np.float32).astype(np.float64)
    ref = M.xent(host, targets, g)
    bound = B.xent(ref, host, np.asarray(targets), g, dtype, chain)
    for k in ("loss", "lse", "d_logits"):
        check(to_np(both[k]), ref[k], bound[k], k)
    bound = B.xent(ref, host, np.asarray(targets), g, dtype, chain, from_lse=True)
    check(to_np(later), ref["d_logits"], bound["d_logits"], "d_logits from lse")
    return both


# terms that one lane adds, the steps of joining, and a change of reference for each of them
XENT_CHAIN = lambda v: 3 * (v / 64 + 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,pad", [(1, 1, 0), (3, 2, 0), (5, 7, 0), (4, 8, 8), (70, 63, 1), (9, 513, 0), (130, 1024, 0), (33, 4096, 0),
                                     (6, 5003, 5), (2, 100352, 0), (3, 100277, 0), (1, 262147, 0), (300, 2050, 0),
                                     (3, 9001, 0), (3, 20000, 0), (3, 60001, 1), (2, 120001, 0), (2, 131072, 0), (2, 131073, 0)])
def test_loss_and_its_gradient(st, dtype, n, v, pad):
    print(dtype, n, v, pad, flush=True)
    rng = np.random.default_rng(v)
    logits = rand((n, v), dtype, 60, 4.0)
    if pad:
        logits = strided(logits, pad)
    targets = np.where(rng.random(n) < 0.2, -100, rng.integers(0, v, n))
    run_xent(st, logits, targets, rng.normal(size=n), dtype, XENT_CHAIN(v))
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [5, 700, 5001, 100352, 200003])
def test_loss_with_ruled_out_classes(st, dtype, v):
    """-inf in some classes, in the target's, in all; large offsets; the type's lowest value."""
    import torch
    n = 8
    logits = rand((n, v), dtype, 61, 2.0)
    inf = float("inf")
    logits[0, ::2] = -inf
    logits[1] = -inf
    logits[2, 3] = -inf
    logits[3, 1:] = -inf
    logits[4] += 30000.0 if dtype == "f32" else 256.0
    logits[5] = torch.finfo(logits.dtype).min
    logits[6, :4] = torch.finfo(logits.dtype).min
    logits[7] = -5.0
    run_xent(st, logits, [1, 0, 3, 0, 2, 4, 1, 4], np.linspace(-1, 2, n), dtype, XENT_CHAIN(v))
    fine(st)


def test_loss_of_nan_and_infinity_and_bad_targets(st):
    import torch
    v = 600
    logits = rand((6, v), "f32", 62)
    logits[1, 5], logits[2, 7] = float("nan"), float("inf")
    g = floats([1.0] * 6)
    want = st.staple_xent_fwd(logits, ints([3] * 6), g=g)
    assert bool(torch.isnan(want["loss"][1])) and bool(torch.isnan(want["d_logits"][1]).any())
    assert float(want["lse"][2]) == float("inf") and float(want["loss"][2]) == float("inf")
    assert bool(torch.isfinite(want["d_logits"][[0, 3, 4, 5]]).all())
    fine(st)
    got = st.staple_xent_fwd(logits, ints([3, 3, 3, v, 2 ** 31 - 1, -1]), g=g)
    assert st.staple_get_device_error() == -5
    assert not bool(got["d_logits"][3:].any()) and not bool(got["loss"][3:].any())
    assert torch.equal(got["lse"][3:], want["lse"][3:]) and torch.equal(got["d_logits"][0], want["d_logits"][0])
    later = st.staple_xent_bwd(g, logits, ints([3, 3, 3, v, 3, -1]), got["lse"])
    assert st.staple_get_device_error() == -5 and not bool(later[3].any()) and not bool(later[5].any())
    assert st.staple_xent_fwd(logits[:0], ints([]))["loss"].shape == (0,)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(40, 333), (5, 5001), (2, 100352), (300, 4097), (2, 151936), (3, 260001)])
def test_loss_in_place_and_to_strided_rows(st, dtype, n, v):
    import torch
    logits, t, g = rand((n, v), dtype, 63, 3.0), ints(np.arange(n) % v), floats(np.linspace(0, 1, n))
    want = st.staple_xent_fwd(logits, t, g=g)
    room = strided(torch.zeros_like(logits), 7)
    got = st.staple_xent_fwd(logits, t, g=g, out={"loss": torch.empty_like(want["loss"]), "lse": torch.empty_like(want["lse"]),
                                                  "d_logits": room})
    assert torch.equal(got["d_logits"], want["d_logits"]) and bool(torch.isnan(room._base[:, v:]).all())
    later = st.staple_xent_bwd(g, logits, t, want["lse"])
    mine, again = logits.clone(), logits.clone()
    got = st.staple_xent_fwd(mine, t, g=g, out={"loss": got["loss"], "lse": got["lse"], "d_logits": mine})
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(st.staple_xent_bwd(g, again, t, want["lse"], out=again), later)
    fine(st)


# -------------------------------------------------------------------------------------- sampling
def run_sample(st, logits, u, **limits):
    import torch
    given = {k: None if v is None else (ints if k == "top_k" else floats)(v) for k, v in limits.items()}
    uu = floats(u)
    got = st.staple_sample(logits, uu, **given)
    fine(st)
    host = {k: None if v is None else v.cpu().numpy() for k, v in given.items()}
    token, logprob = M.sample(to_np(logits), uu.cpu().numpy(), **host)
    assert got["token"].cpu().numpy().tolist() == token.tolist()
    # rounded once from 64 bits; sums of rounded weights are off by far less
    check(to_np(got["logprob"]), logprob, B.E * np.where(np.isfinite(logprob), np.abs(logprob), 0.0) + 1e-7 * 2.0 ** -3, "logprob")
    again = st.staple_sample(logits, uu, **given)
    assert torch.equal(again["token"], got["token"]) and torch.equal(again["logprob"], got["logprob"])
    return got


LIMITS = ["", "k", "p", "m", "kp", "km", "pm", "kpm"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("limits", LIMITS)
@pytest.mark.parametrize("n,v,pad", [(3, 1, 0), (9, 2, 0), (40, 7, 1), (20, 64, 0), (12, 1025, 0), (9, 5003, 5)])
def test_sampling(st, dtype, limits, n, v, pad):
    print(dtype, limits, n, v, pad, flush=True)
    rng = np.random.default_rng(v + len(limits))
    logits = rand((n, v), dtype, 70 + v, 3.0)
    if pad:
        logits = strided(logits, pad)
    run_sample(st, logits, rng.random(n), temperature=np.where(rng.random(n) < 0.1, 0.0, 0.2 + 2 * rng.random(n)),
               top_k=rng.integers(0, min(v, 60) + 2, n) if "k" in limits else None,
               top_p=np.where(rng.random(n) < 0.2, 1.0, rng.random(n)) if "p" in limits else None,
               min_p=np.where(rng.random(n) < 0.3, 0.0, 0.3 * rng.random(n)) if "m" in limits else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(1, 100352), (5, 100277), (2, 262147), (70, 20001)])
def test_sampling_of_whole_vocabularies(st, dtype, n, v):
    print(dtype, n, v, flush=True)
    rng = np.random.default_rng(n)
    logits = rand((n, v), dtype, 71, 2.5)
    u = rng.random(n)
    run_sample(st, logits, u)
    run_sample(st, logits, u, temperature=np.full(n, 0.8), top_k=np.full(n, 50), top_p=np.full(n, 0.95), min_p=np.full(n, 0.02))
    run_sample(st, logits, u, temperature=np.full(n, 1.3), top_p=np.full(n, 0.9))
    run_sample(st, logits, u, top_k=np.full(n, v // 2), temperature=np.full(n, 100.0), top_p=np.full(n, 0.7))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [6, 3000, 9000, 50021])
def test_sampling_of_equal_and_ruled_out_logits(st, dtype, v):
    """Ties at every border, rows without a token, infinities and NaN, the type's lowest value."""
    import torch
    n = 12
    inf, nan = float("inf"), float("nan")
    logits = rand((n, v), dtype, 72, 2.0)
    logits[0] = 1.5
    logits[1] = -inf
    logits[2, ::2] = nan
    logits[3, 1:5] = inf
    logits[4] = torch.finfo(logits.dtype).min
    logits[5, : v - 1] = -inf
    logits[6] = torch.where(torch.arange(v, device="cuda") % 3 == 0, 2.0, -1.0)
    logits[7, 1:] = torch.finfo(logits.dtype).min
    logits[8] = nan
    logits[9] = (torch.arange(v, device="cuda") % 2) * 0.25
    logits[10] = -0.0
    logits[10, ::3] = 0.0
    logits[11, 0] = torch.finfo(logits.dtype).max
    for i, r in enumerate((0.0, 0.25, 0.5, 0.999, 1.0 - 2.0 ** -24)):
        run_sample(st, logits, [r] * n)
        run_sample(st, logits, [r] * n, top_p=[0.5] * n)
        run_sample(st, logits, [r] * n, top_k=[max(1, v // 4)] * n, top_p=[0.25] * n)
        run_sample(st, logits, [r] * n, top_k=[1 + i] * n, min_p=[1.0] * n, temperature=[1e-30] * n)
        run_sample(st, logits, [r] * n, temperature=[float("inf")] * n, top_k=[3] * n)


def by_sorting(l, u, t, k, p, low):
    """One row's token, for rows that the oracle's loops take long for (no ties at a border)."""
    order = np.argsort(-l, kind="stable")
    w = np.exp((l[order] - l[order[0]]) / t)
    count = k if 0 < k < len(l) else len(l)
    if p < 1:
        sums = np.cumsum(w[:count])
        count = 1 + int(np.searchsorted(sums, p * sums[-1]))
    at = np.sort(order[:count][w[:count] >= low])
    sums = np.cumsum(np.exp((l[at] - l.max()) / t))
    return int(at[np.searchsorted(sums, u * sums[-1], side="right")])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(2, 1048577), (3, 2000003), (2, 1 << 22), (260, 30011)])
def test_sampling_of_the_longest_rows(st, dtype, n, v):
    print(dtype, n, v, flush=True)
    logits = rand((n, v), dtype, 74, 3.0)
    host = to_np(logits)
    rng = np.random.default_rng(v)
    f = lambda a: a.astype(np.float32).astype(np.float64)
    u, t, p, low = f(rng.random(n)), f(0.5 + rng.random(n)), f(0.5 + 0.6 * rng.random(n)), f(0.01 * rng.random(n))
    k = np.where(rng.random(n) < 0.5, 0, rng.integers(1, v, n))
    none = np.zeros(n)
    for kk, pp, ll in ((none, none + 1, none), (none, none + 1, low), (k, none + 1, none), (none, p, none), (k, p, low)):
        limits = {}
        if kk is not none:
            limits["top_k"] = ints(kk)
        if (pp < 1).any():
            limits["top_p"] = floats(pp)
        if ll is not none:
            limits["min_p"] = floats(ll)
        got = st.staple_sample(logits, floats(u), temperature=floats(t), **limits)["token"].cpu().numpy()
        rows = range(n) if n < 10 else range(0, n, 37)
        assert [int(got[i]) for i in rows] == [by_sorting(host[i], u[i], t[i], int(kk[i]), pp[i], ll[i]) for i in rows]
    fine(st)


def test_sampling_with_arguments_at_their_ends(st):
    nan, inf = float("nan"), float("inf")
    logits = rand((12, 500), "f32", 73, 2.0)
    ends = [nan, -inf, inf, -1.0, 0.0, 1e-45, 1.0, 2.0, 0.5, -0.0, 3e38, 0.25]
    run_sample(st, logits, [nan, -1.0, inf, 1.0, 2.0, -inf, 0.0, 1e-45, 0.5, -0.0, 0.75, 0.25])
    run_sample(st, logits, [0.7] * 12, temperature=ends)
    run_sample(st, logits, [0.7] * 12, top_p=ends)
    run_sample(st, logits, [0.7] * 12, min_p=ends)
    run_sample(st, logits, [0.7] * 12, top_k=[-2 ** 31, -1, 0, 1, 499, 500, 501, 2 ** 31 - 1, 2, 3, 4, 5])
    assert st.staple_sample(logits[:0], floats([]))["token"].shape == (0,)


def next_to_a_border(kind):
    """Rows of two logits, (-x, 0) at temperature T, and a u, p or min_p that is between 1.5 and 64 times as far from a
    border as the weights' errors reach (the distance, formed in 64 bits, is off by less than the half).  Token 0, of
    weight a = exp(-x / T), is drawn where u < a / (1 + a), kept where p > 1 / (1 + a), kept where min_p <= a.  A weight
    is off by 2^-47 of itself and a unit of 2^-50, the largest one by nothing."""
    from decimal import Decimal, localcontext
    rng = np.random.default_rng(80)
    f32 = lambda a: a.astype(np.float32).astype(np.float64)
    n = 1 << 20
    value = f32(rng.uniform(0.05, 0.45, n) if kind == "u" else rng.uniform(0.55, 0.95, n) if kind == "top_p" else rng.uniform(0.05, 0.95, n))
    t = f32(rng.uniform(0.3, 2.0, n))
    a = {"u": value / (1 - value), "top_p": 1 / value - 1, "min_p": value}[kind]
    x = f32(-t * np.log(a))
    a = np.exp(-x / t)
    error = 2.0 ** -47 * a + 2.0 ** -50
    far = np.abs({"u": a - value * (1 + a), "top_p": value * (1 + a) - 1, "min_p": a - value}[kind])   # a's factor here is 1 at most
    at = np.nonzero((far > 1.5 * error) & (far < 64 * error))[0][:400]
    first = []
    with localcontext() as c:
        c.prec = 40
        for i in at:
            w, v = (Decimal(-x[i]) / Decimal(t[i])).exp(), Decimal(value[i])
            first.append({"u": v * (1 + w) < w, "top_p": v * (1 + w) > 1, "min_p": v <= w}[kind])
    return x[at], t[at], value[at], np.array(first)


@pytest.mark.parametrize("kind", ["u", "top_p", "min_p"])
def test_sampling_next_to_a_border(st, kind):
    """The definition's token, as near to a border as the weights' errors allow."""
    import torch
    x, t, value, first = next_to_a_border(kind)
    n = len(x)
    assert n >= 20 and 0 < first.sum() < n
    logits = torch.stack((floats(-x), torch.zeros(n, device="cuda")), 1)
    limit = {} if kind == "u" else {kind: floats(value)}
    got = st.staple_sample(logits, floats(value if kind == "u" else np.zeros(n)), temperature=floats(t), **limit)["token"]
    fine(st)
    assert (got.cpu().numpy() == 0).tolist() == first.tolist()


def test_sampling_shares(st):
    """Over an even grid of random numbers each token comes up as often as its share says."""
    import torch
    p = torch.tensor([0.05, 0.4, 0.0, 0.25, 0.3], device="cuda")
    n = 4000
    u = (torch.arange(n, device="cuda") + 0.5) / n
    logits = p.log()[None].expand(n, 5)
    got = st.staple_sample(logits, u)["token"]
    share = torch.bincount(got, minlength=5).float() / n
    assert float((share - p).abs().max()) <= 1.0 / n
    fine(st)


def test_workspaces_in_host_memory_are_refused(st):
    import torch
    room = torch.empty(1 << 22, dtype=torch.uint8)
    x, w = rand((100, 64), "f32", 81), torch.ones(64, device="cuda")
    f = st.staple_norm_fwd(x, w_pre=w, save=True)
    dd = st.staple_dedup(ints(np.arange(100) % 3), 3)
    logits = rand((2, 100352), "bf16", 82)
    assert st.lib().staple_sample_workspace_bytes(2, 100352) > 0
    for call in (lambda: st.staple_norm_bwd(None, x, x, None, f["rstd_r"], w_pre=w, workspace=room),
                 lambda: st.staple_embed_bwd(x, dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], workspace=room),
                 lambda: st.staple_sample(logits, floats([0.5, 0.5]), workspace=room)):
        with pytest.raises(ValueError, match="workspace: needs"):
            call()
    fine(st)
