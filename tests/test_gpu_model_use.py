"""Embedding, norms, loss and sampling as they are used: together, captured and replayed, on other
streams, again and again, over rows far apart in memory."""
import os
import sys

import numpy as np
import pytest

import model_bounds as B
from attn_bounds import check
from helpers import to_np
from oracle import model_oracle as M
from test_gpu_attn import TORCH, ints, rand, st  # noqa: F401
from test_gpu_model import XENT_CHAIN, fine, floats
from test_gpu_streams import busy

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


class Step:
    """A small model's training step and its serving step on the library's calls, projections in torch:
    embedding, two seams with norms and gates, logits, loss, and all gradients back to the table."""

    def __init__(self, dtype, seed=0, n=333, vocab=1000, d=264, room=None):
        import torch
        self.n, self.vocab, self.d = n, vocab, d
        self.dtype = getattr(torch, TORCH[dtype])
        self.table = rand((vocab, d), "f32", seed + 100, 0.5)
        self.ids = torch.from_numpy(np.random.default_rng(seed).integers(0, vocab, n).astype(np.int32)).cuda()
        self.targets = torch.roll(self.ids, -1)
        self.targets[::7] = -1
        self.w = [1 + rand((d,), "f32", seed + 101 + i, 0.1) for i in range(4)]
        self.gate = rand((n, d), dtype, seed + 105)
        self.mix = [rand((d, d), dtype, seed + 106 + i, d ** -0.5) for i in range(2)]
        self.g = torch.full((n,), 1.0 / n, device="cuda")
        self.u = torch.rand(n, generator=torch.Generator().manual_seed(seed)).cuda()
        self.k = ints([0, 5, 50] * (n // 3))
        self.p = floats(np.linspace(0.5, 1.2, n))
        self.temperature = floats(np.linspace(0.0, 2.0, n))

    def __call__(self, st, ws=None, **on):
        import torch
        seam = [dict(w_pre=self.w[0], w_post=self.w[1], post=True, gate=self.w[2]), dict(w_pre=self.w[3], gate=self.gate, scale=0.5)]
        space = {} if ws is None else {"workspace": ws}
        dd = st.staple_dedup(self.ids, self.vocab, **on)
        x = st.staple_embed_fwd(self.table, self.ids, scale=4.0, out_dtype=self.dtype, **on)
        xs, zs, fs, h = [], [], [], x
        for mix, how in zip(self.mix, seam):
            z = h @ mix
            f = st.staple_norm_fwd(x, z, save=True, **how, **on)
            xs.append(x), zs.append(z), fs.append(f)
            x, h = f["r"], f["h"]
        logits = h @ self.table.to(h.dtype).T
        token = st.staple_sample(logits, self.u, temperature=self.temperature, top_k=self.k, top_p=self.p, **space, **on)
        loss = st.staple_xent_fwd(logits, self.targets, g=self.g, **on)
        dh, dr, grads = loss["d_logits"] @ self.table.to(h.dtype), None, []
        for i in (1, 0):
            b = st.staple_norm_bwd(dr, dh, xs[i], zs[i], fs[i]["rstd_r"], fs[i]["rstd_z"], **seam[i], **space, **on)
            grads += [b[k] for k in ("dw_pre", "dw_post", "dgate") if b[k] is not None]
            dr, dh = b["dx"], b["dz"] @ self.mix[i].T.contiguous()
        dy = dr + dh
        rows = st.staple_embed_bwd(dy, dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], uniq=dd["uniq"], scale=4.0,
                                   out=torch.zeros(self.vocab, self.d, device="cuda"), **space, **on)
        return [token["token"], token["logprob"], loss["loss"], loss["lse"], loss["d_logits"], *grads, dy, rows]

    def change(self, seed):
        """Other inputs in the same memory."""
        other = Step("f32" if self.dtype.itemsize == 4 else "bf16", seed, self.n, self.vocab, self.d)
        for k in ("table", "ids", "targets", "gate", "u"):
            getattr(self, k).copy_(getattr(other, k))


def workspace(st):
    import torch
    return torch.empty(1 << 26, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_step_is_the_same_every_time(st, dtype):
    import torch
    step = Step(dtype)
    want = step(st)
    fine(st)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for _ in range(5):
        for x, y in zip(step(st), want):
            assert torch.equal(x, y)
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_captured_steps_share_a_workspace(st, dtype):
    """Two graphs that were captured with one workspace, replayed in turn over changed inputs, with
    eager steps that use it too in between."""
    import torch
    ws = workspace(st)
    steps = [Step(dtype, 1), Step(dtype, 2, n=60, vocab=5003, d=520)]
    graphs, outs = [], []
    for s in steps:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s(st, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s(st, ws))
        graphs.append(g)
    for turn in range(4):
        for s, g, out in zip(steps, graphs, outs):
            s.change(10 + turn)
            want = s(st, ws)
            torch.cuda.synchronize()
            g.replay()
            for x, y in zip(out, want):
                assert torch.equal(x, y), turn
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,vocab", [(37, 8201, 70001), (130, 16384, 131080)])
def test_wide_rows_captured_and_replayed(st, dtype, n, d, vocab):
    """Norms whose backward takes two passes and a loss that reads its rows twice, in a graph, with the same calls
    between its replays."""
    import torch
    x, z, dr, dh = (rand((n, d), dtype, 70 + i) for i in range(4))
    logits, targets, g = rand((n, vocab), dtype, 74, 3.0), ints(np.arange(n) * 7 % vocab), floats(np.linspace(-1, 1, n))
    w = 1 + rand((d,), "f32", 75, 0.1)
    ws = workspace(st)

    def run():
        how = dict(w_pre=w, w_post=w, gate=w, post=True)
        f = st.staple_norm_fwd(x, z, save=True, **how)
        b = st.staple_norm_bwd(dr, dh, x, z, f["rstd_r"], f["rstd_z"], workspace=ws, **how)
        loss = st.staple_xent_fwd(logits, targets, g=g)
        return [f["r"], f["h"], *(t for t in b.values() if t is not None), *loss.values()]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for turn in range(4):
        for t in (x, z, dr, dh, logits):
            t.copy_(torch.roll(t, 1, 0))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_memory_of_a_step_on_another_stream_is_not_handed_out(st, dtype):
    import torch
    step = Step(dtype, 3)
    x, z, dh = rand((700, 520), dtype, 120), rand((700, 520), dtype, 121), rand((700, 520), dtype, 122)
    w = 1 + rand((520,), "f32", 123, 0.1)
    logits, t = rand((90, 5001), dtype, 124, 3.0), ints(range(90))
    ones = torch.ones(90, device="cuda")
    half, most = ones * 0.5, ones * 0.9   # kept here until the other stream has used them
    ids = ints(np.arange(700) % 11)
    dd = st.staple_dedup(ids, 11)

    def calls(**on):
        y = st.staple_embed_fwd(x, ids, scale=2.0, **on)
        e = st.staple_embed_bwd(z, dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], max_unique=11, **on)
        f = st.staple_norm_fwd(x, z, w_pre=w, w_post=w, post=True, save=True, **on)
        b = st.staple_norm_bwd(x, dh, x, z, f["rstd_r"], f["rstd_z"], w_pre=w, w_post=w, post=True, **on)
        l = st.staple_xent_fwd(logits, t, g=ones, **on)
        d = st.staple_xent_bwd(ones, logits, t, l["lse"], **on)
        s = st.staple_sample(logits, half, top_k=t, top_p=most, **on)
        return [v for v in (y, e, *f.values(), *b.values(), *l.values(), d, *s.values()) if v is not None]

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        busy(side)
        got = calls(stream=side)
        blocks = [torch.full((1 << s,), 5, dtype=torch.uint8, device="cuda") for s in range(8, 25) for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert all(bool((b == 5).all()) for b in blocks)
    # two streams at once
    other = torch.cuda.Stream()
    for s in (side, other):
        s.wait_stream(torch.cuda.current_stream())
    both = [calls(stream=s) for _ in range(3) for s in (side, other)]
    for s in (side, other):
        torch.cuda.current_stream().wait_stream(s)
    for got in both:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    fine(st)
    step(st)
    fine(st)


# ------------------------------------------------------------------------------------ far offsets
def far_rows(t, stride):
    """The same rows `stride` elements apart, past 2^31 elements in all."""
    import torch
    n, d = t.shape
    room = torch.empty((n - 1) * stride + d, dtype=t.dtype, device="cuda")
    far = torch.as_strided(room, (n, d), (stride, 1))
    far.copy_(t)
    return far


FAR = (1 << 30) + 24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("odd", [0, 1])
def test_rows_past_32_bits(st, dtype, odd):
    """Three rows that begin more than 2^30 elements (2^32 bytes in fp32) apart: every call gives what it
    gives for rows side by side."""
    import torch
    stride, d = FAR + odd, 1003 if odd else 1008
    x, z, w = rand((3, d), dtype, 130), rand((3, d), dtype, 131), 1 + rand((d,), "f32", 132, 0.1)
    how = dict(w_pre=w, w_post=w, post=True)
    f = st.staple_norm_fwd(x, z, save=True, **how)
    g = st.staple_norm_bwd(x, z, x, z, f["rstd_r"], f["rstd_z"], **how)
    far = far_rows(x, stride)
    got = st.staple_norm_fwd(far, z, save=True, out={**{k: torch.empty_like(t) for k, t in f.items()}, "r": far}, **how)
    assert torch.equal(got["r"], f["r"]) and torch.equal(got["h"], f["h"])
    far.copy_(x)
    got = st.staple_norm_bwd(far, z, far, z, f["rstd_r"], f["rstd_z"], out={"dx": far, "dw_pre": torch.empty(d, device="cuda")}, **how)
    assert torch.equal(got["dx"], g["dx"]) and torch.equal(got["dw_pre"], g["dw_pre"])
    # loss and sampling
    t, ones = ints([1, 2, 3]), torch.ones(3, device="cuda")
    limits = dict(top_k=ints([0, 40, 7]), top_p=floats([0.8, 0.9, 1.0]))
    a, s = st.staple_xent_fwd(x, t, g=ones), st.staple_sample(x, ones * 0.4, **limits)
    back = st.staple_xent_bwd(ones, x, t, a["lse"])
    far.copy_(x)
    for k, v in st.staple_sample(far, ones * 0.4, **limits).items():
        assert torch.equal(v, s[k])
    got = st.staple_xent_fwd(far, t, g=ones, out={"loss": torch.empty_like(a["loss"]), "lse": torch.empty_like(a["lse"]), "d_logits": far})
    if odd:   # rows that begin elsewhere between 16-byte addresses lie otherwise in the registers: other orders of sums
        ref = M.xent(to_np(x), [1, 2, 3], np.ones(3))
        bound = B.xent(ref, to_np(x), np.array([1, 2, 3]), np.ones(3), dtype, XENT_CHAIN(d))
        for k, v in got.items():
            check(to_np(v), ref[k], bound[k], k)
    else:
        assert all(torch.equal(v, a[k]) for k, v in got.items())
    far.copy_(x)
    assert torch.equal(st.staple_xent_bwd(ones, far, t, a["lse"], out=far), back)
    # embedding: rows written and read far apart
    ids = ints([2, 0, 2])
    y = st.staple_embed_fwd(x, ids, out=far, scale=2.0)
    assert torch.equal(y, st.staple_embed_fwd(x, ids, scale=2.0))
    dd = st.staple_dedup(ids, 3)
    far.copy_(z)
    maps = (dd["sorted_pos"], dd["seg_start"], dd["n_unique"])
    assert torch.equal(st.staple_embed_bwd(far, *maps, inv=dd["inv"], max_unique=2), st.staple_embed_bwd(z, *maps, inv=dd["inv"], max_unique=2))
    fine(st)


def test_a_table_past_32_bits(st):
    import torch
    vocab, d = 1_100_000, 2048
    table = torch.zeros(vocab, d, dtype=torch.bfloat16, device="cuda")
    ids = ints([vocab - 1, 0, vocab - 1, 1_050_000])
    rows = rand((4, d), "bf16", 140)
    table[ids.long()] = rows
    want = table[ids.long()]
    assert torch.equal(st.staple_embed_fwd(table, ids), want)
    del table
    grad = torch.zeros(vocab, d, device="cuda")
    dd = st.staple_dedup(ids, vocab)
    st.staple_embed_bwd(rows, dd["sorted_pos"], dd["seg_start"], dd["n_unique"], inv=dd["inv"], uniq=dd["uniq"], out=grad)
    assert torch.equal(grad[vocab - 1], rows[0].float() + rows[2].float()) and torch.equal(grad[1_050_000], rows[3].float())
    assert torch.equal(grad[0], rows[1].float()) and int((grad != 0).any(dim=1).sum()) == 3
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_are_sampled_as_few_are(st, dtype):
    """More rows than are worked on at once, rows that begin between 16-byte addresses."""
    import torch
    n, v = 2500, 301
    logits = rand((n, v + 2), dtype, 150, 3.0)[:, 1:-1]
    r = np.random.default_rng(3)
    given = dict(temperature=floats(2 * r.random(n)), top_k=ints(r.integers(0, 60, n)), top_p=floats(0.3 + r.random(n)),
                 min_p=floats(0.1 * r.random(n)))
    u = floats(r.random(n))
    all_rows = st.staple_sample(logits, u, **given)
    for a, b in ((0, 7), (1020, 1030), (2040, 2060), (2493, 2500)):
        few = st.staple_sample(logits[a:b], u[a:b], **{k: t[a:b] for k, t in given.items()})
        for k, t in few.items():
            assert torch.equal(t, all_rows[k][a:b])
    free = st.staple_sample(logits, u)
    assert torch.equal(st.staple_sample(logits[2400:], u[2400:])["token"], free["token"][2400:])
    fine(st)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [301, 7001, 16800, 16900, 32001, 60001, 100352])
def test_rows_are_sampled_alike_alone_and_among_many(st, dtype, v):
    """One workgroup for a row, several, a row in registers: the same tokens to the bit, from rows that begin
    at and between 16-byte addresses."""
    import torch
    n = 130
    r = np.random.default_rng(v)
    u, given = floats(r.random(n)), dict(temperature=floats(0.1 + 1.5 * r.random(n)), min_p=floats(0.2 * r.random(n)))
    more = dict(top_k=ints(r.integers(0, 3000, n)), top_p=floats(0.3 + r.random(n)))
    for pad in (0, 1):
        logits = rand((n, v + pad), dtype, 160, 3.0)[:, pad:]
        for limits in (given, {**given, **more}):
            all_rows = st.staple_sample(logits, u, **limits)
            for a, b in ((0, 1), (40, 47), (120, 130)):
                few = st.staple_sample(logits[a:b], u[a:b], **{k: t[a:b] for k, t in limits.items()})
                for k, t in few.items():
                    assert torch.equal(t, all_rows[k][a:b])
    fine(st)


# ------------------------------------------------------------------------------------ the example
def plain(example):
    """The example's functions in torch's own operations."""
    import torch

    class Embed:
        @staticmethod
        def apply(table, ids, batch, dtype):
            return table[ids.long()].to(dtype)

    class AddNorm:
        @staticmethod
        def apply(x, z, weight):
            r = x if z is None else x + z
            h = r * torch.rsqrt(r.pow(2).mean(dim=1, keepdim=True) + 1e-6) * weight
            return h if z is None else (r, h)

    class Loss:
        @staticmethod
        def apply(logits, target):
            return torch.nn.functional.cross_entropy(logits, target.long(), ignore_index=-100)

    return dict(Embed=Embed, AddNorm=AddNorm, Loss=Loss)


def test_the_examples_gradients(st, monkeypatch):
    """A loss and all its gradients through the example's own functions, and with torch's operations in their
    place.  Both are fp32: the operands' relative differences are some hundred roundings in each of
    the ten stages that a gradient passes, by sums of up to 1000 terms: 2^-24 512 10 of its largest
    element."""
    import torch
    sys.path.insert(0, EXAMPLES)
    try:
        import attention_ffn_layers as example
    finally:
        sys.path.remove(EXAMPLES)
    model = example.Model(torch.float32, seed=4)
    gen = torch.Generator().manual_seed(9)
    lens = [40, 1, 90]
    ids = torch.randint(example.VOCAB, (sum(lens),), generator=gen, dtype=torch.int32).cuda()
    cu = example.offsets(lens)
    target = torch.roll(ids, -1)
    target[cu[1:].long() - 1] = -100

    def run():
        for p in model.parameters():
            p.grad = None
        loss = example.Loss.apply(model.forward(ids, cu), target)
        loss.backward()
        return loss.detach(), [p.grad.clone() for p in model.parameters()]

    loss, grads = run()
    fine(st)
    for name, f in plain(example).items():
        monkeypatch.setattr(example, name, f)
    want, others = run()
    most = 2.0 ** -24 * 512 * 10
    assert abs(float(loss - want)) <= most * float(want)
    for a, b in zip(grads, others):
        assert float((a - b).abs().max()) <= most * float(b.abs().max())
