"""Row strides so large that a head's rows pass the 2^31 bytes of a buffer: every
kernel in its form with 64-bit addresses, against the one without."""
import pytest

from test_gpu_attn import cu, rand, st  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,h,hk,d,window,sinks", [
    ([70], 2, 1, 128, 0, 0), ([33, 60], 4, 2, 96, 20, 3), ([70], 2, 2, 64, 0, 0), ([40, 1, 50], 2, 1, 40, 0, 0),
    ([1100], 1, 1, 128, 0, 0), ([1100], 1, 1, 64, 200, 5)])   # the last two in parts
def test_rows_past_a_buffer(st, dtype, lens, h, hk, d, window, sinks):
    import torch
    n = sum(lens)
    size = 2 if dtype == "bf16" else 4
    stride = ((1 << 32) // size // n + 1024) // 8 * 8   # the last rows lie past 2^32 bytes
    c = cu(lens)
    mask = dict(window=window, sinks=sinks)
    ops = dict(zip(("q", "k", "v", "do"), (rand((n, m, d), dtype, 440 + i) for i, m in enumerate((h, hk, hk, h)))))
    buf = torch.empty(n * stride + h * d, dtype=ops["q"].dtype, device="cuda")
    view = lambda t: buf.as_strided(t.shape, (stride, d, 1))

    def run(x, out=None, grads=None):
        f = st.staple_attn_fwd(x["q"], x["k"], x["v"], c, c, out=out, **mask)
        return f | st.staple_attn_bwd(x["do"], x["q"], x["k"], x["v"], f["o"], f["lse"], c, c, out=grads, **mask)

    want = run(ops)
    for name, t in ops.items():
        print(dtype, lens, d, name, flush=True)
        view(t).copy_(t)
        got = run(ops | {name: view(t)})
        for m in want:
            assert torch.equal(got[m], want[m]), (name, m)
    for name in ("o", "dq", "dk", "dv"):   # results into such rows
        out = {m: view(want[m]) if m == name else torch.empty_like(want[m]) for m in want}
        got = run(ops, {m: out[m] for m in ("o", "lse")}, {m: out[m] for m in ("dq", "dk", "dv")})
        for m in want:
            assert torch.equal(got[m], want[m]), (name, m)
    assert st.staple_get_device_error() == 0
