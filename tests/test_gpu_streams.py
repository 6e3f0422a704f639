"""Calls on a stream other than the current one."""
import pytest

from test_gpu_attn import cu, ints, make_cache, rand, st  # noqa: F401

pytestmark = pytest.mark.gpu


def busy(stream):
    """Work that holds the stream up for some milliseconds."""
    import torch
    with torch.cuda.stream(stream):
        x = torch.ones(4096, 4096, device="cuda")
        for _ in range(20):
            x = torch.tanh(x @ x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_memory_of_a_call_on_another_stream_is_not_handed_out(st, dtype):
    """While calls with workspaces wait on a held up stream, the current one allocates and fills
    blocks of every size that they could have left: neither side touches the other's."""
    import torch
    q, do = rand((1300, 4, 64), dtype, 300), rand((1300, 4, 64), dtype, 301)
    k, v = rand((1300, 1, 64), dtype, 302), rand((1300, 1, 64), dtype, 303)
    c = cu([900, 400])
    lens = [5000, 300]
    kp, vp, table, ln, refs = make_cache(dtype, lens, 2, 64, 16, 304, width=320, spare=40)
    qd, rows = rand((2, 4, 64), dtype, 305), ints([0, 1])

    def calls(kq, vq, t, n, r, **on):
        f = st.staple_attn_fwd(q, k, v, c, c, **on)
        b = st.staple_attn_bwd(do, q, k, v, f["o"], f["lse"], c, c, **on)
        st.staple_kv_extend(r, t, n, rows, k_pages=kq[None], v_pages=vq[None], **on)
        st.staple_kv_append(k[:2].expand(2, 2, 64), v[:2].expand(2, 2, 64), kq, vq, t, n, rows, **on)
        d = st.staple_attn_decode_paged(qd, kq, vq, t, n, **on)
        p = st.staple_kv_compact(r, t, n, kq[None], vq[None], **on)
        return [*f.values(), *b.values(), *d.values(), kq, vq, p["table"], p["refs"], p["n_live"]]

    state = (kp.nan_to_num(7), vp.nan_to_num(7), table, ln, refs)
    want = calls(*(x.clone() for x in state))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        busy(side)
        with torch.cuda.stream(side):   # the cache, which the calls change
            mine = [x.clone() for x in state]
        got = calls(*mine, stream=side)
        blocks = [torch.full((1 << s,), 5, dtype=torch.uint8, device="cuda") for s in range(8, 25) for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert all(bool((x == 5).all()) for x in blocks)
    assert st.staple_get_device_error() == 0


@pytest.mark.parametrize("raw", [True, False])
def test_calls_go_to_the_current_stream(st, raw, monkeypatch):
    """With and without torch's raw handle of the current stream."""
    import torch
    if not raw:
        monkeypatch.setattr(st, "_raw_stream", None)
    assert st._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert st._stream(None) == side.cuda_stream != torch.cuda.default_stream().cuda_stream
    assert st._stream(None) == torch.cuda.current_stream().cuda_stream
