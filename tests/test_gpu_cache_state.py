"""The paged key-value cache at the ends of its arguments and where a step cannot
go on: what is read, and what stays as it is."""
import pytest

from attn_bounds import check
from helpers import to_np
from test_gpu_attn import decode_ref, ints, make_cache, rand, st  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = 2 ** 63 - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(FAR, 0), (FAR, 3), (FAR, FAR), (3001, 3), (3000, 1), (2999, 1), (1, FAR)])
def test_decode_window_past_every_key(st, dtype, window, sinks):
    """Windows and sinks as wide as the sequences and far wider, where many keys would be missed."""
    lens, h, hk, d, page = [3000, 70, 1], 8, 2, 64, 16
    print(dtype, window, sinks, flush=True)
    k, v, table, ln, _ = make_cache(dtype, lens, hk, d, page, 200)
    q = rand((3, h, d), dtype, 201)
    got = st.staple_attn_decode_paged(q, k, v, table, ln, window=window, sinks=sinks)
    (o, lse), (bo, bl) = decode_ref(dtype, q, k, v, table, ln, min(window, 1 << 40), min(sinks, 1 << 40), d ** -0.5)
    assert st.staple_get_device_error() == 0
    check(to_np(got["o"]), o, bo, "o")
    check(to_np(got["lse"]), lse, bl, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_len", [40, 33, 32, 16, 0])
def test_decode_of_a_sequence_past_the_bound_leaves_the_cache(st, dtype, max_len):
    """One sequence is longer than max_len, one as long: the first one's cache stays as it is."""
    import torch
    lens, h, hk, d, page = [41, max_len], 4, 2, 64, 16
    print(dtype, max_len, flush=True)
    k, v, table, ln, _ = make_cache(dtype, lens, hk, d, page, 210)
    q, kn, vn = rand((2, h, d), dtype, 211), rand((2, hk, d), dtype, 212), rand((2, hk, d), dtype, 213)
    want_k, want_v = k.clone(), v.clone()
    if max_len:
        st.staple_kv_append(kn[1:], vn[1:], want_k, want_v, table, ln, ints([1]))
    got = st.staple_attn_decode_paged(q, k, v, table, ln, k_new=kn, v_new=vn, max_len=max_len)
    assert st.staple_get_device_error() == -5
    assert torch.equal(k.nan_to_num(7), want_k.nan_to_num(7)) and torch.equal(v.nan_to_num(7), want_v.nan_to_num(7))
    # the cut one's result is that of the keys before the bound
    (o, lse), (bo, bl) = decode_ref(dtype, q, want_k, want_v, table, ints([max_len, max_len]), 0, 0, d ** -0.5)
    check(to_np(got["o"]), o, bo, "o")
    check(to_np(got["lse"]), lse, bl, "lse")
