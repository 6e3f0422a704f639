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
