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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_refused_step_leaves_the_cache_and_can_be_done_again(st, dtype):
    """Beams of one parent, with a shared, partly filled last page, and a row that fills its page
    run out of pages: neither an append nor an attention call of the same step writes anything.
    With pages freed, the same step gives what it gives in a pool that was large enough."""
    import torch
    h, hk, d, page, layers = 4, 2, 64, 16, 2
    lens = [21, 16, 30, 0, 0]
    kids = ints([3, 4])

    def cache(more):
        k, v, table, ln, refs = make_cache(dtype, lens, hk, d, page, 220, width=3, spare=2, layers=layers)
        k, v = (torch.cat([t, torch.full_like(t[:, :more], float("nan"))], dim=1) for t in (k, v))
        refs = torch.cat([refs, torch.zeros_like(refs[:more])])
        refused = torch.full((5,), 7, dtype=torch.int32, device="cuda")
        st.staple_kv_fork(refs, table, ln, ints([0, 0]), kids, page_size=page, refused=refused)
        assert refused.tolist() == [7, 7, 7, 0, 0]
        refused[:] = 0
        return k, v, table, ln, refs, refused

    rows = ints([0, 3, 4, 1])
    q, kn, vn = (rand((layers, 4, n, d), dtype, 221 + i) for i, n in enumerate((h, hk, hk)))

    def step(c, how):
        k, v, table, ln, refs, refused = c
        st.staple_kv_extend(refs, table, ln, rows, k_pages=k, v_pages=v, refused=refused)
        for i in range(layers):
            if how == "append":
                st.staple_kv_append(kn[i], vn[i], k[i], v[i], table, ln, rows, refused=refused)
                got = st.staple_attn_decode_paged(q[i], k[i], v[i], table, ln, seqs=rows, refused=refused)
            else:
                got = st.staple_attn_decode_paged(q[i], k[i], v[i], table, ln, seqs=rows, k_new=kn[i], v_new=vn[i],
                                                  refused=refused)
        return got

    for how in ("append", "attend"):
        print(dtype, how, flush=True)
        c = cache(0)   # two pages are free and the step needs four: three copies on write, and one page more
        before = [t.clone() for t in c]
        step(c, how)
        assert st.staple_get_device_error() == -8
        assert c[5].tolist() == [1, 1, 0, 1, 1]
        for name, a, b in zip(("k", "v", "table", "lens", "refs"), c, before):
            assert torch.equal(a.float().nan_to_num(7), b.float().nan_to_num(7)), name
        st.staple_kv_free(c[4], c[2], c[3], ints([2]), page_size=page, refused=c[5])
        got = step(c, how)
        assert st.staple_get_device_error() == 0 and c[5].tolist() == [0] * 5
        large = cache(6)
        want = step(large, how)
        assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
        for s in (0, 1, 3, 4):
            n = int(c[3][s])
            assert n == int(large[3][s])
            for a, b in ((c[0], large[0]), (c[1], large[1])):
                one, two = (t[:, tab[s].long()[:2]].transpose(2, 3).flatten(1, 2)[:, :n]
                            for t, tab in ((a, c[2]), (b, large[2])))
                assert torch.equal(one, two), (how, s)


def test_growth_marks_the_rows_that_it_leaves(st):
    """Rows that ask for nothing are never marked; bad counts and lengths are, the others grow."""
    import torch
    k, v, table, ln, refs = make_cache("bf16", [16, 5, 30, 9], 1, 8, 16, 230, width=3, spare=3, layers=1)
    ln[3] = -2
    refused = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    st.staple_kv_extend(refs, table, ln, ints([0, 1, 2, 3, 9]), ints([0, -1, 1, 1, 1]), k_pages=k, v_pages=v, refused=refused)
    assert st.staple_get_device_error() == -5
    assert refused.tolist() == [0, 1, 0, 1] and ln.tolist() == [16, 5, 31, -2]
    st.staple_kv_extend(refs, table, ln, ints([0, 1]), ints([33, 0]), k_pages=k, v_pages=v, refused=refused)   # past its width
    assert st.staple_get_device_error() == -8 and refused.tolist() == [1, 0, 0, 1] and ln.tolist() == [16, 5, 31, -2]
    with pytest.raises(ValueError):
        st.staple_kv_extend(refs, table, ln, ints([0]), k_pages=k, v_pages=v, refused=refused[:3])


@pytest.mark.parametrize("lens,h,hk,d,page,window,sinks", [
    ([37], 16, 16, 128, 16, 0, 0), ([300, 2, 90], 8, 2, 64, 32, 50, 4), ([5000, 17], 8, 2, 128, 64, 0, 0),
    ([700], 40, 1, 96, 16, 0, 0)])
def test_decode_weights_are_not_rounded_to_bf16(st, lens, h, hk, d, page, window, sinks):
    """Between the bf16 operands and the bf16 result a weight is off by 2^-17 of it (what two bf16
    numbers leave of it) and the bounds of fp32 arithmetic."""
    import numpy as np

    from attn_bounds import bounds
    from oracle import attn_oracle as A
    print(lens, h, hk, d, flush=True)
    k, v, table, ln, _ = make_cache("bf16", lens, hk, d, page, 240)
    q = rand((len(lens), h, d), "bf16", 241)
    got = st.staple_attn_decode_paged(q, k, v, table, ln, window=window, sinks=sinks)
    (o, _), _ = decode_ref("bf16", q, k, v, table, ln, window, sinks, d ** -0.5)
    nq, nk, nv, nt = (to_np(t) for t in (q, k, v, table))
    bound = np.zeros(o.shape)
    for i, n in enumerate(lens):
        j = np.arange(n)
        ks, vs = nk[nt[i, j // page], :, j % page], nv[nt[i, j // page], :, j % page]
        see = A.visible(1, n, window, sinks)
        for x in range(h):
            ops = nq[i:i + 1, x], ks[:, x // (h // hk)], vs[:, x // (h // hk)]
            out = A.attend(*ops, see, d ** -0.5)
            weights = (out["p"] @ np.abs(ops[2]))[0]
            bound[i, x] = bounds("f32", *ops, out, see, d ** -0.5)["o"][0] + 2.0 ** -17 * weights + 2.0 ** -8 * np.abs(out["o"][0])
    check(to_np(got["o"]), o, bound, "o")
