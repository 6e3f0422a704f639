"""Host-side arithmetic of the attention and cache entry points at the ends of
their arguments' ranges: nothing is enqueued."""
import ctypes
import os

import pytest

P = 256   # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    from token_indexed_ffn_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libstaple.so is not built (run `python -m token_indexed_ffn_amd.build`)")
    _lib.load()
    return _lib


def cache(L, **change):
    f = dict(n_layers=1, n_pages=8, n_kv_heads=16, page_size=16, head_dim=128, n_rows=64, max_pages=4096, dtype=1,
             k_pages=P, v_pages=P, refs=P, table=P, lens=P)
    f.update(change)
    return L.Kv(**f)


def decode(L, **change):
    f = dict(n_seqs=2, n_heads=16, max_len=65536, window=0, sinks=0, scale=0.1, seqs=None, q=L.Heads(P, 2048, 128),
             k_new=L.Heads(None, 0, 0), v_new=L.Heads(None, 0, 0), o=L.Heads(P, 2048, 128), lse=None)
    f.update(change)
    return L.AttnDecode(**f)


def decode_bytes(L, **change):
    return L.load().staple_attn_decode_workspace_bytes(ctypes.byref(cache(L)), ctypes.byref(decode(L, **change)))


FAR = 2 ** 63 - 1


@pytest.mark.parametrize("n_seqs", [1, 2, 64])
@pytest.mark.parametrize("max_len", [1, 64, 1000, 65536])
def test_a_window_that_hides_nothing_splits_like_none(L, n_seqs, max_len):
    """The workspace tells how the cache is split: a window of max_len keys or more, and as many
    sinks, leave every key visible."""
    want = decode_bytes(L, n_seqs=n_seqs, max_len=max_len)
    for window, sinks in ((max_len, 0), (max_len, 1), (FAR, 0), (FAR, 1), (FAR, FAR), (1, FAR), (2 ** 62, 2 ** 62)):
        assert decode_bytes(L, n_seqs=n_seqs, max_len=max_len, window=window, sinks=sinks) == want, (window, sinks)


@pytest.mark.parametrize("n_seqs", [(1 << 19) + 1, 1 << 60, 1 << 62, FAR])
def test_decode_refuses_more_rows_than_a_launch_has(L, n_seqs):
    """Sequences times heads: past 2^23, and past 64 bits in the last three."""
    lib, c, a = L.load(), ctypes.byref(cache(L)), ctypes.byref(decode(L, n_seqs=n_seqs, seqs=P))
    assert lib.staple_attn_decode_workspace_bytes(c, a) == 0
    assert lib.staple_attn_decode_paged(c, a, P, 1 << 40, None) == -2


def test_pages_of_more_bytes_than_32_bits_count_are_refused(L):
    """A page's pieces of 16 bytes are numbered in 32 bits, and so is what lies a stride past the last."""
    lib, h = L.load(), ctypes.byref(L.Heads(P, 1 << 20, 128))
    fine = dict(n_kv_heads=8192, page_size=1024, head_dim=128)   # 2^31 bytes in bf16
    for change in (dict(fine, n_kv_heads=8193), dict(fine, dtype=0), dict(fine, n_kv_heads=65535, dtype=0)):
        c = ctypes.byref(cache(L, **change))
        d = ctypes.byref(decode(L, n_heads=change["n_kv_heads"], n_seqs=1))
        assert lib.staple_kv_append(c, h, h, 1, None, 1, None, None) == -2
        assert lib.staple_kv_extend(c, P, None, 1, P, 1 << 30, None) == -2
        assert lib.staple_kv_compact(c, P, P, P, P, 1 << 30, None) == -2
        assert lib.staple_kv_copy_pages(c, P, P, 1, None) == -2
        assert lib.staple_attn_decode_paged(c, d, P, 1 << 40, None) == -2
    c = ctypes.byref(cache(L, **fine))
    assert lib.staple_kv_copy_pages(c, P, P, 0, None) == 0 and lib.staple_kv_extend(c, P, None, 0, P, 0, None) == 0


def attn(L, **change):
    f = dict(n_seqs=1, total_q=64, total_k=64, n_heads=1, n_kv_heads=1, head_dim=64, window=0, sinks=0, scale=0.125,
             dtype=1, cu_q=P, cu_k=P, lse=P, **{n: L.Heads(P, 256, 64) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")})
    f.update(change)
    return L.Attn(**f)


ROWS = 1 << 29
BF16_TILES = (1 << 23) - 4096 - 4        # workgroups of one head that are left for tokens and sequences


@pytest.mark.parametrize("within,past", [
    (dict(total_q=ROWS), dict(total_q=ROWS + 1)),
    (dict(total_k=ROWS), dict(total_k=ROWS + 1)),
    (dict(total_q=ROWS // 4, n_heads=4), dict(total_q=ROWS // 4 + 1, n_heads=4)),
    (dict(total_k=ROWS // 4, n_heads=4, n_kv_heads=4), dict(total_k=ROWS // 4 + 1, n_heads=4, n_kv_heads=4)),
    (dict(n_seqs=BF16_TILES), dict(n_seqs=BF16_TILES + 1)),
    (dict(n_seqs=BF16_TILES - 8, total_q=8 * 128), dict(n_seqs=BF16_TILES - 7, total_q=8 * 128)),
    (dict(dtype=0, n_seqs=(1 << 24) - 4102), dict(dtype=0, n_seqs=(1 << 24) - 4101)),   # 64 tokens are two tiles
    (dict(n_heads=100), dict(n_heads=65536)),
])
def test_packed_attention_limits_are_the_headers(L, within, past):
    """A workspace is asked for up to the limit; past it the call is refused."""
    lib = L.load()
    assert lib.staple_attn_bwd_workspace_bytes(ctypes.byref(attn(L, **within))) > 0
    a = ctypes.byref(attn(L, **past))
    assert lib.staple_attn_bwd_workspace_bytes(a) == 0
    assert lib.staple_attn_fwd(a, P, 1 << 60, None) == -2 and lib.staple_attn_bwd(a, P, 1 << 60, None) == -2


def test_cache_list_limits_are_the_headers(L):
    """Past the limit: unsupported.  At it the next check speaks, a missing operand."""
    lib, c, n = L.load(), ctypes.byref(cache(L)), 1 << 23
    for call in (lambda n: lib.staple_kv_append(c, None, None, n, P, n, None, None),
                 lambda n: lib.staple_kv_fork(c, None, None, n, None), lambda n: lib.staple_kv_free(c, None, n, None),
                 lambda n: lib.staple_kv_copy_pages(c, None, None, n, None)):
        assert call(n) == -1 and call(n + 1) == -2
    for change in (dict(n_layers=16384), dict(n_pages=1 << 31), dict(n_rows=1 << 31), dict(max_pages=1 << 31), dict(n_kv_heads=65536)):
        assert lib.staple_kv_copy_pages(ctypes.byref(cache(L, **change)), P, P, 0, None) == -2, change
    seqs = 1 << 19   # of 16 heads
    d = decode(L, n_seqs=seqs, seqs=P, max_len=4096)
    d.q.data = None
    assert lib.staple_attn_decode_paged(c, ctypes.byref(d), P, 1 << 60, None) == -1
    d.n_seqs = seqs + 1
    assert lib.staple_attn_decode_paged(c, ctypes.byref(d), P, 1 << 60, None) == -2
