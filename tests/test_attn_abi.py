"""Host-side refusals of the attention and cache entry points: nothing is enqueued."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from token_indexed_ffn_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libstaple.so is not built (run `python -m token_indexed_ffn_amd.build`)")
    _lib.load()
    return _lib


P = 256   # an aligned address that is never dereferenced: every call below is refused first


def attn(L, **change):
    f = dict(n_seqs=1, total_q=4, total_k=4, n_heads=4, n_kv_heads=2, head_dim=64, window=0, sinks=0, scale=0.125,
             dtype=1, cu_q=P, cu_k=P, lse=P, **{n: L.Heads(P, 256, 64) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")})
    f.update(change)
    return L.Attn(**f)


BAD_ATTN = [
    (dict(dtype=7), -2), (dict(head_dim=0), -2), (dict(head_dim=12), -2), (dict(head_dim=136), -2),
    (dict(n_kv_heads=3), -1), (dict(n_kv_heads=0), -1), (dict(total_q=-1), -1), (dict(n_seqs=-1), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(total_q=1 << 32), -2), (dict(cu_q=None), -1), (dict(cu_k=None), -1), (dict(lse=None), -1),
]


@pytest.mark.parametrize("change,status", BAD_ATTN, ids=lambda c: str(c))
def test_attention_refuses(L, change, status):
    a = attn(L, **change)
    lib = L.load()
    assert lib.staple_attn_fwd(ctypes.byref(a), P, 1 << 40, None) == status
    assert lib.staple_attn_bwd(ctypes.byref(a), P, 1 << 40, None) == status


@pytest.mark.parametrize("which", ["q", "k", "v", "o", "d_o", "dq", "dk", "dv"])
@pytest.mark.parametrize("bad", [(None, 256, 64), (P + 8, 256, 64), (P, 257, 64), (P, 256, 60), (P, -256, 64)])
def test_attention_refuses_operands(L, which, bad):
    a = attn(L, **{which: L.Heads(*bad)})
    lib = L.load()
    if which in ("q", "k", "v", "o"):
        assert lib.staple_attn_fwd(ctypes.byref(a), P, 1 << 40, None) == -1
    assert lib.staple_attn_bwd(ctypes.byref(a), P, 1 << 40, None) == -1


def test_attention_workspace_and_empty_calls(L):
    lib = L.load()
    a = attn(L)
    need = lib.staple_attn_bwd_workspace_bytes(ctypes.byref(a))
    assert need >= 4 * 4 * 4
    assert lib.staple_attn_bwd(ctypes.byref(a), P, need - 1, None) == -3
    assert lib.staple_attn_bwd(ctypes.byref(a), None, need, None) == -1
    long = attn(L, n_seqs=1, total_q=4, total_k=4096)
    need = lib.staple_attn_fwd_workspace_bytes(ctypes.byref(long))
    assert need > 0 and lib.staple_attn_fwd_workspace_bytes(None) == 0
    assert lib.staple_attn_fwd_workspace_bytes(ctypes.byref(attn(L, n_seqs=1, total_q=4, total_k=64))) == 0
    assert lib.staple_attn_fwd(ctypes.byref(long), P, need - 1, None) == -3
    assert lib.staple_attn_fwd(ctypes.byref(long), None, need, None) == -1
    assert lib.staple_attn_fwd(None, P, 1 << 40, None) == -1
    assert lib.staple_attn_bwd_workspace_bytes(None) == 0
    assert lib.staple_attn_fwd(ctypes.byref(attn(L, n_seqs=0)), None, 0, None) == 0
    assert lib.staple_attn_fwd(ctypes.byref(attn(L, total_q=0)), None, 0, None) == 0
    assert lib.staple_attn_bwd(ctypes.byref(attn(L, total_q=0, total_k=0)), None, 0, None) == 0


def kv(L, **change):
    f = dict(n_layers=1, n_pages=8, n_kv_heads=2, page_size=16, head_dim=64, n_rows=4, max_pages=4, dtype=1,
             k_pages=P, v_pages=P, refs=P, table=P, lens=P)
    f.update(change)
    return L.Kv(**f)


BAD_KV = [
    (dict(dtype=2), -2), (dict(head_dim=20), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(page_size=2048), -2), (dict(n_layers=0), -1), (dict(n_pages=0), -1), (dict(n_rows=0), -1),
    (dict(max_pages=0), -1), (dict(n_kv_heads=0), -1), (dict(n_layers=20000), -2),
]


@pytest.mark.parametrize("change,status", BAD_KV, ids=lambda c: str(c))
def test_cache_calls_refuse_bad_caches(L, change, status):
    lib, c, h = L.load(), kv(L, **change), L.Heads(P, 128, 64)
    c, h = ctypes.byref(c), ctypes.byref(h)
    d = decode(L)
    assert lib.staple_kv_append(c, h, h, 1, None, 1, None, None) == status
    assert lib.staple_kv_extend(c, P, None, 1, P, 1 << 30, None) == status
    assert lib.staple_kv_fork(c, P, P, 1, None) == status
    assert lib.staple_kv_free(c, P, 1, None) == status
    assert lib.staple_kv_compact(c, P, P, P, P, 1 << 30, None) == status
    assert lib.staple_kv_copy_pages(c, P, P, 1, None) == status
    assert lib.staple_attn_decode_paged(c, ctypes.byref(d), P, 1 << 30, None) == status


def test_cache_calls_refuse_missing_state(L):
    lib, h = L.load(), ctypes.byref(L.Heads(P, 128, 64))
    no = lambda n: ctypes.byref(kv(L, **{n: None}))
    for n in ("k_pages", "v_pages", "table", "lens"):
        assert lib.staple_kv_append(no(n), h, h, 1, None, 1, None, None) == -1
        assert lib.staple_attn_decode_paged(no(n), ctypes.byref(decode(L)), P, 1 << 30, None) == -1
    for n in ("k_pages", "v_pages", "table", "lens", "refs"):
        assert lib.staple_kv_extend(no(n), P, None, 1, P, 1 << 30, None) == -1
        assert lib.staple_kv_compact(no(n), P, P, P, P, 1 << 30, None) == -1
    for n in ("table", "lens", "refs"):
        assert lib.staple_kv_fork(no(n), P, P, 1, None) == -1
        assert lib.staple_kv_free(no(n), P, 1, None) == -1
    odd = ctypes.byref(kv(L, k_pages=P + 4))
    assert lib.staple_kv_append(odd, h, h, 1, None, 1, None, None) == -1


def test_cache_calls_refuse_bad_arguments(L):
    lib, c = L.load(), ctypes.byref(kv(L))
    h = L.Heads(P, 128, 64)
    hp, off = ctypes.byref(h), ctypes.byref(L.Heads(P + 2, 128, 64))
    assert lib.staple_kv_append(c, hp, off, 1, None, 1, None, None) == -1
    assert lib.staple_kv_append(c, hp, hp, 2, None, 1, None, None) == -1      # one row each
    assert lib.staple_kv_append(c, hp, hp, 5, None, 5, None, None) == -1      # rows past the table
    assert lib.staple_kv_append(c, hp, hp, -1, P, 1, P, None) == -1
    assert lib.staple_kv_append(ctypes.byref(kv(L, n_layers=2)), hp, hp, 1, None, 1, None, None) == -1
    need = lib.staple_kv_extend_workspace_bytes(c, 3)
    assert need > 0
    assert lib.staple_kv_extend(c, P, None, 3, P, need - 1, None) == -3
    assert lib.staple_kv_extend(c, P, None, 3, None, need, None) == -1
    assert lib.staple_kv_extend(c, None, None, 3, P, need, None) == -1
    assert lib.staple_kv_extend(c, P, None, -3, P, need, None) == -1
    assert lib.staple_kv_extend(c, P, None, 4097, P, 1 << 30, None) == -2
    assert lib.staple_kv_extend(c, None, None, 0, None, 0, None) == 0
    need = lib.staple_kv_compact_workspace_bytes(c)
    assert lib.staple_kv_compact(c, P, P, P, P, need - 1, None) == -3
    assert lib.staple_kv_compact(c, None, P, P, P, need, None) == -1
    assert lib.staple_kv_compact(c, P, P, None, P, need, None) == -1
    for call in (lib.staple_kv_fork, lib.staple_kv_copy_pages):
        assert call(c, None, P, 1, None) == -1 and call(c, P, P, -1, None) == -1 and call(c, P, P, 0, None) == 0
    assert lib.staple_kv_free(c, None, 1, None) == -1 and lib.staple_kv_free(c, None, 0, None) == 0


def decode(L, **change):
    f = dict(n_seqs=2, n_heads=4, max_len=64, window=0, sinks=0, scale=0.125, seqs=None, q=L.Heads(P, 256, 64),
             k_new=L.Heads(None, 0, 0), v_new=L.Heads(None, 0, 0), o=L.Heads(P, 256, 64), lse=None)
    f.update(change)
    return L.AttnDecode(**f)


def test_decode_refuses(L):
    lib, c = L.load(), ctypes.byref(kv(L))
    H = L.Heads
    for change in (dict(n_seqs=-1), dict(n_heads=3), dict(n_heads=0), dict(max_len=65), dict(max_len=-1), dict(window=-1),
                   dict(sinks=-1), dict(scale=float("nan")), dict(n_seqs=5), dict(q=H(None, 256, 64)),
                   dict(q=H(P + 4, 256, 64)), dict(o=H(P, 255, 64)), dict(k_new=H(P, 128, 64)),
                   dict(k_new=H(P, 128, 64), v_new=H(P, 128, 63))):
        assert lib.staple_attn_decode_paged(c, ctypes.byref(decode(L, **change)), P, 1 << 30, None) == -1, change
    assert lib.staple_attn_decode_paged(c, None, P, 1 << 30, None) == -1
    assert lib.staple_attn_decode_paged(ctypes.byref(kv(L, n_layers=2)), ctypes.byref(decode(L)), P, 1 << 30, None) == -1
    assert lib.staple_attn_decode_paged(c, ctypes.byref(decode(L, n_seqs=0)), None, 0, None) == 0


def test_binding_refuses_tensors_of_the_wrong_kind(L):
    import torch
    import token_indexed_ffn_amd as st
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):   # host tensors
        st.staple_attn_fwd(x, x, x, off, off)
    with pytest.raises(ValueError):
        st.staple_attn_decode_paged(x, x[None], x[None], off[None], off)
    with pytest.raises(ValueError):
        st.staple_kv_free(off, off[None], off, off, page_size=16)
