"""Host-side refusals of embedding, norms, loss and sampling: nothing is enqueued."""
import ctypes
import os

import pytest
import torch

import token_indexed_ffn_amd as st


@pytest.fixture(scope="module")
def L():
    from token_indexed_ffn_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libstaple.so is not built (run `python -m token_indexed_ffn_amd.build`)")
    _lib.load()
    return _lib


P = 256   # an aligned address that is never dereferenced: every call below is refused first
NAN, INF = float("nan"), float("inf")


def embed_fwd(L, **change):
    f = dict(table=P, vocab=10, d=64, dtype=1, ids=P, n=4, scale=1.0, y=P, y_stride=64, out_dtype=1)
    f.update(change)
    return L.load().staple_embed_fwd(*f.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), -2), (dict(out_dtype=2), -2), (dict(n=-1), -1), (dict(vocab=0), -1), (dict(d=0), -1),
    (dict(d=1 << 21), -2), (dict(n=1 << 30), -2), (dict(vocab=1 << 31), -2), (dict(scale=NAN), -1),
    (dict(scale=INF), -1), (dict(table=None), -1), (dict(table=P + 1), -1), (dict(ids=None), -1), (dict(y=None), -1),
    (dict(y=P + 2, out_dtype=0), -1), (dict(y_stride=63), -1), (dict(y_stride=-64, n=1), -1), (dict(n=0, table=None), 0)], ids=str)
def test_embedding_refuses(L, change, status):
    assert embed_fwd(L, **change) == status


def embed_bwd(L, **change):
    f = dict(dy=P, dy_stride=64, dtype=1, n=400, d=64, scale=1.0, sorted_pos=P, inv=P, seg_start=P, n_unique=P,
             max_unique=8, uniq=None, grad=P, grad_rows=8, accumulate=0, ws=P, ws_bytes=1 << 40)
    f.update(change)
    return L.load().staple_embed_bwd(*f.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), -2), (dict(n=-1), -1), (dict(d=0), -1), (dict(d=1 << 21), -2), (dict(n=1 << 30), -2),
    (dict(n=1 << 29, d=1 << 13), -2), (dict(scale=NAN), -1), (dict(max_unique=-1), -1), (dict(max_unique=9), -1),
    (dict(grad_rows=-1), -1), (dict(dy=None), -1), (dict(dy=P + 1), -1), (dict(dy_stride=-1), -1),
    (dict(sorted_pos=None), -1), (dict(inv=None), -1), (dict(seg_start=None), -1), (dict(n_unique=None), -1),
    (dict(grad=None), -1), (dict(grad=P + 2), -1), (dict(ws_bytes=16), -3), (dict(ws=None), -1), (dict(ws=P + 8), -1),
    (dict(n=0, dy=None), 0)], ids=str)
def test_embedding_gradient_refuses(L, change, status):
    assert embed_bwd(L, **change) == status


def test_embedding_gradient_workspace(L):
    size = L.load().staple_embed_bwd_workspace_bytes
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(40, 0) == 0 and size(40, 1 << 21) == 0
    assert size(400, 64) > 0
    assert embed_bwd(L, ws_bytes=size(400, 64) - 1) == -3


def norm(L, **change):
    f = dict(n_rows=4, d=64, dtype=1, r_dtype=1, w_dtype=1, pre=1, post=1, scale=1.0, eps=1e-6)
    f.update({n: L.Rows(P, 64) for n in ("x", "z", "r", "h", "gate")})
    f.update({n: P for n in ("w_pre", "w_post", "rstd_r", "rstd_z")})
    f.update({n: L.Rows(P, 64) for n in ("dr", "dh", "dx", "dz", "dgate")})
    f.update(dw_pre=P, dw_post=P)
    assert set(change) <= set(f)
    f.update(change)
    return L.Norm(*f.values())


BOTH = [
    (dict(dtype=2), -2), (dict(r_dtype=2), -2), (dict(w_dtype=2), -2), (dict(dtype=0, r_dtype=1), -2),
    (dict(n_rows=-1), -1), (dict(n_rows=1 << 22), -2), (dict(d=0), -1), (dict(d=16385), -2),
    (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1),
    (dict(eps=INF), -1), (dict(w_pre=P + 1), -1), (dict(w_post=P + 1), -1),
]


@pytest.mark.parametrize("change,status", BOTH, ids=str)
def test_norms_refuse(L, change, status):
    a = ctypes.byref(norm(L, **change))
    assert L.load().staple_norm_fwd(a, None) == status
    assert L.load().staple_norm_bwd(a, P, 1 << 40, None) == status


@pytest.mark.parametrize("name", ["x", "z", "r", "h", "gate"])
@pytest.mark.parametrize("bad", [(P + 1, 64), (P, -64)])
def test_norm_forward_refuses_operands(L, name, bad):
    assert L.load().staple_norm_fwd(ctypes.byref(norm(L, **{name: L.Rows(*bad)})), None) == -1


def test_norm_forward_refuses_combinations(L):
    call = lambda **k: L.load().staple_norm_fwd(ctypes.byref(norm(L, **k)), None)
    none = L.Rows(None, 0)
    assert call(x=none, z=none) == -1
    assert call(z=none, post=0, gate=none) == -1              # r is x and has no place of its own
    assert call(z=none, post=1, gate=none, r=none) == -1
    assert call(z=none, post=0, r=none) == -1                 # a gate of nothing
    assert call(z=none, post=0, gate=none, r=none, pre=0) == -1
    assert call(r=none) == -1 and call(h=none) == -1
    assert call(r=L.Rows(P, 63)) == -1 and call(h=L.Rows(P, 0)) == -1
    assert call(n_rows=0, r=none) == 0
    assert L.load().staple_norm_fwd(None, None) == -1


@pytest.mark.parametrize("name", ["dr", "dh", "r", "z", "dx", "dz", "dgate", "gate"])
@pytest.mark.parametrize("bad", [(P + 1, 64), (P, -64)])
def test_norm_backward_refuses_operands(L, name, bad):
    assert L.load().staple_norm_bwd(ctypes.byref(norm(L, **{name: L.Rows(*bad)})), P, 1 << 40, None) == -1


def test_norm_backward_refuses_combinations(L):
    call = lambda **k: L.load().staple_norm_bwd(ctypes.byref(norm(L, **k)), P, 1 << 40, None)
    none = L.Rows(None, 0)
    for missing in ("dh", "z"):
        assert call(**{missing: none}) == -1
    assert call(r=none, z=none, post=0, gate=none) == -1      # nothing to form r from
    assert call(x=L.Rows(P + 1, 64)) == -1
    assert call(rstd_r=None) == -1 and call(rstd_z=None) == -1
    assert call(pre=0, dr=none) == -1                         # no gradient comes in
    assert call(dw_pre=P + 2) == -1 and call(dw_post=P + 2) == -1
    assert call(dx=L.Rows(P, 63)) == -1 and call(dz=L.Rows(P, 0)) == -1 and call(dgate=L.Rows(P, 60)) == -1
    assert call(gate=L.Rows(P, 0), dgate=L.Rows(P + 2, 0)) == -1
    lib, a = L.load(), norm(L)
    need = lib.staple_norm_bwd_workspace_bytes(ctypes.byref(a))
    assert need >= 2 * 64 * 4 and lib.staple_norm_bwd_workspace_bytes(None) == 0
    assert lib.staple_norm_bwd(ctypes.byref(a), P, need - 1, None) == -3
    assert lib.staple_norm_bwd(ctypes.byref(a), None, need, None) == -1
    assert lib.staple_norm_bwd(ctypes.byref(a), P + 8, need, None) == -1
    # three vectors with a shared gate, none where no sum is asked for
    assert lib.staple_norm_bwd_workspace_bytes(ctypes.byref(norm(L, gate=L.Rows(P, 0)))) == need // 2 * 3
    assert lib.staple_norm_bwd_workspace_bytes(ctypes.byref(norm(L, dw_pre=None, dw_post=None))) == 0


def xent(L, **change):
    f = dict(logits=P, stride=100, n=4, vocab=100, dtype=1, targets=P, loss=P, lse=P, g=P, d_logits=P, d_stride=100)
    f.update(change)
    fwd = L.load().staple_xent_fwd(*f.values(), None)
    f.pop("loss")
    return fwd, L.load().staple_xent_bwd(*f.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), -2), (dict(n=-1), -1), (dict(n=1 << 22), -2), (dict(vocab=0), -1),
    (dict(vocab=(1 << 22) + 1), -2), (dict(stride=-1), -1), (dict(logits=None), -1), (dict(logits=P + 1), -1),
    (dict(targets=None), -1), (dict(lse=None), -1), (dict(g=None), -1), (dict(d_logits=None), -1),
    (dict(d_logits=P + 1), -1), (dict(d_stride=99), -1), (dict(n=0, logits=None, lse=None), 0)], ids=str)
def test_loss_refuses(L, change, status):
    assert xent(L, **change) == (status, status)


def test_loss_refuses_without_its_outputs(L):
    assert xent(L, loss=None)[0] == -1
    # the gradient and what it starts from come together
    lib = L.load()
    assert lib.staple_xent_fwd(P, 100, 4, 100, 1, P, P, P, None, P, 100, None) == -1
    assert lib.staple_xent_fwd(P, 100, 4, 100, 1, P, P, P, P, None, 100, None) == -1


def sample(L, **change):
    f = dict(logits=P, stride=100, n=4, vocab=100, dtype=1, u=P, temperature=P, top_k=P, top_p=P, min_p=P, token=P,
             logprob=P, ws=P, ws_bytes=1 << 40)
    f.update(change)
    return L.load().staple_sample(*f.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), -2), (dict(n=-1), -1), (dict(n=1 << 22), -2), (dict(vocab=0), -1),
    (dict(vocab=(1 << 22) + 1), -2), (dict(stride=-1), -1), (dict(logits=None), -1), (dict(logits=P + 1), -1),
    (dict(u=None), -1), (dict(token=None), -1), (dict(n=0, logits=None), 0)], ids=str)
def test_sampling_refuses(L, change, status):
    assert sample(L, **change) == status


def test_sampling_workspace(L):
    lib = L.load()
    assert lib.staple_sample_workspace_bytes(0, 100) == 0 and lib.staple_sample_workspace_bytes(1, 1 << 23) == 0
    need = lib.staple_sample_workspace_bytes(4, 100352)
    if need:
        assert sample(L, vocab=100352, stride=100352, ws_bytes=need - 1) == -3
        assert sample(L, vocab=100352, stride=100352, ws=None) == -1


def test_the_binding_refuses_what_is_not_on_the_device():
    f, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    v = torch.zeros(4)
    for call in (lambda: st.staple_embed_fwd(f, i), lambda: st.staple_norm_fwd(f), lambda: st.staple_norm_fwd(f, f),
                 lambda: st.staple_norm_bwd(f, f, f, None, v), lambda: st.staple_xent_fwd(f, i),
                 lambda: st.staple_xent_bwd(v, f, i, v), lambda: st.staple_sample(f, v),
                 lambda: st.staple_embed_bwd(f, i, torch.zeros(5, dtype=torch.int32), i, inv=i)):
        with pytest.raises(ValueError):
            call()


def test_the_binding_refuses_combinations():
    f, i, v = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(8)
    seg = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="given as out"):
        st.staple_embed_bwd(f, i, seg, i, inv=i, uniq=i)
    with pytest.raises(ValueError, match="given as out"):
        st.staple_embed_bwd(f, i, seg, i, inv=i, accumulate=True)
    with pytest.raises(ValueError, match="unique tokens"):
        st.staple_embed_bwd(f, i, seg, i, inv=i, out=f, max_unique=5)
    with pytest.raises(ValueError, match="unique tokens"):
        st.staple_embed_bwd(f, i, seg, i, inv=i, uniq=i, out=torch.zeros(9, 8), max_unique=5)
    with pytest.raises(ValueError, match="seg_start"):
        st.staple_embed_bwd(f, i, i, i, inv=i)
    with pytest.raises(ValueError, match="not done"):
        st.staple_norm_fwd(f, f, w_post=v)
    with pytest.raises(ValueError, match="not done"):
        st.staple_norm_fwd(f, f, w_pre=v, pre=False)
    with pytest.raises(ValueError, match="one dtype"):
        st.staple_norm_fwd(f, f, w_pre=v, w_post=v.bfloat16(), post=True)
    with pytest.raises(TypeError):
        st.staple_norm_fwd(f.double(), f.double())
    with pytest.raises(ValueError, match="x, z or both"):
        st.staple_norm_fwd(None)
    with pytest.raises(ValueError, match="x, z or both"):
        st.staple_norm_bwd(f, f, None)


def test_the_binding_refuses_two_types_of_one_output():
    f, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="out_dtype"):
        st.staple_embed_fwd(f, i, out=f, out_dtype=torch.bfloat16)
    # one of them, or both alike: refused for where the tensors are
    for how in (dict(out=f), dict(out_dtype=torch.bfloat16), dict(out=f, out_dtype=torch.float32)):
        with pytest.raises(ValueError, match="device"):
            st.staple_embed_fwd(f, i, **how)


def test_a_workspace_elsewhere_is_refused():
    """The kernels write there: host memory, another device's, or the gaps of a strided tensor are not handed to them."""
    here, room = torch.device("cpu"), torch.empty(64, dtype=torch.uint8)
    assert st._ws(64, room, here, None) is room and st._ws(0, None, here, None) is None
    for device, workspace in ((torch.device("cuda", 0), room), (here, torch.empty(256, dtype=torch.uint8)[::2]),
                              (here, torch.empty(64, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError, match="workspace: needs"):
            st._ws(64, workspace, device, None)
    with pytest.raises(ValueError, match="required"):
        st._ws(65, room, here, None)


def test_packed_norm_arguments_are_the_structure(L):
    head = (5, 8, 1, 0, 1, 1, 0, 0.5, 1e-6)
    rows = [(1000 + 8 * i, 10 + i) for i in range(10)]
    ends = [2000 + 8 * i for i in range(6)]
    flat = [v for r in rows for v in r]
    whole = bytes(L.Norm(*head, *rows[:5], *ends[:4], *rows[5:], *ends[4:]))
    assert L.pack_norm_bwd(*head, *flat[:10], *ends[:4], *flat[10:], *ends[4:]) == whole
    first = L.Norm(*head, *rows[:5], *ends[:4])
    assert L.pack_norm_fwd(*head, *flat[:10], *ends[:4]) == bytes(first)
