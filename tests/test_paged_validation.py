"""CPU: refusals of the per-head norm and paged-cache entry points, by the binding (dtype,
shape, stride and alignment checks made before the device check) and by the C ABI."""

import ctypes

import pytest
import torch

import block_sparse_attention_tcgen05_b200 as bsa
from block_sparse_attention_tcgen05_b200 import _lib, build

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def _norm(S=8, D=64, dt=BF):
    return (torch.zeros(1, 4, S, D, dtype=dt), torch.zeros(1, 2, S, D, dtype=dt), torch.ones(D),
            torch.ones(D), torch.ones(S, D // 2), torch.zeros(S, D // 2))


@pytest.mark.parametrize("backward", [False, True])
def test_norm_arguments(backward):
    q, k, qw, kw, c, s = _norm()

    def f(q, k, *a, **kw):
        if backward:
            return bsa.qk_norm_rotation_backward(q, k, q, k, *a, **kw)
        return bsa.qk_norm_rotation(q, k, *a, **kw)
    _raises("q: dtype", f, q.double(), k, qw, kw, c, s)
    _raises("k: dtype", f, q, k.float(), qw, kw, c, s)
    _raises("k: shape", f, q, k[:, :, :7], qw, kw, c, s)
    _raises("q_weight: dtype", f, q, k, qw.half(), kw, c, s)
    _raises("k_weight: dtype", f, q, k, qw, kw.to(BF), c, s)
    _raises("q_weight: shape", f, q, k, torch.ones(32), kw, c, s)
    _raises("cos: shape", f, q, k, qw, kw, torch.ones(8, 64), s)
    _raises("sin: shape", f, q, k, qw, kw, c, torch.ones(9, 32))
    _raises("positions for 8 tokens", f, q, k, qw, kw, c[:7], s[:7])
    _raises("positions: dtype", f, q, k, qw, kw, c, s, positions=torch.zeros(8, dtype=torch.int64))
    _raises("positions: shape", f, q, k, qw, kw, c, s, positions=torch.zeros(9, dtype=I32))
    _raises("last dimension", f, torch.zeros(1, 4, 64, 8, dtype=BF).transpose(2, 3), k, qw, kw, c, s)
    odd = torch.zeros(1, 4, 8, 66, dtype=BF)[..., :64]
    _raises("multiples of 16 bytes", f, odd, k, qw, kw, c, s)
    off = torch.zeros(1 * 4 * 8 * 64 + 1, dtype=BF)[1:].view(1, 4, 8, 64)
    _raises("multiples of 16 bytes", f, off, k, qw, kw, c, s)
    _raises("CUDA tensors only", f, q, k, qw, kw, c, s)
    if not backward:
        _raises("q_out: shape", f, q, k, qw, kw, c, s, q_out=k)
        _raises("k_out: dtype", f, q, k, qw, kw, c, s, k_out=k.float())


def test_table_arguments():
    c, n = torch.zeros(3, dtype=I32), torch.ones(3, dtype=I32)
    t, fr = torch.zeros(3, 4, dtype=I32), torch.zeros(5, dtype=I32)
    f = bsa.paged_block_tables
    _raises("context_lens: dtype", f, c.long(), n, t, fr, 3, 16, 9)
    _raises("new_lens: shape", f, c, n[:2], t, fr, 3, 16, 9)
    _raises("block_table: 2 rows", f, c, n, t[:2], fr, 3, 16, 9)
    _raises("rows must be contiguous", f, c, n, torch.zeros(4, 3, dtype=I32).t(), fr, 3, 16, 9)
    _raises("rows may not overlap", f, c, n, torch.zeros(1, 4, dtype=I32).expand(3, 4), fr, 3, 16, 9)
    _raises("free_pages: dtype", f, c, n, t, fr.long(), 3, 16, 9)
    _raises("CUDA tensors only", f, c, n, t, fr, 3, 16, 9)


def _paged():
    kc = torch.zeros(5, 2, 16, 64, dtype=BF)
    return (torch.zeros(4, 3, 64, dtype=BF), kc, kc.clone(), torch.zeros(2, 3, dtype=I32),
            torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32))


def test_attention_arguments():
    q, kc, vc, t, cu, ctx = _paged()
    f = bsa.paged_chunk_attention
    _raises("q: dtype", f, q.float(), kc, vc, t, cu, ctx)
    _raises("k_cache: dtype", f, q, kc.half(), vc, t, cu, ctx)
    _raises("v_cache: shape", f, q, kc, vc[:4], t, cu, ctx)
    _raises("k_cache: shape", f, torch.zeros(4, 3, 128, dtype=BF), kc, vc, t, cu, ctx)
    _raises("not a multiple", f, torch.zeros(3, 3, 64, dtype=BF), kc, vc, t, cu, ctx)
    _raises("k_cache: may not be broadcast", f, q, kc[:1].expand(5, 2, 16, 64), vc, t, cu, ctx)
    _raises("k_cache: pointer and strides", f, q, torch.zeros(5, 2, 16, 68, dtype=BF)[..., :64], vc, t, cu, ctx)
    _raises("block_table: dtype", f, q, kc, vc, t.long(), cu, ctx)
    _raises("cu_new: shape", f, q, kc, vc, t, cu[:2], ctx)
    _raises("context_lens: dtype", f, q, kc, vc, t, cu, ctx.long())
    _raises("page_mask", f, q, kc, vc, t, cu, ctx, page_mask=torch.ones(2, 2, 3))
    _raises("page_mask: shape", f, q, kc, vc, t, cu, ctx, page_mask=torch.ones(2, 2, 4, dtype=torch.bool))
    _raises("page_mask: shape", f, q, kc, vc, t, cu, ctx, page_mask=torch.ones(2, 3, 3, dtype=torch.bool))
    _raises("out: dtype", f, q, kc, vc, t, cu, ctx, out=q.float())
    _raises("workspace: dtype", f, q, kc, vc, t, cu, ctx, workspace=q)
    _raises("CUDA tensors only", f, q, kc, vc, t, cu, ctx)


def test_append_arguments():
    q, kc, vc, *_ = _paged()
    k = torch.zeros(2, 3, 64, dtype=BF)
    w, cos, pos = torch.ones(64), torch.ones(9, 32), torch.zeros(3, dtype=I32)
    f = bsa.paged_qk_norm_append
    ok = (q, k, k, w, w, cos, cos, pos, pos, kc, vc)

    def with_(i, x):
        return ok[:i] + (x,) + ok[i + 1:]
    _raises("q: dtype", f, *with_(0, q.float()))
    _raises("k: shape", f, *with_(1, k[:, :2]))
    _raises("v: shape", f, *with_(2, k[:1]))
    _raises("positions: shape", f, *with_(7, pos[:2]))
    _raises("slots: dtype", f, *with_(8, pos.long()))
    _raises("k_cache: dtype", f, *with_(9, kc.half()))
    _raises("v_cache: shape", f, *with_(9, kc[:, :1]))
    _raises("CUDA tensors only", f, *ok)


def _cache(dtype=_lib.BSA_BF16, page=16, D=64, n=8, Hkv=2, stride=None, k=1 << 20):
    st = stride if stride is not None else D
    return _lib.PagedCache(k, 1 << 20, n, page, Hkv, D, dtype, Hkv * page * D, page * D, st,
                           Hkv * page * D, page * D, D)


def test_c_abi_refusals(lib):
    fake, null = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)
    h = _lib.Heads(1 << 20, 64, 64, 64)
    bad_h = _lib.Heads((1 << 20) + 2, 64, 64, 64)
    no_h = _lib.Heads(0, 64, 64, 64)
    sh = _lib.Shape(1, 4, 2, 8, 8, 64, _lib.BSA_BF16)

    def norm(shape=sh, q=h, w=fake, n_pos=8, eps=1e-6):
        return lib.bsa_qk_norm_rotation(q, h, shape, w, fake, 1, fake, fake, n_pos, null, 0, eps, 1, h, h, null)
    assert norm(q=no_h) == norm(q=bad_h) == norm(w=null) == norm(n_pos=7) == norm(eps=-1.0) == -1
    assert norm(eps=float("nan")) == -1
    assert norm(_lib.Shape(1, 4, 2, 8, 8, 96, 0)) == norm(_lib.Shape(1, 4, 2, 8, 8, 64, 7)) == -2
    assert norm(_lib.Shape(1, 4, 0, 8, 8, 64, 0)) == norm(_lib.Shape(1, 4, 2, 8, 9, 64, 0)) == -1
    assert norm(_lib.Shape(1, 4, 2, 0, 0, 64, 0)) == 0  # nothing to do: no launch
    assert lib.bsa_qk_norm_rotation_workspace_bytes(sh) > 0
    assert lib.bsa_qk_norm_rotation_backward(h, h, h, h, sh, fake, fake, 1, fake, fake, 8, null, 0, 1e-6, 1, h, h,
                                             fake, fake, fake, 8, null) == _lib.BSA_ERR_WORKSPACE
    assert lib.bsa_qk_norm_rotation_backward(h, h, h, h, sh, fake, fake, 1, fake, fake, 8, null, 0, 1e-6, 1, h, h,
                                             null, fake, fake, 1 << 20, null) == _lib.BSA_ERR_INVALID_ARG
    odd = ctypes.c_void_p((1 << 20) + 16)
    assert lib.bsa_qk_norm_rotation_backward(h, h, h, h, sh, fake, fake, 1, fake, fake, 8, null, 0, 1e-6, 1, h, h,
                                             fake, fake, odd, 1 << 20, null) == _lib.BSA_ERR_INVALID_ARG

    def tables(R=2, page=16, n_pages=9, T=4, stride=3, cu=fake):
        return lib.bsa_paged_block_tables(fake, fake, R, fake, 3, stride, fake, 2, T, page, n_pages, fake, fake,
                                          cu, fake, null)
    assert tables(page=24) == tables(page=8) == tables(page=512) == tables(R=4097) == -2
    assert tables(n_pages=1 << 27) == -2
    assert tables(R=-1) == tables(T=-1) == tables(stride=2) == tables(cu=null) == -1

    def attend(c=None, R=2, T=4, Hq=4, max_new=1, width=3, q=h, ws=fake, nbytes=1 << 40):
        return lib.bsa_paged_chunk_attention(q, c or _cache(), fake, width, width, fake, fake, R, T, Hq, max_new,
                                             null, 0, 0, 0.0, 1, h, ws, nbytes, null)
    assert attend(_cache(_lib.BSA_F32)) == attend(_cache(page=24)) == attend(_cache(D=96)) == -2
    assert attend(_cache(n=1 << 27)) == attend(R=4097) == attend(width=1 << 25) == -2
    assert attend(R=4096, width=1 << 23) == -2
    assert attend(_cache(stride=68)) == attend(_cache(k=0)) == attend(_cache(k=(1 << 20) + 8)) == -1
    assert attend(Hq=3) == attend(max_new=-1) == attend(q=bad_h) == attend(q=no_h) == -1
    assert attend(ws=null) == attend(nbytes=64) == _lib.BSA_ERR_WORKSPACE
    assert attend(ws=odd) == -1
    assert attend(T=0) == attend(R=0) == attend(max_new=0) == 0
    assert lib.bsa_paged_attention_workspace_bytes(_cache(), 2, 4, 4, 1, 3) > 0
    assert lib.bsa_paged_attention_workspace_bytes(_cache(D=96), 2, 4, 4, 1, 3) == 0

    def append(c=None, T=3, pos=fake, q=h):
        return lib.bsa_paged_qk_norm_append(q, h, h, T, 4, fake, fake, 1, fake, fake, 8, pos, fake, 1e-6, 1, h,
                                            c or _cache(), null)
    assert append(_cache(_lib.BSA_F32)) == -2 and append(pos=null) == append(q=bad_h) == append(T=-1) == -1
    assert append(T=0) == 0
