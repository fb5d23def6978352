"""GPU parity: per-head norm with rotation, forward and backward, vs the float64 oracle.

Tolerances are derived. u is half a step of the output type (torch.finfo.eps / 2), e = 2^-24.
Forward: the sum of squares, its root, three products and a difference are at most 20
roundings in fp32, relative to |y_a| + |y_b| of a pair; then one rounding of the output.
Backward: 40 such roundings on the terms r|g| and r^3 |x| mean|g x|, then the output's; a
weight gradient is a sum of N = B S H fp32 terms: at most (N + 40) e of their absolute sum.
"""

import numpy as np
import pytest
import torch

from oracle import norm_rotation as nr

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _bsa():
    import block_sparse_attention_tcgen05_b200 as bsa
    return bsa


def _u(dt):
    return torch.finfo(dt).eps / 2


def _tensor(g, B, H, S, D, dt, layout):
    x = torch.randn(B, H, S, D, generator=g, dtype=torch.float64) * 1.5
    x = x.to(dt).to(DEV)
    if layout == "tokens":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "fused":  # a slice with other heads behind it
        pad = torch.full((B, S, H + 3, D), float("nan"), dtype=dt, device=DEV)
        pad[:, :, 1:H + 1] = x.transpose(1, 2)
        return pad[:, :, 1:H + 1].transpose(1, 2)
    return x


def _inputs(B, Hq, Hkv, S, D, dt, layout, n_pos=None, seed=0, wdt=torch.float32):
    g = torch.Generator().manual_seed(seed)
    q, k = (_tensor(g, B, h, S, D, dt, layout) for h in (Hq, Hkv))
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(wdt).to(DEV) for _ in range(2))
    a = torch.rand(n_pos or S, D // 2, generator=g, dtype=torch.float64) * 20 - 10
    return q, k, qw, kw, a.cos().float().to(DEV), a.sin().float().to(DEV)


def _np(t):
    return t.double().cpu().numpy()


def _check_forward(got, x, w, cos, sin, eps, inter):
    xd, wd, c, s = _np(x), _np(w), _np(cos), _np(sin)
    ref = nr.norm_rotation(xd, wd, c, s, eps, inter)
    y = np.abs(xd / np.sqrt((xd * xd).mean(-1, keepdims=True) + eps) * wd)
    a, b = nr._pairs(y, inter)
    size = nr._unpair(a + b, a + b, inter)
    err = np.abs(_np(got) - ref)
    tol = _u(x.dtype) * (np.abs(ref) + 20 * E * size) + 20 * E * size + (6e-8 if x.dtype == torch.float16 else 0)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("D,inter", [(64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("B,Hq,Hkv,S,layout", [(1, 2, 2, 1, "heads"), (2, 6, 2, 37, "fused"),
                                               (1, 5, 5, 130, "tokens"), (3, 24, 8, 16, "heads")])
def test_forward(dt, D, inter, B, Hq, Hkv, S, layout):
    q, k, qw, kw, cos, sin = _inputs(B, Hq, Hkv, S, D, TYPES[dt], layout)
    qo, ko = _bsa().qk_norm_rotation(q, k, qw, kw, cos, sin, eps=1e-5, interleaved=inter)
    assert qo.is_contiguous() and ko.is_contiguous()
    _check_forward(qo, q, qw, cos, sin, 1e-5, inter)
    _check_forward(ko, k, kw, cos, sin, 1e-5, inter)


def test_weights_of_the_inputs_type_and_in_place():
    q, k, qw, kw, cos, sin = _inputs(2, 3, 1, 21, 128, torch.bfloat16, "fused", wdt=torch.bfloat16)
    bsa = _bsa()
    qo, ko = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin)
    _check_forward(qo, q, qw, cos, sin, 1e-6, True)
    qi, ki = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin, q_out=q, k_out=k)
    assert qi is q and torch.equal(q, qo) and torch.equal(k, ko)


def test_positions_padding_and_bad_positions():
    B, H, S, D = 2, 3, 9, 64
    q, k, qw, kw, cos, sin = _inputs(B, H, H, S, D, torch.float32, "tokens", n_pos=40)
    pos = torch.randint(0, 40, (B, S), dtype=torch.int32)
    pos[0, 4] = -1
    pos[1, 2] = 40
    pos[1, 3] = -7
    bsa = _bsa()
    bsa.device_status()
    qo = torch.full((B, H, S, D), 5.0, device=DEV)
    ko = torch.full((B, H, S, D), 5.0, device=DEV)
    bsa.qk_norm_rotation(q, k, qw, kw, cos, sin, positions=pos.to(DEV), q_out=qo, k_out=ko)
    assert bsa.device_status()[0] == -1  # BSA_ERR_INVALID_ARG, for the two outside the table
    for b in range(B):
        ok = (pos[b] >= 0) & (pos[b] < 40)
        p = pos[b][ok].long().to(DEV)
        for out, x, w in ((qo, q, qw), (ko, k, kw)):
            _check_forward(out[b][:, ok], x[b][:, ok], w, cos[p], sin[p], 1e-6, True)
            assert (out[b][:, ~ok] == 5.0).all()
    # padding alone is no error; skipped rows get zero gradients and do not count in the sums
    pos = torch.tensor([3, -1, 5, -1, 0, 1, 2, 39, -1], dtype=torch.int32)
    dq, dk = torch.ones_like(qo), torch.ones_like(ko)
    g = bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, cos, sin, positions=pos.to(DEV))
    assert bsa.device_status()[0] == 0
    assert (g[0][:, :, pos < 0] == 0).all() and (g[0][:, :, pos >= 0] != 0).any()
    live = pos >= 0
    sub = bsa.qk_norm_rotation_backward(dq[:, :, live].contiguous(), dk[:, :, live].contiguous(),
                                        q[:, :, live].contiguous(), k[:, :, live].contiguous(), qw, kw,
                                        cos, sin, positions=pos[live].to(DEV))
    assert torch.equal(sub[0], g[0][:, :, live])
    # the two sums of the same N terms in other orders: 2 (N + 40) e of the absolute sum
    N = B * H * int(live.sum())
    size = (q.abs() * 3 * qw.abs().max() * 4).sum()
    assert ((sub[2] - g[2]).abs() <= 2 * (N + 40) * E * size).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("D,inter", [(64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("B,Hq,Hkv,S,layout", [(1, 1, 1, 1, "heads"), (2, 6, 2, 37, "fused"),
                                               (1, 12, 4, 530, "tokens")])
def test_backward(dt, D, inter, B, Hq, Hkv, S, layout):
    q, k, qw, kw, cos, sin = _inputs(B, Hq, Hkv, S, D, TYPES[dt], layout, seed=3)
    g = torch.Generator().manual_seed(4)
    dq = _tensor(g, B, Hq, S, D, TYPES[dt], "heads")
    dk = _tensor(g, B, Hkv, S, D, TYPES[dt], "tokens")
    bsa = _bsa()
    got = bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, cos, sin, eps=1e-5, interleaved=inter)
    again = bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, cos, sin, eps=1e-5, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # sums in a fixed order
    for x, w, d, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        xd, wd, dd, c, s = _np(x), _np(w), _np(d), _np(cos), _np(sin)
        rx, rw = nr.norm_rotation_backward(dd, xd, wd, c, s, 1e-5, inter)
        r = 1 / np.sqrt((xd * xd).mean(-1, keepdims=True) + 1e-5)
        a, b = nr._pairs(np.abs(dd), inter)
        z = nr._unpair(a + b, a + b, inter)       # bounds |z|
        size = r * z * np.abs(wd) + r ** 3 * np.abs(xd) * (z * np.abs(wd * xd)).mean(-1, keepdims=True)
        u = _u(x.dtype)
        tol = u * np.abs(rx) + (1 + u) * 40 * E * size + (6e-8 if dt == "f16" else 0)
        err = np.abs(_np(dx) - rx)
        assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
        N = B * S * x.shape[1]
        tw = (N + 40) * E * (z * np.abs(xd) * r).reshape(-1, D).sum(0)
        assert (np.abs(_np(dw) - rw) <= tw).all()


def test_backward_against_differences_and_broadcast_gradients():
    """fp32 gradients against central differences of the float64 definition; an output
    gradient broadcast over heads and tokens (strides of 0) is read as its copy is."""
    B, H, S, D = 1, 3, 4, 64
    q, k, qw, kw, cos, sin = _inputs(B, H, 1, S, D, torch.float32, "heads", seed=5)
    g = torch.Generator().manual_seed(6)
    d = torch.randn(1, 1, 1, D, generator=g).to(DEV)
    dq, dk = d.expand(B, H, S, D), d.expand(B, 1, S, D)
    bsa = _bsa()
    got = bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, cos, sin)
    same = bsa.qk_norm_rotation_backward(dq.contiguous(), dk.contiguous(), q, k, qw, kw, cos, sin)
    assert all(torch.equal(a, b) for a, b in zip(got, same))
    rng = np.random.default_rng(7)
    x, w, c, s = _np(q), _np(qw), _np(cos), _np(sin)
    h = 1e-5
    for _ in range(4):
        ex, ew = rng.standard_normal(x.shape), rng.standard_normal(D)

        def loss(t):
            return (_np(dq) * nr.norm_rotation(x + t * ex, w + t * ew, c, s)).sum()
        num = (loss(h) - loss(-h)) / (2 * h)
        ana = (_np(got[0]) * ex).sum() + (_np(got[2]) * ew).sum()
        # each gradient entry is within 40 e of terms no larger than |d| |w| |x| r^3-sized sums:
        # 100 e times their absolute sum covers both, the difference's own error is ~1e-9
        size = (np.abs(_np(got[0]) * ex).sum() + np.abs(_np(got[2]) * ew).sum() +
                np.abs(ex).sum() * 8 * np.abs(_np(d)).max())
        assert abs(num - ana) <= 100 * E * size + 1e-7


def test_empty_and_graph_and_other_stream():
    bsa = _bsa()
    q, k, qw, kw, cos, sin = _inputs(1, 4, 2, 33, 128, torch.bfloat16, "fused")
    e = bsa.qk_norm_rotation(q[:, :, :0], k[:, :, :0], qw, kw, cos, sin)
    assert e[0].shape == (1, 4, 0, 128)
    none = bsa.qk_norm_rotation(q[:, :, :0], k[:, :, :0], qw, kw, cos[:0], sin[:0])
    assert none[1].shape == (1, 2, 0, 128)
    g = bsa.qk_norm_rotation_backward(e[0], e[1], q[:, :, :0], k[:, :, :0], qw, kw, cos, sin)
    assert (g[2] == 0).all() and (g[3] == 0).all() and g[0].shape == (1, 4, 0, 128)
    want = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin)
    wantg = bsa.qk_norm_rotation_backward(*want, q, k, qw, kw, cos, sin)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin)
            grads = bsa.qk_norm_rotation_backward(*out, q, k, qw, kw, cos, sin)
        for t in (*out, *grads):
            t.zero_()
        graph.replay()
        graph.replay()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wantg), (*out, *grads)))


def test_heads_from_a_fused_projection_go_into_block_sparse_attention():
    """As a layer runs it: q and k normed and rotated out of the projection's slices, then the
    block-sparse call on them, against the same arithmetic in float64 (attention tolerances of
    its own parity tests)."""
    import oracle
    bsa = _bsa()
    S, D, H, Hkv, C = 512, 64, 4, 2, 8
    g = torch.Generator().manual_seed(9)
    x = torch.randn(1, S, H + 2 * Hkv, D, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:].contiguous()
    _, _, qw, kw, cos, sin = _inputs(1, H, Hkv, S, D, torch.bfloat16, "heads")
    qo, ko = bsa.qk_norm_rotation(q, k, qw, kw, cos, sin)
    lab = (torch.arange(S) // 64).to(torch.int32)
    mask = torch.rand(C, C, generator=g) < 0.4
    mask |= torch.eye(C, dtype=torch.bool)
    out = bsa.centroid_compensated_attention(qo, ko, v, lab.to(DEV), lab.to(DEV), mask.to(DEV))
    rq, rk = (torch.tensor(nr.norm_rotation(_np(a), _np(w), _np(cos), _np(sin))).to(torch.bfloat16).double().numpy()
              for a, w in ((q, qw), (k, kw)))
    ref = oracle.centroid_compensated_attention(rq, rk, _np(v), lab.numpy(), lab.numpy(), mask.numpy())
    err = np.abs(_np(out) - ref)
    assert err.max() <= 2e-2 and np.linalg.norm(err) <= 5e-3 * np.linalg.norm(ref)
