"""qk_norm_rotation under autograd: what it refuses (CPU), and its gradients (GPU) against the
explicit backward call, bit for bit, and against float64 differentiation of the definition."""

import numpy as np
import pytest
import torch

import block_sparse_attention_tcgen05_b200 as bsa

DEV = "cuda"


def _args(S=8, D=64, dt=torch.bfloat16, dev="cpu", B=1, Hq=4, Hkv=2, seed=0, wdt=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, Hq + Hkv, D, generator=g).to(dt).to(dev)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(wdt).to(dev) for _ in range(2)]
    a = torch.rand(S, D // 2, generator=g, dtype=torch.float64) * 9
    return x, *w, a.cos().float().to(dev), a.sin().float().to(dev)


def _split(x, Hq=4):
    x = x.transpose(1, 2)
    return x[:, :Hq], x[:, Hq:]


def test_refusals():
    x, qw, kw, c, s = _args()
    q, k = _split(x.requires_grad_())
    f = bsa.qk_norm_rotation
    for kwargs in ({"q_out": torch.empty(1, 4, 8, 64, dtype=x.dtype)}, {"k_out": k}):
        with pytest.raises(ValueError, match="written outside autograd"):
            f(q, k, qw, kw, c, s, **kwargs)
    with pytest.raises(ValueError, match="written outside autograd"):  # the output alone
        f(q.detach(), k.detach(), qw, kw, c, s, q_out=torch.empty(1, 4, 8, 64, dtype=x.dtype, requires_grad=True))
    with pytest.raises(ValueError, match="no gradient is computed for the rotation"):
        f(q, k, qw, kw, c.clone().requires_grad_(), s)
    # argument checks are those of the plain call
    with pytest.raises(ValueError, match="k: shape"):
        f(q, k[:, :, :7], qw, kw, c, s)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        f(q, k, qw, kw, c, s)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors only"):
        f(q, k, qw, kw, c, s, q_out=q)


def _definition(x, qw, kw, cos, sin, Hq, eps=1e-6):
    """Interleaved pairs, in the type of its arguments."""
    out = []
    for t, w in zip(_split(x, Hq), (qw, kw)):
        y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps) * w
        a, b = y[..., ::2], y[..., 1::2]
        out.append(torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dt,wdt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                    (torch.float32, torch.float32)])
@pytest.mark.parametrize("inter", [True, False])
def test_gradients_are_those_of_the_backward_call(dt, wdt, inter):
    x, qw, kw, c, s = _args(37, 64, dt, DEV, 2, wdt=wdt)
    pos = torch.arange(37, dtype=torch.int32, device=DEV)
    pos[5] = -1
    leaves = [t.clone().requires_grad_() for t in (x, qw, kw)]
    q, k = _split(leaves[0])
    qo, ko = bsa.qk_norm_rotation(q, k, *leaves[1:], c, s, positions=pos, eps=1e-5, interleaved=inter)
    assert qo.requires_grad and ko.requires_grad and qo.is_contiguous()
    plain = bsa.qk_norm_rotation(*_split(x), qw, kw, c, s, positions=pos, eps=1e-5, interleaved=inter)
    live = pos >= 0
    assert all(torch.equal(a[:, :, live], b[:, :, live]) for a, b in zip((qo, ko), plain))
    dq, dk = torch.randn_like(qo), torch.randn_like(ko)
    torch.autograd.backward((qo, ko), (dq, dk))
    want = bsa.qk_norm_rotation_backward(dq, dk, *_split(x), qw, kw, c, s, positions=pos, eps=1e-5, interleaved=inter)
    gq, gk = _split(leaves[0].grad)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])
    for leaf, w in zip(leaves[1:], want[2:]):
        assert leaf.grad.dtype == wdt and torch.equal(leaf.grad, w.to(wdt))


@pytest.mark.gpu
def test_gradients_of_every_layout_and_of_one_side_alone():
    """Broadcast gradients (of a sum), transposed ones, one output that nothing uses, weights
    alone, and tensors without a gradient."""
    x, qw, kw, c, s = _args(21, 64, torch.float32, DEV)
    q, k = (t.contiguous() for t in _split(x))

    def grads(loss, weights=(qw, kw)):
        leaves = [t.clone().requires_grad_() for t in (q, k, *weights)]
        loss(*bsa.qk_norm_rotation(*leaves, c, s)).backward()
        return [t.grad for t in leaves]

    def want(dq, dk):
        return bsa.qk_norm_rotation_backward(dq, dk, q, k, qw, kw, c, s)
    one, none = torch.ones_like(q), torch.zeros_like(k)
    m = torch.randn(4, 64, 21, device=DEV)
    for loss, dq in ((lambda a, b: a.sum(), one), (lambda a, b: (a[0].transpose(1, 2) * m).sum(), m.transpose(1, 2)[None]),
                     (lambda a, b: 2 * a[:, 1:3, 4:, 3:].sum(), None)):
        if dq is None:
            dq = torch.zeros_like(q)
            dq[:, 1:3, 4:, 3:] = 2
        assert all(torch.equal(a, b) for a, b in zip(grads(loss), want(dq.contiguous(), none)))
    w = [t.clone().requires_grad_() for t in (qw, kw)]
    qo, ko = bsa.qk_norm_rotation(q, k, *w, c, s)
    (qo.sum() + ko.sum()).backward()
    for a, b in zip(w, want(one, torch.ones_like(k))[2:]):
        assert torch.equal(a.grad, b)
    with torch.no_grad():
        qi = q.clone()
        assert not bsa.qk_norm_rotation(q, k, *w, c, s)[0].requires_grad
        assert bsa.qk_norm_rotation(qi, k, *w, c, s, q_out=qi)[0] is qi
    assert not bsa.qk_norm_rotation(q, k, qw, kw, c, s)[0].requires_grad
    leaf = q.clone().requires_grad_()
    g, = torch.autograd.grad(bsa.qk_norm_rotation(leaf, k, qw, kw, c, s)[0].square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


@pytest.mark.gpu
def test_a_training_step_through_attention():
    """A fused projection, its heads normed and rotated, dense attention and a loss, in fp32:
    gradients of the projection's weights and of the norms' against the same step in float64.
    Every fp32 operation is within 2^-24 of its terms; a gradient passes some 10 products over at
    most 384 terms: 2^-24 * 4000 of the gradients' largest entry bounds them with a wide margin."""
    B, S, D, Hq, Hkv, W = 1, 24, 64, 4, 2, 96
    g = torch.Generator().manual_seed(3)
    _, qw, kw, c, s = _args(S, D)
    h = torch.randn(B, S, W, generator=g)
    proj = torch.randn(W, (Hq + 2 * Hkv) * D, generator=g) / 10
    target = torch.randn(B, Hq, S, D, generator=g)

    def step(own, dev, dt):
        leaves = [t.to(dev, dt, copy=True).requires_grad_() for t in (proj, qw, kw)]
        x = (h.to(dev, dt) @ leaves[0]).view(B, S, Hq + 2 * Hkv, D)
        qk = x[:, :, :Hq + Hkv]
        cs = c.to(dev, dt), s.to(dev, dt)
        if own:
            q, k = bsa.qk_norm_rotation(*_split(qk, Hq), *leaves[1:], *cs)
        else:
            q, k = _definition(qk, *leaves[1:], *cs, Hq)
        v = x[:, :, Hq + Hkv:].transpose(1, 2)
        k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
        o = torch.softmax(q @ k.transpose(2, 3) / D ** 0.5, -1) @ v
        (o - target.to(dev, dt)).square().mean().backward()
        return [t.grad.double().cpu() for t in leaves]
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    got = step(True, DEV, torch.float32)
    torch.backends.cuda.matmul.allow_tf32 = old
    for a, b in zip(got, step(False, "cpu", torch.float64)):
        assert (a - b).abs().max() <= 2.0 ** -24 * 4000 * b.abs().max()


@pytest.mark.gpu
def test_a_captured_step_and_another_stream():
    x, qw, kw, c, s = _args(33, 128, torch.bfloat16, DEV)
    leaves = [t.clone().requires_grad_() for t in (*_split(x), qw, kw)]
    dq, dk = torch.randn(1, 4, 33, 128, device=DEV), torch.randn(1, 2, 33, 128, device=DEV)

    def step():
        return torch.autograd.grad(bsa.qk_norm_rotation(*leaves, c, s), leaves, (dq.to(x.dtype), dk.to(x.dtype)))
    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        other = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = step()
        graph.replay()
    st.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(want, other, got))
