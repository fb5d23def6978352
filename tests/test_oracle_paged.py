"""CPU pins of the oracle of the per-head norm with rotation and of the paged cache: closed
forms, gradients against differences, library attention, and hand-worked tables."""

import numpy as np
import pytest
import torch

from oracle import norm_rotation as nr
from oracle import paged


def _angles(S, D, rng):
    a = rng.uniform(-7, 7, (S, D // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rotation_is_a_scaled_complex_rotation(interleaved):
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((3, 5, 64)), np.ones(64)
    cos, sin = _angles(5, 64, rng)
    y = nr.norm_rotation(x, w, cos, sin, 0.0, interleaved)
    # rows keep their direction's length: root mean square 1
    assert np.allclose((y * y).mean(-1), 1.0, atol=1e-12)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) if interleaved else (x[..., :32] + 1j * x[..., 32:])
    z = z / np.sqrt((x * x).mean(-1, keepdims=True)) * (cos + 1j * sin)
    got = (y[..., 0::2] + 1j * y[..., 1::2]) if interleaved else (y[..., :32] + 1j * y[..., 32:])
    assert np.abs(got - z).max() < 1e-12
    # inner products of equal angle differences are equal: the rotation is relative
    q = nr.rotate(x[0], cos, sin, interleaved)
    back = nr.rotate(q, cos, -sin, interleaved)
    assert np.abs(back - x[0]).max() < 1e-12


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rotation_gradient_against_differences(interleaved):
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((2, 3, 64)), 1 + 0.2 * rng.standard_normal(64)
    cos, sin = _angles(3, 64, rng)
    d = rng.standard_normal(x.shape)
    dx, dw = nr.norm_rotation_backward(d, x, w, cos, sin, 1e-3, interleaved)

    def loss(x, w):
        return (d * nr.norm_rotation(x, w, cos, sin, 1e-3, interleaved)).sum()
    h = 1e-5
    for _ in range(5):
        ex, ew = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        num = (loss(x + h * ex, w) - loss(x - h * ex, w)) / (2 * h)
        assert abs(num - (dx * ex).sum()) < 1e-7 * (np.abs(dx * ex).sum() + 1)
        num = (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h)
        assert abs(num - (dw * ew).sum()) < 1e-7 * (np.abs(dw * ew).sum() + 1)


def test_block_tables_by_hand():
    # pages of 16: request 0 has 15 tokens in page 7 and takes 3 (one old page, one new);
    # request 1 takes nothing; request 2 starts; request 3 lacks pages
    table = np.full((4, 3), -1)
    table[0, 0] = 7
    slots, pos, cu, taken, t = paged.paged_block_tables([15, 32, 0, 0], [3, 0, 2, 17], table,
                                                        [5, 9, 2], 24, 16)
    assert slots[:5].tolist() == [7 * 16 + 15, 5 * 16, 5 * 16 + 1, 9 * 16, 9 * 16 + 1]
    assert slots[5:21].tolist() == [2 * 16 + i for i in range(16)] and slots[21] == -1
    assert pos[:6].tolist() == [15, 16, 17, 0, 1, 0] and cu.tolist() == [0, 3, 3, 5, 22]
    assert taken == 4 and slots[22:].tolist() == [-1, -1] == pos[22:].tolist()
    assert t.tolist() == [[7, 5, -1], [-1] * 3, [9, -1, -1], [2, -1, -1]]


@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_is_library_attention_on_the_gathered_keys(causal):
    rng = np.random.default_rng(2)
    Hq, Hkv, D, page = 4, 2, 64, 16
    ctx, new = [20, 0], [5, 3]
    kc, vc = rng.standard_normal((6, Hkv, page, D)), rng.standard_normal((6, Hkv, page, D))
    table = np.array([[4, 1], [3, -1]])
    q = rng.standard_normal((Hq, 8, D))
    out, _ = paged.paged_chunk_attention(q, kc, vc, table, [0, 5, 8], ctx, causal)
    for r, (t0, t1) in enumerate(((0, 5), (5, 8))):
        L = ctx[r] + new[r]
        k = kc[table[r][:-(-L // page)]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        v = vc[table[r][:-(-L // page)]].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        see = torch.ones(new[r], L, dtype=torch.bool).tril(ctx[r]) if causal else None
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[:, t0:t1]), torch.tensor(k).repeat_interleave(2, 0),
            torch.tensor(v).repeat_interleave(2, 0), attn_mask=see).numpy()
        assert np.abs(out[:, t0:t1] - ref).max() < 1e-12
    # a mask that keeps one page, and one that keeps none
    mask = np.zeros((2, Hkv, 2), bool)
    mask[0, 0, 1] = True
    out, _ = paged.paged_chunk_attention(q, kc, vc, table, [0, 5, 8], ctx, causal, mask)
    assert (out[2:] == 0).all() and (out[:2, 5:] == 0).all() and (out[:2, :5] != 0).any()
