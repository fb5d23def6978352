"""GPU parity: block tables, cache writes and attention over a paged cache vs the oracle.

Attention tolerance, derived: with u half a step of the cache's type, each weight is rounded
once (u of spread = sum_j w_j |v_j|) and the output once (u |out|). fp32: a product over D and
one over n keys, both at most 2^-23 a step, the logits' error acting on the weights through
the exponential (twice it, for the sum too) and 2^-21 for the exponentials: relative to the
spread (n + 2 D L + 8) 2^-23 with L the largest sum |scale q_d k_d|.
"""

import numpy as np
import pytest
import torch

from oracle import norm_rotation as nr
from oracle import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _bsa():
    import block_sparse_attention_tcgen05_b200 as bsa
    return bsa


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _np(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- block tables
def _table_case(rng, R, page, max_ctx, max_new, spare=0, width_extra=1):
    ctx = rng.integers(0, max_ctx + 1, R)
    new = rng.integers(0, max_new + 1, R)
    need = -(-(ctx + new) // page)
    order = rng.permutation(int(need.sum()) + 8)
    table = np.full((R, int(need.max(initial=0)) + width_extra), -1)
    at = 0
    for r in range(R):
        have = -(-int(ctx[r]) // page)
        table[r, :have] = order[at:at + have]
        at += have
    return ctx, new, table, order[at:len(order) - 8 + spare], len(order)


@pytest.mark.parametrize("R,page,max_ctx,max_new", [(1, 16, 5, 1), (1, 256, 0, 700), (7, 32, 100, 40),
                                                    (300, 64, 500, 33), (1030, 16, 40, 3)])
def test_block_tables(R, page, max_ctx, max_new):
    bsa = _bsa()
    ctx, new, table, free, n_pages = _table_case(np.random.default_rng(R), R, page, max_ctx, max_new)
    T = int(new.sum()) + 5
    want = paged.paged_block_tables(ctx, new, table, free, T, page)
    t = _i32(table)
    for _ in range(2):  # the same call again writes the same entries
        got = bsa.paged_block_tables(_i32(ctx), _i32(new), t, _i32(free), T, page, n_pages)
        for g, w in zip((*got[:3], t), (*want[:3], want[4])):
            assert (g.cpu().numpy() == w).all()
        assert got[3].item() == want[3]
    assert bsa.device_status()[0] == 0


def test_block_tables_without_enough_pages():
    bsa = _bsa()
    ctx, new, table, free, n_pages = _table_case(np.random.default_rng(5), 9, 16, 60, 60)
    need = len(free)
    free = free[:need - 4]
    want = paged.paged_block_tables(ctx, new, table, free, int(new.sum()), 16)
    t = _i32(table)
    got = bsa.paged_block_tables(_i32(ctx), _i32(new), t, _i32(free), int(new.sum()), 16, n_pages)
    assert got[3].item() == want[3] == need and (got[0].cpu().numpy() == want[0]).all()
    assert (t.cpu().numpy() == want[4]).all() and (want[0] == -1).any()
    assert bsa.device_status()[0] == 0  # a short pool is the caller's to see in `taken`


def test_block_tables_bad_contents():
    """Negative lengths, a table row too short, a page outside the cache, more tokens than
    the packed length: no entry out of bounds, an error in the device status."""
    bsa = _bsa()
    for ctx, new, T in (([-3, 4], [2, 3], 8), ([0, 40], [2, 30], 40), ([15, 0], [1, 1], 4), ([0, 0], [9, 9], 12),
                        ([2 ** 31 - 1, 5], [3, 2 ** 31 - 1], 16)):
        guard = _i32(np.full((4, 4), 77))
        guard[1:3, :3] = -1
        guard[1, 0] = 900
        table = guard[1:3, :3]
        got = bsa.paged_block_tables(_i32(ctx), _i32(new), table, _i32([1, 2, 3, 4, 5, 6]), T, 16, 8)
        assert bsa.device_status()[0] == -1
        s = got[0].cpu()
        assert ((s >= -1) & (s < 8 * 16)).all()
        assert (got[2].cpu() <= T).all() and (got[2].cpu() >= 0).all()
        assert (guard[0] == 77).all() and (guard[3] == 77).all() and (guard[:, 3] == 77).all()


def test_block_tables_empty():
    bsa = _bsa()
    e = _i32(np.zeros(0))
    s, p, cu, taken = bsa.paged_block_tables(e, e, _i32(np.zeros((0, 3))), e, 6, 16, 4)
    assert (s == -1).all() and (p == -1).all() and cu.tolist() == [0] and taken.item() == 0
    s, p, cu, taken = bsa.paged_block_tables(_i32([4]), _i32([0]), _i32([[2]]), e, 0, 16, 4)
    assert s.numel() == 0 and cu.tolist() == [0, 0] and taken.item() == 0


# ---------------------------------------------------------------- append
def _cache(g, n_pages, Hkv, page, D, dt, interleave=False):
    if interleave:  # keys and values in turn, page by page, in one tensor
        kv = torch.randn(n_pages, 2, Hkv, page, D, generator=g).to(dt).to(DEV)
        return kv[:, 0], kv[:, 1]
    return tuple(torch.randn(n_pages, Hkv, page, D, generator=g).to(dt).to(DEV) for _ in range(2))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("D,page,Hq,Hkv,T,inter", [(64, 16, 4, 2, 1, True), (128, 64, 6, 2, 45, False),
                                                   (64, 256, 5, 5, 200, False), (128, 32, 24, 8, 130, True)])
def test_append(dt, D, page, Hq, Hkv, T, inter):
    bsa = _bsa()
    g = torch.Generator().manual_seed(T)
    n_pages = T // page + 4
    kc, vc = _cache(g, n_pages, Hkv, page, D, TYPES[dt], interleave=T > 100)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(TYPES[dt]).to(DEV).transpose(0, 1)
    q, k, v = x[:Hq], x[Hq:Hq + Hkv], x[Hq + Hkv:]
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g).to(DEV) for _ in range(2))
    a = torch.rand(500, D // 2, generator=g) * 9
    cos, sin = a.cos().to(DEV), a.sin().to(DEV)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32).to(DEV)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32).to(DEV)
    if T > 10:
        slots[3] = -1
        pos[5] = -1
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.full((Hq, T, D), 3.0, dtype=TYPES[dt], device=DEV)
    bsa.paged_qk_norm_append(q, k, v, qw, kw, cos, sin, pos, slots, kc, vc, interleaved=inter, q_out=qo)
    assert bsa.device_status()[0] == 0
    # the same pass as qk_norm_rotation, bit for bit, at the slots; the rest as it was
    rq, rk = bsa.qk_norm_rotation(q[None], k[None], qw, kw, cos, sin, positions=pos, interleaved=inter,
                                  q_out=torch.full((1, Hq, T, D), 3.0, dtype=TYPES[dt], device=DEV))
    assert torch.equal(qo, rq[0])
    for t in range(T):
        s = int(slots[t])
        if s >= 0 and int(pos[t]) >= 0:
            k0[s // page, :, s % page] = rk[0][:, t]
            v0[s // page, :, s % page] = v[:, t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_slot_outside_the_cache():
    bsa = _bsa()
    g = torch.Generator().manual_seed(0)
    pool = torch.zeros(6, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    x = torch.randn(3, 3, 64, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.ones(64, device=DEV)
    cos, sin = torch.ones(4, 32, device=DEV), torch.zeros(4, 32, device=DEV)
    kc, vc = pool[1:3], pool[3:5]
    qo = bsa.paged_qk_norm_append(x[:1], x[1:2], x[2:], w, w, cos, sin, _i32([0, 1, 2]), _i32([32, -2, 5]), kc, vc)
    assert bsa.device_status()[0] == -1
    assert torch.isfinite(qo.float()).all()
    assert (pool[0] == 0).all() and (pool[5] == 0).all()
    assert (kc[0, 0, 5] != 0).all() and int((kc != 0).any(-1).sum()) == 1


# ---------------------------------------------------------------- attention
def _attention_case(seed, ctx, new, Hq, Hkv, D, page, dt, keep=None, gain=1.0, interleave=False, nan=True):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    n_pages = sum(need) + 3
    order = rng.permutation(n_pages)
    kc, vc = _cache(g, n_pages, Hkv, page, D, dt, interleave)
    width = max(need + [1])
    table = np.full((len(ctx), width), -1)
    at = 0
    mask = None if keep is None else rng.random((len(ctx), Hkv, width)) < keep
    for r, m in enumerate(need):
        table[r, :m] = order[at:at + m]
        at += m
        end = (ctx[r] + new[r]) % page
        if nan and end:
            kc[table[r, m - 1], :, end:] = float("nan")
            vc[table[r, m - 1], :, end:] = float("inf")
        if nan and mask is not None:  # what a page mask drops is never read into a result
            for h in range(Hkv):
                for j in range(m):
                    if not mask[r, h, j]:
                        kc[table[r, j], h] = float("nan")
                        vc[table[r, j], h] = float("nan")
    if nan:
        kc[order[at:]] = float("nan")
        vc[order[at:]] = float("nan")
    T = sum(new)
    q = (torch.randn(Hq, T + 3, D, generator=g) * gain).to(dt).to(DEV)
    cu = np.concatenate([[0], np.cumsum(new)])
    return q, kc, vc, table, cu, mask


def _check(out, q, kc, vc, table, cu, ctx, causal, mask, scale=None):
    kd, vd = np.nan_to_num(_np(kc), posinf=0), np.nan_to_num(_np(vc), posinf=0)
    ref, spread = paged.paged_chunk_attention(_np(q), kd, vd, table, cu, ctx, causal, mask, scale)
    D = q.shape[2]
    n = max(c + cu[i + 1] - cu[i] for i, c in enumerate(ctx))
    # sum |q_d k_d| <= |q| |k|
    L = np.linalg.norm(_np(q), axis=-1).max() * np.linalg.norm(kd, axis=-1).max() * (scale or D ** -0.5)
    u = torch.finfo(q.dtype).eps / 2
    tol = u * (spread + np.abs(ref)) * (1 + 2 * u) + (n + 2 * D * L + 8) * 2.0 ** -23 * spread + 1e-7
    T = cu[-1]
    err = np.abs(_np(out) - ref)[:, :T]
    assert np.isfinite(err).all()
    assert (err <= tol[:, :T]).all(), (err / tol[:, :T]).max()


def _run(ctx, new, Hq, Hkv, D, page, dt="bf16", causal=True, keep=None, seed=0, gain=1.0, max_new=None,
         scale=None, interleave=False, nan=True):
    bsa = _bsa()
    q, kc, vc, table, cu, mask = _attention_case(seed, ctx, new, Hq, Hkv, D, page, TYPES[dt], keep, gain,
                                                 interleave, nan)
    out = torch.full_like(q, 7.0)
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32(ctx), causal=causal, page_mask=m,
                              max_new=max(new) if max_new is None else max_new, scale=scale, out=out)
    assert bsa.device_status() == (0, 0)
    assert (out[:, cu[-1]:] == 7.0).all()  # rows behind the last request
    _check(out, q, kc, vc, table, cu, ctx, causal, mask, scale)
    return out, q, kc, vc, table, cu, mask


# single tokens and short runs: the token kernel
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f16", 128), ("f16", 64)])
@pytest.mark.parametrize("Hq,Hkv,page,ctx,new", [
    (3, 1, 16, [0], [1]),                       # the very first token
    (8, 2, 16, [15, 16, 17, 0, 200], [1] * 5),  # page borders
    (24, 8, 64, [700, 3, 64], [1] * 3),
    (5, 5, 256, [300, 511], [1, 1]),            # no shared heads, pages past a chunk
    (6, 2, 32, [40, 0, 333], [2, 5, 1]),        # up to 15 rows
    (16, 1, 32, [100, 31], [1, 1]),             # 16 rows
])
def test_tokens(dt, D, Hq, Hkv, page, ctx, new):
    _run(ctx, new, Hq, Hkv, D, page, dt)


@pytest.mark.parametrize("causal", [True, False])
def test_tokens_page_mask_and_empty_rows(causal):
    out, *_ , mask = _run([90, 5, 200, 31], [1, 2, 1, 1], 6, 3, 64, 16, "f16", causal, keep=0.3, seed=4)
    assert (_np(out)[:, 1:3] == 0).all() or mask[1].any()


def test_tokens_many_requests_with_empty_ones():
    rng = np.random.default_rng(0)
    ctx = rng.integers(0, 400, 70).tolist()
    new = rng.integers(0, 3, 70).tolist()
    _run(ctx, new, 4, 2, 64, 16, "bf16", True, seed=2)


def test_tokens_long_context_splits():
    """One request whose keys go over many CTAs, with a large logit range."""
    _run([9000], [1], 4, 2, 128, 64, "bf16", True, seed=3, gain=4.0)


# chunks: the tile kernel
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f16", 128), ("f16", 64)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,page,ctx,new", [
    (1, 1, 16, [0], [17]),
    (2, 1, 128, [128], [128]),        # tiles and chunks that end on their borders
    (3, 1, 64, [70], [90]),           # 270 rows: a second tile pair of 14 rows
    (2, 2, 256, [300], [130]),
    (1, 1, 32, [0], [300]),
])
def test_chunks(dt, D, causal, Hq, Hkv, page, ctx, new):
    _run(ctx, new, Hq, Hkv, D, page, dt, causal)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f16", 128), ("f16", 64)])
@pytest.mark.parametrize("ctx,new,causal", [([300], [40], True), ([0], [300], True), ([2300], [20], False)])
def test_chunks_whose_logits_rise(dt, D, ctx, new, causal):
    """Later keys whose logits are far above the first ones' (a hundred and more base-2 units in
    some rows, a little in others), rows that see only the first ones beside them."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(40, ctx, new, 2, 1, D, 64, TYPES[dt], None, 1.0, False, True)
    order = table[0]
    for j in range(3, len(order)):
        kc[order[j]] *= 1.0 + 2.0 * (j % 4)
    q[:, ::5] *= 4.0
    out = torch.full_like(q, 7.0)
    bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32(ctx), causal=causal, max_new=max(new), out=out)
    assert bsa.device_status() == (0, 0) and (out[:, cu[-1]:] == 7.0).all()
    _check(out, q, kc, vc, table, cu, ctx, causal, None)


@pytest.mark.parametrize("ctx,n", [(600, 40), (2300, 20), (600, 1)])
@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64)])
def test_first_keys_at_minus_infinity(dt, D, ctx, n):
    """The first 128 keys' logits are all -infinity (their weight is 0); the later ones are far
    above 0 in some rows and far below in others."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(45, [ctx], [n], 2, 1, D, 64, TYPES[dt], None, 1.0, False, True)
    used = table[0]
    q[1] *= 40.0
    kc[..., 0] = 0.0
    q[0, :, 0], q[1, :, 0] = 60.0, 0.5
    kc[used[2:], :, :, 0] = torch.where(torch.isnan(kc[used[2:], :, :, 1]), float("nan"), -40.0).to(kc.dtype)
    kc[used[:2], :, :, 0] = float("-inf")
    out = bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32([ctx]), causal=True, max_new=n)
    assert bsa.device_status() == (0, 0)
    mask = np.ones((1, 1, len(used)), dtype=bool)
    mask[..., :2] = False
    clean = kc.clone()
    clean[used[:2]] = 0.0
    _check(out, q, clean, vc, table, cu, [ctx], True, mask)


@pytest.mark.parametrize("ctx,n", [([600, 30], [40, 3]), ([9000], [1]), ([2300], [20])])
def test_output_in_place_of_the_queries(ctx, n):
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(46, ctx, n, 4, 2, 128, 16, torch.bfloat16)
    args = (kc, vc, _i32(table), _i32(cu), _i32(ctx))
    want = bsa.paged_chunk_attention(q, *args, max_new=max(n))
    got = bsa.paged_chunk_attention(q, *args, max_new=max(n), out=q)
    assert got is q or got.data_ptr() == q.data_ptr()
    assert torch.equal(got[:, :cu[-1]], want[:, :cu[-1]])


@pytest.mark.parametrize("R", [3, 40])
def test_a_wide_block_table_changes_nothing(R):
    """A table much wider than the requests (the order of the work depends on its reach)."""
    bsa = _bsa()
    rng = np.random.default_rng(47)
    ctx, new = list(rng.integers(0, 2300, R)), list(rng.integers(0, 90, R))
    ctx[0], new[0] = 2300, 300
    q, kc, vc, table, cu, _ = _attention_case(47, ctx, new, 4, 2, 64, 32, torch.float16)
    wide = np.full((R, 16384), -1)
    wide[:, :table.shape[1]] = table
    got = [bsa.paged_chunk_attention(q, kc, vc, _i32(t), _i32(cu), _i32(ctx), max_new=300)[:, :cu[-1]]
           for t in (table, wide)]
    assert bsa.device_status() == (0, 0) and torch.equal(*got)
    _check(got[1], q[:, :cu[-1]], kc, vc, table, cu, ctx, True, None)


def test_chunks_split_keys():
    _run([2500], [20], 2, 1, 128, 64, "bf16", True, seed=5, gain=3.0)
    _run([4200], [9], 2, 1, 64, 16, "f16", False, seed=6)


@pytest.mark.parametrize("page,keep", [(16, 0.3), (32, 0.05), (128, 0.5), (256, 0.5)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_page_mask(page, keep, causal):
    _run([300, 0, 77], [40, 33, 129], 4, 2, 64, page, "bf16", causal, keep=keep, seed=page)


def test_mixed_batch_with_empty_requests():
    _run([33, 0, 500, 10, 64, 0], [1, 70, 0, 18, 2, 1], 6, 2, 128, 32, "bf16", True, seed=8)
    _run([33, 0, 500, 10, 64, 0], [1, 70, 0, 18, 2, 1], 6, 2, 64, 16, "f16", False, keep=0.5, seed=9)


def test_interleaved_cache_scale_and_default_bound():
    out, q, kc, vc, table, cu, _ = _run([50], [40], 4, 2, 128, 16, scale=0.05, interleave=True, nan=False)
    bsa = _bsa()
    # token-major q and out, bound left out
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    ot = torch.empty(q.shape[1], 4, 128, dtype=q.dtype, device=DEV).transpose(0, 1)
    bsa.paged_chunk_attention(qt[:, :40], kc, vc, _i32(table), _i32(cu), _i32([50]), scale=0.05, out=ot[:, :40])
    assert torch.equal(ot[:, :40], out[:, :40])


def test_broadcast_masks_and_shared_pages():
    """One mask row for all requests and heads; two requests that share their context pages."""
    bsa = _bsa()
    g = torch.Generator().manual_seed(11)
    kc, vc = _cache(g, 8, 2, 32, 64, torch.bfloat16)
    q = torch.randn(4, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    table, cu, ctx = np.array([[5, 2, 7], [5, 2, 1]]), np.array([0, 1, 2]), [70, 64]
    mask = np.array([1, 0, 1], bool)
    out = bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32(ctx), max_new=1,
                                    page_mask=torch.from_numpy(mask).to(DEV)[None])
    _check(out, q, kc, vc, table, cu, ctx, True, np.broadcast_to(mask, (2, 2, 3)))


def test_bad_device_contents_stay_in_bounds():
    """A page outside the cache, lengths past the table, tokens past the packed length, more
    new tokens than the bound: recorded, and nothing outside is read or written."""
    bsa = _bsa()
    g = torch.Generator().manual_seed(12)
    kc, vc = _cache(g, 4, 1, 16, 64, torch.bfloat16)
    for T, max_new, cu, ctx, table in (
            (1, 1, [0, 1], [20], [[1, 99]]), (40, 40, [0, 40], [0], [[1, -5, 2]]),
            (1, 1, [0, 1], [4000], [[1, 2]]), (40, 40, [0, 40], [-9], [[0, 1, 2]]),
            (2, 1, [0, 2], [3], [[1, 2]]), (40, 40, [7, 900], [3], [[1, 2, 3]]), (40, 40, [30, 2], [3], [[1, 2, 3]]),
            (1, 1, [0, 1], [2 ** 31 - 1], [[1, 2]])):
        q = torch.randn(24, T, 64, generator=g).to(torch.bfloat16).to(DEV)
        guard = torch.full((26, T, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32(ctx), max_new=max_new, out=guard[1:25])
        assert bsa.device_status()[0] == -1, (T, cu, ctx)
        assert (guard[0] == 9).all() and (guard[25] == 9).all() and torch.isfinite(guard.float()).all()


def test_an_invalid_page_counts_as_masked():
    bsa = _bsa()
    g = torch.Generator().manual_seed(13)
    kc, vc = _cache(g, 6, 2, 16, 64, torch.bfloat16)
    for n in (1, 30):
        q = torch.randn(2, n, 64, generator=g).to(torch.bfloat16).to(DEV)
        ctx, cu = [40], np.array([0, n])
        table = np.array([[3, 1, 4, 0, 5]])
        bad = table.copy()
        bad[0, 1] = 6
        out = bsa.paged_chunk_attention(q, kc, vc, _i32(bad), _i32(cu), _i32(ctx), max_new=n)
        assert bsa.device_status()[0] == -1
        mask = np.ones((1, 2, 5), bool)
        mask[0, :, 1] = False
        _check(out, q, kc, vc, table, cu, ctx, True, mask)


@pytest.mark.parametrize("n,ctx", [(1, 40), (1, 3000), (40, 100), (20, 2500)])
def test_nan_and_infinite_queries_give_nan_in_their_rows_alone(n, ctx):
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(50, [ctx], [n], 4, 2, 64, 16, torch.bfloat16)
    want = bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32([ctx]), max_new=n)
    q[1, 0, 3] = float("nan")
    q[2, n - 1] = float("inf")
    out = bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32([ctx]), max_new=n)
    assert torch.isnan(out[1, 0]).all() and torch.isnan(out[2, n - 1]).all()
    ok = torch.ones(4, n, dtype=torch.bool)
    ok[1, 0] = ok[2, n - 1] = False
    assert torch.equal(out[:, :n][ok], want[:, :n][ok])


def test_a_cache_past_32_bits_of_elements():
    """Pages whose elements lie past 2^31 and 2^32 bytes into the pool, written and read by every
    kernel."""
    bsa = _bsa()
    Hkv, page, D = 4, 64, 128
    n_pages = (1 << 31) // (Hkv * page * D) + 40  # 4.3 GB
    pool = torch.empty(n_pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    values = torch.empty_like(pool)
    g = torch.Generator().manual_seed(51)
    pages = [n_pages - 1, 2, n_pages - 7, n_pages - 2, n_pages // 2 + 1]
    small = torch.randn(5, Hkv, page, D, generator=g).to(torch.bfloat16).to(DEV)
    for i, p in enumerate(pages):
        pool[p] = small[i]
    for n in (1, 50):
        ctx = [5 * page - n]
        q = torch.randn(8, n, D, generator=g).to(torch.bfloat16).to(DEV)
        args = (_i32([0, n]), _i32(ctx))
        far = bsa.paged_chunk_attention(q, pool, pool, _i32([pages]), *args, max_new=n)
        near = bsa.paged_chunk_attention(q, small, small, _i32([[0, 1, 2, 3, 4]]), *args, max_new=n)
        assert torch.equal(far, near)
    x = torch.randn(4, 3 * 4, D, generator=g).to(torch.bfloat16).to(DEV)
    w, cos, sin = torch.ones(D, device=DEV), torch.ones(9, 64, device=DEV), torch.zeros(9, 64, device=DEV)
    slots = [pages[0] * page + 5, pages[2] * page, 7]
    bsa.paged_qk_norm_append(x[:, :3], x[:, 3:6], x[:, 6:9], w, w, cos, sin, _i32([0, 1, 2]), _i32(slots), pool, values)
    _, rk = bsa.qk_norm_rotation(x[None, :, :3], x[None, :, 3:6], w, w, cos, sin)
    for t, (p, row) in enumerate(((pages[0], 5), (pages[2], 0), (0, 7))):
        assert torch.equal(pool[p, :, row], rk[0, :, t]) and torch.equal(values[p, :, row], x[:, 6 + t])
    assert bsa.device_status()[0] == 0


def test_empty_calls():
    bsa = _bsa()
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    e = torch.empty(3, 0, 64, dtype=torch.bfloat16, device=DEV)
    assert bsa.paged_chunk_attention(e, kc, kc, _i32([[0]]), _i32([0, 0]), _i32([5])).shape == (3, 0, 64)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 2.0)
    bsa.paged_chunk_attention(q, kc, kc, _i32(np.zeros((0, 4))), _i32([0]), _i32(np.zeros(0)), out=out)
    bsa.paged_chunk_attention(q, kc, kc, _i32([[0, 1]]), _i32([0, 0]), _i32([5]), out=out)
    assert bsa.device_status()[0] == 0 and (out == 2.0).all()


def test_graph_two_calls_and_streams():
    """Two calls in one captured graph, replayed over changed inputs, and the same calls on
    two streams at once."""
    bsa = _bsa()
    a = _attention_case(20, [700, 5], [1, 1], 6, 2, 64, 16, torch.bfloat16)
    b = _attention_case(21, [900], [60], 6, 2, 64, 32, torch.bfloat16)

    def call(c, ctx, n):
        q, kc, vc, table, cu, _ = c
        return q, kc, vc, _i32(table), _i32(cu), _i32(ctx), n
    ca, cb = call(a, [700, 5], 1), call(b, [900], 60)

    def run(c):
        return bsa.paged_chunk_attention(*c[:6], max_new=c[6])
    run(ca), run(cb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa, ob = run(ca), run(cb)
    ca[0].mul_(-0.5)
    cb[0].mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa[:, :2], run(ca)[:, :2]) and torch.equal(ob[:, :60], run(cb)[:, :60])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            outs.append((run(ca), oa, 2))
        with torch.cuda.stream(s2):
            outs.append((run(cb), ob, 60))
    torch.cuda.synchronize()
    assert all(torch.equal(x[:, :n], y[:, :n]) for x, y, n in outs)


def test_a_video_generated_chunk_by_chunk():
    """The operators together, as a generator runs them: three steps of ragged chunks, each
    with its tables, its keys normed, rotated and appended, and its attention; against dense
    arithmetic on each request's whole sequence."""
    bsa = _bsa()
    g = torch.Generator().manual_seed(30)
    R, Hq, Hkv, D, page, n_pages, dt = 3, 6, 2, 64, 16, 40, torch.bfloat16
    kc, vc = (torch.full((n_pages, Hkv, page, D), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    table = _i32(np.full((R, 12), -1))
    free = torch.randperm(n_pages, generator=g).to(torch.int32).to(DEV)
    a = torch.rand(200, D // 2, generator=g) * 6
    cos, sin = a.cos().to(DEV), a.sin().to(DEV)
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g).to(DEV) for _ in range(2))
    ctx = np.zeros(R, int)
    past = [np.zeros((2, Hkv, 0, D)) for _ in range(R)]
    for new in ([30, 1, 17], [1, 1, 1], [5, 40, 0]):
        T = sum(new) + 2
        slots, pos, cu, taken = bsa.paged_block_tables(_i32(ctx), _i32(new), table, free, T, page, n_pages)
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dt).to(DEV).transpose(0, 1)
        q, k, v = x[:Hq], x[Hq:Hq + Hkv], x[Hq + Hkv:]
        qo = bsa.paged_qk_norm_append(q, k, v, qw, kw, cos, sin, pos, slots, kc, vc,
                                      q_out=torch.zeros(Hq, T, D, dtype=dt, device=DEV))
        out = bsa.paged_chunk_attention(qo, kc, vc, table, cu, _i32(ctx), max_new=max(new))
        assert bsa.device_status()[0] == 0
        free = free[int(taken):]
        cun = cu.cpu().numpy()
        for r in range(R):
            s = slice(cun[r], cun[r + 1])
            p = np.arange(ctx[r], ctx[r] + new[r])
            rk = nr.norm_rotation(_np(k[:, s]), _np(kw), _np(cos)[p], _np(sin)[p])
            rk = torch.tensor(rk).to(dt).double().numpy()
            past[r] = np.concatenate([past[r], np.stack([rk, _np(v[:, s])])], 2)
            K, V = past[r]
            for h in range(Hq):
                for i in range(new[r]):
                    lim = ctx[r] + i + 1
                    lg = K[h // 3, :lim] @ _np(qo[h, cun[r] + i]) / 8
                    w = np.exp(lg - lg.max())
                    w /= w.sum()
                    err = np.abs(_np(out[h, cun[r] + i]) - w @ V[h // 3, :lim])
                    # u of spread and of |out| for the weights and the output, and a half
                    # step of each key (u sum |q_d k_d| scale <= 2^-8 * 8, on both sums)
                    tol = 2.0 ** -8 * (1 + 2 * 8) * (w @ np.abs(V[h // 3, :lim])) + 2.0 ** -8 * np.abs(w @ V[h // 3, :lim])
                    assert (err <= tol + 1e-6).all()
        ctx += np.array(new)
