"""GPU parity of the paged-cache and head-norm calls at their edges, vs the oracle (tolerances
as derived in test_parity_paged.py)."""

import ctypes
import threading

import numpy as np
import pytest
import torch

from test_parity_paged import DEV, _attention_case, _bsa, _check, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,keep", [(128, 64, None), (64, 16, None), (64, 32, 0.3)])
def test_few_chunks_whose_halves_differ(D, page, keep):
    """Requests of one to three chunks of 128 keys, logits of tens of base-2 units that differ
    between a chunk's halves: the halves of a row agree on its reference in every one of many
    runs (each half ends its part of such a short pass at a time of its own)."""
    bsa = _bsa()
    rng = np.random.default_rng(60)
    ctx, new = rng.integers(20, 300, 48).tolist(), rng.integers(9, 60, 48).tolist()
    q, kc, vc, table, cu, mask = _attention_case(60, ctx, new, 4, 2, D, page, torch.bfloat16, keep, 1.0)
    kc *= 4.0  # logits of some +-15 base-2 units at the rows' maxima
    kc[::2] *= 0.25
    args = (q, kc, vc, _i32(table), _i32(cu), _i32(ctx))
    m = None if mask is None else torch.from_numpy(mask).to(DEV)

    def run():
        return bsa.paged_chunk_attention(*args, causal=False, max_new=max(new), page_mask=m)[:, :cu[-1]]
    first = run()
    assert bsa.device_status() == (0, 0)
    _check(first, q[:, :cu[-1]], kc, vc, table, cu, ctx, False, mask)
    again = [run() for _ in range(200)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, x) for x in again)


@pytest.mark.parametrize("new,want", [([2, 0, 1], -1), ([0, 0, 0], 0)])
@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.float16, 64)])
def test_a_block_table_without_columns(dt, D, new, want):
    """No key is left for any token: zeros, and an error for each request that has tokens."""
    bsa = _bsa()
    kc = torch.full((2, 2, 16, D), float("nan"), dtype=dt, device=DEV)
    q = torch.ones(6, 5, D, dtype=dt, device=DEV)
    cu = np.concatenate([[0], np.cumsum(new)])
    for layout in ("heads", "tokens"):
        out = torch.full((6, 5, D) if layout == "heads" else (5, 6, D), 7.0, dtype=dt, device=DEV)
        out = out if layout == "heads" else out.transpose(0, 1)
        bsa.paged_chunk_attention(q, kc, kc, _i32(np.zeros((3, 0))), _i32(cu), _i32([0, 4, 0]), out=out)
        assert bsa.device_status()[0] == want
        assert (out[:, :cu[-1]] == 0).all() and (out[:, cu[-1]:] == 7.0).all()
    mask = torch.ones(3, 2, 0, dtype=torch.bool, device=DEV)
    out = bsa.paged_chunk_attention(q, kc, kc, _i32(np.zeros((3, 0))), _i32([-3, 2, 900, 1 << 30]), _i32([0] * 3),
                                    page_mask=mask)
    assert bsa.device_status()[0] == -1 and (out == 0).all()


def test_a_bound_of_no_new_tokens():
    """max_new = 0: a request of one token gets its row, one of more is recorded, and without
    tokens nothing is written."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(61, [40, 7], [1, 1], 4, 2, 64, 16, torch.bfloat16)
    args = (q, kc, vc, _i32(table))
    ws = torch.empty(bsa.paged_attention_workspace_bytes(q, kc, _i32(table), 0), dtype=torch.uint8, device=DEV)
    got = bsa.paged_chunk_attention(*args, _i32(cu), _i32([40, 7]), max_new=0, workspace=ws)
    want = bsa.paged_chunk_attention(*args, _i32(cu), _i32([40, 7]), max_new=1)
    assert bsa.device_status()[0] == 0 and torch.equal(got[:, :2], want[:, :2])
    bsa.paged_chunk_attention(*args, _i32([0, 1, 3]), _i32([40, 6]), max_new=0)
    assert bsa.device_status()[0] == -1
    out = torch.full_like(q, 7.0)
    bsa.paged_chunk_attention(*args, _i32([0, 0, 0]), _i32([40, 6]), max_new=0, out=out)
    assert bsa.device_status()[0] == 0 and (out == 7.0).all()


def test_threads_with_thousands_of_requests():
    """Host threads whose calls have different numbers of requests (and so of shared memory) at
    the same time, each on a stream of its own and straight into the C entry point, so that no
    lock of the interpreter orders them: every call is accepted and right."""
    bsa = _bsa()
    from block_sparse_attention_tcgen05_b200 import _lib
    lib = _lib.load()
    g = torch.Generator().manual_seed(62)
    kc = torch.randn(40, 1, 16, 64, generator=g).to(torch.bfloat16).to(DEV)
    cache = _lib.PagedCache(kc.data_ptr(), kc.data_ptr(), 40, 16, 1, 64, _lib.BSA_BF16, 1024, 1024, 64, 1024, 1024, 64)

    def case(R):
        rng = np.random.default_rng(R)
        q = torch.randn(1, R, 64, generator=g).to(torch.bfloat16).to(DEV)
        return q, _i32(rng.integers(0, 40, (R, 5))), _i32(np.arange(R + 1)), _i32(rng.integers(0, 79, R))
    cases = [case(R) for R in (4096, 2100, 4000, 2300)]
    want = [bsa.paged_chunk_attention(c[0], kc, kc, *c[1:], max_new=1) for c in cases]
    outs = [torch.zeros_like(w) for w in want]
    spaces = [torch.empty(bsa.paged_attention_workspace_bytes(c[0], kc, c[1], 1), dtype=torch.uint8, device=DEV)
              for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    refused = []

    def work(i):
        q, table, cu, ctx = cases[i]
        R = q.shape[1]
        heads, to = (_lib.Heads(t.data_ptr(), 0, R * 64, 64) for t in (q, outs[i]))
        vp = ctypes.c_void_p
        args = (heads, cache, vp(table.data_ptr()), 5, 5, vp(cu.data_ptr()), vp(ctx.data_ptr()), R, R, 1, 1, vp(0), 0,
                0, 0.0, 1, to, vp(spaces[i].data_ptr()), spaces[i].numel(), vp(streams[i].cuda_stream))
        for _ in range(2000):
            st = lib.bsa_paged_chunk_attention(*args)
            if st:
                refused.append((R, st))
                return
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    q, table, cu, ctx = cases[1]
    _check(want[1], q, kc, kc, table.cpu().numpy(), cu.cpu().numpy(), ctx.cpu().numpy(), True, None)
    assert bsa.device_status()[0] == 0


@pytest.mark.parametrize("ctx,n", [(600, 40), (2300, 20), (100, 60), (600, 1)])
@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.float16, 64)])
def test_first_keys_far_below(ctx, n, dt, D):
    """The first 128 keys' logits are finite and so far below the later ones (2^29 base-2 units in
    fp16, 2^99 in bf16) that a difference from them keeps nothing of a later logit; those reach
    from some 30 to above 100 units."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(63, [ctx], [n], 2, 1, D, 64, dt)
    used = table[0]
    far = 65504.0 if dt == torch.float16 else 1e15
    q[0] *= 8.0
    q[1] *= 30.0
    q[..., 0] = far
    kc[..., 0] = 0.0
    kc[used[:2], :, :, 0] = -far
    rest = kc[used[-1], :, (ctx + n) % 64:] if (ctx + n) % 64 else kc[used[-1], :, :0]
    rest.fill_(float("nan"))
    out = bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32([ctx]), causal=True, max_new=n)
    assert bsa.device_status() == (0, 0)
    if ctx < 128:  # rows that see only such keys have a softmax of differences past 2^20: a mean
        seen = vc[used[:2], 0].reshape(-1, D)[:ctx + 1].float()
        assert torch.isfinite(out[:, :n]).all()
        assert (out[:, 0] <= seen.amax(0)).all() and (out[:, 0] >= seen.amin(0)).all()
        return
    mask = np.ones((1, 1, len(used)), dtype=bool)
    mask[..., :2] = False
    clean, qc = kc.clone(), q.clone()
    clean[used[:2]] = 0.0
    qc[..., 0] = 0.0
    _check(out, qc, clean, vc, table, cu, [ctx], True, mask)


@pytest.mark.parametrize("ctx,n", [(600, 40), (2300, 20), (90, 30), (600, 1)])
@pytest.mark.parametrize("dt,D,sign", [(torch.bfloat16, 128, 1), (torch.bfloat16, 64, -1), (torch.float16, 64, 1),
                                       (torch.float16, 128, -1)])
def test_logits_past_the_weights_range(ctx, n, dt, D, sign):
    """All logits of a row have one size, up to 2^30 base-2 units in fp16 and 2^60 in bf16, where one
    rounding of a logit is more than the weights' range: equal logits give the mean of the
    values, a few larger ones theirs."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(64, [ctx], [n], 3, 1, D, 64, dt)
    live = ~torch.isnan(kc[..., :1])
    top = 65504.0 if dt == torch.float16 else 2.0 ** 30
    q.zero_()
    q[..., 0] = sign * top * (0.5 + 0.5 * torch.rand(q.shape[:2], generator=torch.Generator().manual_seed(65))).to(DEV)
    kc.copy_(torch.where(live, torch.zeros_like(kc), kc))
    kc[..., 0] = torch.where(live[..., 0], torch.full_like(kc[..., 0], top / 2), kc[..., 0])
    args = (kc, vc, _i32(table), _i32(cu), _i32([ctx]))
    out = bsa.paged_chunk_attention(q, *args, causal=True, max_new=n)
    assert bsa.device_status() == (0, 0)
    _check(out, torch.zeros_like(q), torch.zeros_like(kc), vc, table, cu, [ctx], True, None)
    # one key of twice the size, or half of it where the sign asks for that
    used = table[0]
    kc[used[1], :, 5, 0] = top if sign > 0 else top / 4
    out = bsa.paged_chunk_attention(q, *args, causal=True, max_new=n)
    want = vc[used[1], 0, 5]
    if ctx >= 70:
        assert torch.equal(out[:, :n], want.expand(3, n, D))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ctx,new", [([90, 5, 200, 31], [1, 2, 1, 1]), ([90, 5, 1900, 31, 3], [20, 30, 90, 17, 60]),
                                     ([300, 0, 40], [40, 1, 9])])
def test_heads_without_a_page_get_exact_zeros(causal, ctx, new):
    """Every (request, KV head) whose mask keeps none of its pages, among others that keep some:
    rows of zeros, whatever stood there, in both kernels."""
    bsa = _bsa()
    q, kc, vc, table, cu, mask = _attention_case(66, ctx, new, 6, 3, 64, 16, torch.float16, 0.5)
    rng = np.random.default_rng(67)
    need = [-(-(c + n) // 16) for c, n in zip(ctx, new)]
    empty = rng.random((len(ctx), 3)) < 0.4
    empty[0] = [False, True, False]
    for r, h in np.argwhere(empty):
        mask[r, h, :need[r]] = False
        for j in range(need[r]):
            kc[table[r, j], h] = float("nan")
            vc[table[r, j], h] = float("nan")
    out = torch.full_like(q, 7.0)
    bsa.paged_chunk_attention(q, kc, vc, _i32(table), _i32(cu), _i32(ctx), causal=causal, max_new=max(new),
                              page_mask=torch.from_numpy(mask).to(DEV), out=out)
    assert bsa.device_status() == (0, 0) and (out[:, cu[-1]:] == 7.0).all()
    none = [(r, h) for r in range(len(ctx)) for h in range(3) if not mask[r, h, :need[r]].any()]
    assert len(none) >= empty.sum() > 0 and len(none) < 3 * len(ctx)
    for r, h in none:
        assert (out[2 * h:2 * h + 2, cu[r]:cu[r + 1]] == 0).all()
    _check(out, q, kc, vc, table, cu, ctx, causal, mask)


@pytest.mark.parametrize("n", [1, 40])
def test_a_cache_laid_out_token_by_token(n):
    """Pages whose rows hold all heads of a token (a row's stride above a head's), of a wider
    buffer: the same bits as of the cache laid out by heads."""
    bsa = _bsa()
    q, kc, vc, table, cu, _ = _attention_case(68, [300, 77], [n, n], 6, 3, 64, 32, torch.bfloat16)
    wide = torch.full((kc.shape[0], 32, 2, 4, 64), float("nan"), dtype=kc.dtype, device=DEV)
    wide[:, :, 0, :3], wide[:, :, 1, :3] = kc.transpose(1, 2), vc.transpose(1, 2)
    k2, v2 = (wide[:, :, i, :3].transpose(1, 2) for i in range(2))
    args = (_i32(table), _i32(cu), _i32([300, 77]))
    want = bsa.paged_chunk_attention(q, kc, vc, *args, max_new=n)
    got = bsa.paged_chunk_attention(q, k2, v2, *args, max_new=n)
    assert bsa.device_status() == (0, 0) and torch.equal(got[:, :2 * n], want[:, :2 * n])
    _check(got, q, kc, vc, table, cu, [300, 77], True, None)
