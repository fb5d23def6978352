"""GPU parity of the paged-cache and head-norm calls at their edges, vs the oracle (tolerances
as derived in test_parity_paged.py)."""

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
