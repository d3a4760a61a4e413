"""The target's side of a step on what only the device sees to be wrong, and on values that are not
finite: what is reported, what still is answered, and that nothing else changes."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")
if torch.cuda.is_available():
    from _target import Batch, gen, i32, new_cache, workspace

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEVICE_CHECK = 5


def noise(t, seed):
    """Random values in every element of t."""
    return t.copy_(torch.randn(t.shape, generator=gen(seed), device="cuda"))


# ------------------------------------------------------------------------- appending

STARTS = [
    # starts of 3 requests, and the rows (of request, place) that are certainly its own
    ([0, 3, 2, 9], {0: (0, 0), 1: (0, 1), 4: (2, 2), 8: (2, 6)}),
    ([0, 1 << 30, 2, 9], {}),
    ([5, 2, 7, 9], {7: (2, 0), 8: (2, 1)}),
    ([9, 5, 1, 3], {}),
    ([0, 3, -(1 << 31), 9], {}),
    ([0, 3, (1 << 31) - 1, 9], {0: (0, 0), 2: (0, 2)}),
]


@pytest.mark.parametrize("starts,own", STARTS, ids=[str(s[0]) for s in STARTS])
def test_append_of_starts_that_descend(starts, own):
    """A row whose request begins behind it counts as none: nothing is written in front of a request's
    tokens, nor for a request whose rows are refused."""
    batch = Batch([3, 7, 9], [20, 40, 5], 16, packed=True, N=9)
    rows = 16
    k, v = (noise(t, 60 + j) for j, t in enumerate(new_cache(batch, 2, 64, BF16, fill=0.0)))
    want_k, want_v = k.clone(), v.clone()
    x = torch.randn(rows, 8, 64, generator=gen(62), device="cuda").to(BF16)
    q, new_k, new_v = x[:, :4], x[:, 4:6], x[:, 6:]
    q_out = torch.full((rows, 4, 64), 5.0, dtype=BF16, device="cuda")
    ws = workspace()
    ds.cache_append(ds.PagedCache(k, v), new_k, new_v, batch.pages, batch.lens, ws, q=q, q_out=q_out, starts=i32(starts),
                    nodes=9)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    good = [b for b in range(3) if 0 <= starts[b] <= starts[b + 1] <= rows and starts[b + 1] - starts[b] <= 9]
    may = torch.zeros(rows, dtype=torch.bool, device="cuda")   # rows of a request that is none of the bad
    free_k = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    for b in good:
        may[starts[b]:starts[b + 1]] = True
        page, line = batch.place(b, [batch.lengths[b] + i for i in range(min(starts[b + 1] - starts[b], batch.counts[b]))])
        free_k[page, line] = True
    assert torch.equal(k[~free_k], want_k[~free_k]) and torch.equal(v[~free_k], want_v[~free_k])
    assert (q_out[~may] == 5.0).all()
    for row, (b, i) in own.items():
        page, line = batch.place(b, [batch.lengths[b] + i])
        assert torch.equal(k[page, line][0], new_k[row]) and torch.equal(v[page, line][0], new_v[row])
        assert torch.equal(q_out[row], q[row])
