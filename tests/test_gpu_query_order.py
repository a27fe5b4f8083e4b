"""The attention kernels' waits and stores in order: the same call gives the
same bits while other work delays its copies, and rows that are summed again
key by key end with those sums."""
import math

import pytest
import torch

from query_cases import Paged
from test_gpu_query import make, pkg, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_decode_repeats_itself_beside_copies(pkg, D):  # noqa: F811
    """Units of 0 to 5 tiles whose last ones are a few keys, so that the last
    copies overtake the ones before, while another stream keeps the memory
    busy."""
    mem = [(131 * r) % 600 for r in range(60)]
    c = Paged(200 + D, D, 4, 4, 16, [1] * len(mem), mem)
    big = torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    busy = torch.cuda.Stream()
    with make(pkg, D, 4) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        ref, _, tol = c.reference()
        want = c.call(s, cache)
        within(want, ref, tol)
        meta = (c.i32(c.q_off), c.i32(c.start), c.i32(c.kv), c.tables.cuda(), cache, c.layer)
        torch.cuda.synchronize()
        outs = []
        for _ in range(20):
            with torch.cuda.stream(busy):
                for _ in range(4):
                    big[1].copy_(big[0], non_blocking=True)
            outs += [s.attend(c.q, *meta, max_q_len=1) for _ in range(10)]
        torch.cuda.synchronize()
        assert s.last_query_error() == (0, 0)
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,mem,H", [(130, 100, 2), (20, 3000, 1)])
def test_rows_summed_again_end_with_those_sums(pkg, D, n, mem, H):  # noqa: F811
    """A key that only the last query sees makes all other rows of its tile
    odd: their first sums, NaN in every dim, are stored over by a warp's other
    threads -- in the output (130 queries) and in parts of the keys (20)."""
    G = 4
    c = Paged(210 + n, D, H, G, 16, [n], [mem])
    ref, rl, tol = c.reference()
    last = c.kv[0] - 1
    b, o = int(c.tables[0, last // 16]), last % 16
    c.v[b, o] = math.nan
    c.sync_cache()
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        outs = []
        for _ in range(20):
            lse = torch.zeros(c.q.shape[:2], device="cuda")
            outs.append((c.call(s, cache, lse=lse), lse))
        assert s.last_query_error() == (0, 0)
    out, lse = outs[0]
    within(out[:n - 1], ref[:n - 1], tol[:n - 1])
    assert ((lse[:n - 1].double() - rl[:n - 1]).abs() <= 2.0 ** -14 + 2.0 ** -18 * rl[:n - 1].abs()).all()
    assert torch.isnan(out[n - 1]).all()
    for x, y in outs[1:]:
        assert torch.equal(x[:n - 1], out[:n - 1]) and torch.equal(y[:n - 1], lse[:n - 1])
