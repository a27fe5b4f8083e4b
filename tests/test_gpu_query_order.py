"""The attention kernels' waits under load: the same call gives the same bits
while other work delays its copies."""
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
