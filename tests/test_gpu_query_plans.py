"""Calls whose launch follows from bounds far from the lengths: block tables of
an engine's longest context, and long own keys behind a long prefix with few
KV heads."""
import pytest
import torch

from query_cases import Paged
from test_gpu_query import check_attend, make, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


def widen(c, width):
    """A table row as long as an engine's longest request; what lies behind a
    request's keys is no block."""
    t = torch.full((c.tables.shape[0], width), -7, dtype=torch.int32)
    t[:, :c.tables.shape[1]] = c.tables
    c.tables = t
    return c


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("n,mem,shared", [([1], [0], 0), ([1], [2100], 0), ([1, 1, 1], [5, 700, 90], 0),
                                          ([1] * 20, [(61 * r) % 500 for r in range(20)], 37),
                                          ([3, 1, 0, 2], [40, 0, 9, 300], 0), ([17, 40], [100, 3], 0)])
def test_tables_of_the_longest_context(pkg, D, n, mem, shared):  # noqa: F811
    for width in (8192, 1 << 16):  # 131 k and 1 M positions in blocks of 16
        check_attend(pkg, widen(Paged(500 + D, D, 1, 4, 16, n, mem, shared), width))


@pytest.mark.parametrize("D,H,R,shared,mem", [(128, 1, 2, 70001, [40000, 3]), (64, 2, 3, 65536, [0, 9000, 17]),
                                              (128, 1, 9, 20000, [3000 + 700 * r for r in range(9)])])
def test_long_own_keys_behind_a_long_prefix(pkg, D, H, R, shared, mem):  # noqa: F811
    assert shared * R * H * D * 4 >= 64 << 20
    check_attend(pkg, Paged(510 + D, D, H, 4, 16, [1] * R, mem, shared=shared, extra_rows=2))


def test_wide_tables_in_a_graph(pkg):  # noqa: F811
    """As an engine captures it: one graph for lengths that change between
    its replays."""
    D, H, G = 128, 2, 4
    c = widen(Paged(520, D, H, G, 16, [1] * 4, [900, 30, 2000, 400]), 8192)
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        start, kv, tables = c.i32(c.start), c.i32(c.kv), c.tables.cuda()
        out, off = torch.zeros(4, H * G, D, dtype=c.q.dtype, device="cuda"), c.i32(c.q_off)
        run = lambda o: s.attend(c.q, off, start, kv, tables, cache, c.layer, max_q_len=1, out=o)  # noqa: E731
        run(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(out)
        for cut in (0, 1, 29, 30):
            kv.copy_(c.i32([max(0, x - cut) for x in c.kv]))
            start.copy_(c.i32([max(0, x - cut - 1) for x in c.kv]))
            graph.replay()
            assert torch.equal(out, run(torch.zeros_like(out)))
        assert s.last_query_error() == (0, 0)
