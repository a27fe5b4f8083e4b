"""Scores that are NaN or +inf reach the rows that see them as NaN, in the
output and in the log-sum-exp, wherever their key stands in a tile."""
import math

import pytest
import torch

from query_cases import Paged
from test_gpu_query import make, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


def run(pkg, s, c, causal=False):  # noqa: F811
    lse = torch.zeros(c.q.shape[:2], device="cuda")
    out = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache), causal, lse=lse)
    assert s.last_query_error() == (0, 0)
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 20, 70])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_seen_key_that_is_not_finite(pkg, D, n, bad):  # noqa: F811
    """One element of one key of KV head 1, at every place of 16 in both
    halves of a tile: its heads' rows are NaN, the other head's as before."""
    H, G = 2, 4
    c = Paged(300 + n, D, H, G, 16, [n], [400])
    c.q.copy_(c.q.abs())  # with a key element of +inf: a score of +inf
    with make(pkg, D, H) as s:
        clean, clean_lse = run(pkg, s, c)
        assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
        for j in [*range(128, 144), *range(192, 208)]:
            b, o = int(c.tables[0, j // 16]), j % 16
            was = c.k_cache[c.layer, b, o, 1, 7].clone()
            c.k_cache[c.layer, b, o, 1, 7] = bad
            out, lse = run(pkg, s, c)
            c.k_cache[c.layer, b, o, 1, 7] = was
            assert torch.isnan(out[:, G:]).all(), (j, out[:, G:][~torch.isnan(out[:, G:])][:4])
            assert torch.isnan(lse[:, G:]).all(), (j, lse[:, G:][~torch.isnan(lse[:, G:])][:4])
            assert torch.equal(out[:, :G], clean[:, :G]) and torch.equal(lse[:, :G], clean_lse[:, :G])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_key_of_the_prefix_that_is_not_finite(pkg, bad):  # noqa: F811
    """The same for a prefix that has a grid of its own: all who see it."""
    R, H, G, D, shared = 40, 4, 4, 128, 2000
    kv = [shared + 9 + r for r in range(R)]
    kv[2] = 100  # does not see the key
    c = Paged(301, D, H, G, 16, [1] * R, [0] * R, shared=shared, kv=kv)
    c.q.copy_(c.q.abs())
    with make(pkg, D, H) as s:
        clean, clean_lse = run(pkg, s, c, True)
        for j in range(1024, 1040):
            b, o = int(c.shared_blocks[j // 16]), j % 16
            was = c.k_cache[c.layer, b, o, 1, 7].clone()
            c.k_cache[c.layer, b, o, 1, 7] = bad
            out, lse = run(pkg, s, c, True)
            c.k_cache[c.layer, b, o, 1, 7] = was
            sees = torch.tensor([r != 2 for r in range(R)], device="cuda")
            assert torch.isnan(out[sees, G:2 * G]).all() and torch.isnan(lse[sees, G:2 * G]).all(), j
            assert torch.equal(out[:, :G], clean[:, :G]) and torch.equal(out[:, 2 * G:], clean[:, 2 * G:])
            assert torch.equal(out[2], clean[2]) and torch.equal(lse[2], clean_lse[2])
