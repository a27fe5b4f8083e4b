"""Decode's output against fp64 at the precision of its result: the
probabilities that meet the values are not a rounding of their own."""
import math

import pytest
import torch

from query_cases import Paged
from test_gpu_query import make, pkg, within  # noqa: F401

pytestmark = pytest.mark.gpu


def fine_tolerance(c, causal, scale=None, polynomial=0.0):
    """The bound of query_cases.attend_reference without its term for
    probabilities rounded to bf16 (2^-8 A) and, but for a prefix with a grid of
    its own, for exponentials by a polynomial (2^-17 A):

      * the result's own rounding: 2^-8 |out|;
      * a probability p as the sum of two bf16 values, p rounded and the
        remainder rounded: the remainder is at most 2^-8 p, its rounding 2^-8
        of that: 2^-16 A;
      * scores (4 c A) and sums over n keys as there, the latter twice, as
        the two values' products are sums of their own: 4 n 2^-24 A.
    """
    out, _, _ = c.reference(causal, scale)
    scale = 1 / math.sqrt(c.D) if scale is None else scale
    tol = torch.zeros_like(out)
    H, G, D = c.H, c.G, c.D
    for r in range(len(c.kv)):
        j = torch.arange(c.kv[r])
        if not len(j):
            continue
        blk = c.tables[r][(j // c.block)].long()
        if c.shared:
            blk = torch.where(j < c.shared, c.shared_blocks[(j // c.block).clamp(max=len(c.shared_blocks) - 1)].long(), blk)
        K, V = c.k[blk, j % c.block].double(), c.v[blk, j % c.block].double()
        for t in range(c.q_off[r], c.q_off[r + 1]):
            lim = min(c.kv[r], c.start[r] + t - c.q_off[r] + 1) if causal else c.kv[r]
            if lim <= 0:
                continue
            x = c.q[t].double().view(H, G, D)
            s = torch.einsum("hgd,nhd->hgn", x, K[:lim]) * scale
            S = (torch.einsum("hgd,nhd->hgn", x.abs(), K[:lim].abs()) * scale).amax(-1)
            e = 2.0 ** -24 * (D + 2) * S + 2.0 ** -22 * (s.abs().amax(-1) + 2)
            A = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), V[:lim].abs())
            tol[t] = (2.0 ** -8 * out[t].view(H, G, D).abs()
                      + A * (2.0 ** -16 + polynomial + 4 * e[..., None] + 4 * lim * 2.0 ** -24)).reshape(H * G, D)
    return out, tol


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 5, 16])
@pytest.mark.parametrize("n,mem,shared,block", [
    ([1, 1, 1, 1], [0, 17, 300, 1111], 0, 16),      # one cluster a unit
    ([1] * 40, [(97 * r) % 800 for r in range(40)], 37, 24),  # one CTA a unit
    ([1], [30011], 0, 16),                          # parts that a grid joins
    ([3, 1], [64, 700], 0, 5)])                     # rows that see less than their unit; key by key
def test_decode_at_the_results_precision(pkg, D, G, n, mem, shared, block):  # noqa: F811
    H = 2
    if max(n) * G > 16 and D != 256:
        n = [1] * len(n)  # (for more rows the probabilities are rounded there)
    c = Paged(400 + D + G, D, H, G, block, n, mem, shared, qscale=1.5)
    for causal in (True, False):
        out, tol = fine_tolerance(c, causal)
        with make(pkg, D, H) as s:
            got = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache), causal)
            assert s.last_query_error() == (0, 0)
        within(got, out, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_cancel(pkg, D):  # noqa: F811
    """Values of alternating sign: the result is far below the sum of the
    products' magnitudes, where rounded probabilities would show."""
    c = Paged(450 + D, D, 2, 4, 16, [1] * 3, [999, 1999, 400])
    sign = torch.where(torch.arange(c.block, device="cuda") % 2 == 0, 1.0, -1.0)[None, :, None, None]
    c.v.copy_((100 * sign + c.v.double()).to(c.v.dtype))
    c.q.mul_(0.25)  # nearly equal weights
    c.sync_cache()
    out, tol = fine_tolerance(c, True)
    with make(pkg, D, 2) as s:
        got = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache))
        assert s.last_query_error() == (0, 0)
    within(got, out, tol)


@pytest.mark.parametrize("D,shared,block", [(64, 520, 16), (128, 260, 16), (128, 275, 24)])
def test_decode_behind_a_prefix_at_the_results_precision(pkg, D, shared, block):  # noqa: F811
    """A prefix that has a grid of its own, by its bytes, in which four keys
    carry nearly all weight, nearly equally, with values that cancel."""
    R, H, G = 64, 8, 4
    assert shared * R * H * D * 4 >= 64 << 20
    c = Paged(460 + D, D, H, G, block, [1] * R, [r % 7 for r in range(R)], shared=shared)
    c.q.mul_(0.25)
    c.q[..., 0] = 8
    c.k[..., 0] = -80 / math.sqrt(D)  # e^-7 of the weight
    for i, j in enumerate((3, 50, 131, 200)):
        b, o = int(c.shared_blocks[j // block]), j % block
        c.k[b, o, :, 0] = 0
        c.v[b, o] += 100 * (-1) ** i
    c.sync_cache()
    out, tol = fine_tolerance(c, True, polynomial=2.0 ** -17)
    with make(pkg, D, H) as s:
        got = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache))
        assert s.last_query_error() == (0, 0)
    within(got, out, tol)
