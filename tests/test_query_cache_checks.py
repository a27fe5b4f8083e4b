"""append and attend refuse a cache that lacks what they would reach into, before anything is
launched: on the CPU, with tensors whose device number is -1 and a library
that only counts its calls."""
import pytest
import torch

BF = torch.bfloat16


class Counting:
    def __init__(self, B):
        self.B, self.calls = B, 0

    def __getattr__(self, name):
        if name.startswith("is_query_"):
            def call(*args):
                self.calls += 1
                return 0
            return call
        return getattr(self.B, name)


@pytest.fixture
def store(monkeypatch):
    from kv_cache_injection_gather_b200 import binding as B
    from kv_cache_injection_gather_b200 import store as S
    monkeypatch.setattr(S, "B", Counting(B))
    s = S.FactStore.__new__(S.FactStore)
    s.L, s.H, s.D, s.device = 4, 2, 64, -1
    s.handle, s.query, s._no_query = None, 1, 0
    s.count = lambda: S.B.calls
    yield s
    s.query = None


def described(layers, heads, dim, device=-1, known=True):
    from kv_cache_injection_gather_b200 import binding as B
    c = B.is_cache_t(block_size=16)
    if known:
        c.holds = (layers, heads, dim, device)
    return c


def calls(s, cache, layer):
    x, i = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, dtype=torch.int32)
    return (lambda: s.append(x, x, i, i.long(), cache, layer, stream=0),
            lambda: s.attend(x, torch.zeros(4, dtype=torch.int32), i, i, i[:, None].contiguous(), cache, layer, out=x,
                             stream=0))


@pytest.mark.parametrize("holds,layer", [((4, 1, 64), 0), ((4, 2, 32), 1), ((1, 2, 64), 1), ((3, 2, 64), 3),
                                         ((4, 2, 64, 0), 0)])
def test_a_cache_that_is_too_small_or_elsewhere_is_refused(store, holds, layer):
    for call in calls(store, described(*holds), layer):
        with pytest.raises(ValueError):
            call()
    assert store.count() == 0


def test_caches_that_hold_the_stores_rows_and_bare_structs_are_taken(store):
    for cache, layer in ((described(4, 2, 64), 3), (described(1, 2, 64), 0), (described(9, 3, 128), 3),
                         (described(4, 2, 64), 4), (described(0, 0, 0, known=False), 2)):
        before = store.count()
        for call in calls(store, cache, layer):
            call()
        assert store.count() == before + 3  # append; attend's work space and itself


@pytest.mark.gpu
def test_cache_desc_knows_its_tensors():
    import kv_cache_injection_gather_b200 as pkg
    k = torch.zeros(3, 5, 16, 2, 64, dtype=BF, device="cuda")
    assert pkg.cache_desc(k, k).holds == (3, 2, 64, 0)
    assert pkg.cache_desc(k, k, head_major=True).holds == (3, 16, 64, 0)
